// First factor of the low-rank adapters for gfx950:
//   H[m][r] = bf16(scale[a] sum_k X[m,k] La[a][r,k]),  a = ids[m].
//
// Bound by reading X and the adapters in use once.  A workgroup takes 16 rows
// of X, finds their distinct adapters and forms, for each of those it is
// given, RT x 16 ranks for the rows that name it: its eight waves take the
// 64-wide K blocks in turn (two 16x16x32 bf16 MFMAs per 16 ranks and block),
// and their fp32 partial tiles meet in LDS, summed in wave order.  Rows of
// other adapters are not loaded (zeros in the operand), so each row of X is
// read once per RT x 16 ranks however the requests are mixed.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bf16.h"
#include "fp8gemm_routed.h"

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int WAVES = 8, ROWS = 16;

template <int RT>
__global__ __launch_bounds__(WAVES * 64) void lora_shrink_kernel(const uint16_t *X, const uint16_t *La,
                                                                 const int32_t *ids, const float *scale,
                                                                 uint16_t *H, int M, int K, int R, int G) {
  __shared__ v4f s_part[WAVES][RT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int fr = lane & 15, fg = lane >> 4;
  const int m0 = blockIdx.x * ROWS, r0 = blockIdx.y * RT * 16;
  // lanes fr, fr + 16, ... hold row fr's adapter; `first` marks the first row of each
  int id = m0 + fr < M ? ids[m0 + fr] : -1;
  if (id < 0 || id >= G) id = -1;
  bool first = id >= 0;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) first = first && !(i < fr && (int)lane_of((uint32_t)id, i) == id);
  unsigned todo = (unsigned)__ballot(first) & 0xFFFFu;
  const u32x4 zero = {0, 0, 0, 0};
  for (int n = 0; todo; todo &= todo - 1, ++n) {
    if (n % gridDim.z != blockIdx.z) continue;
    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    const bool mine = id == ad;
    const uint16_t *xp = X + (size_t)(m0 + fr) * K + fg * 8;
    const uint16_t *lp = La + ((size_t)ad * R + r0 + fr) * K + fg * 8;
    v4f acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int k = wave * 64; k < K; k += WAVES * 64) {
      u32x4 x[2], l[RT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[h] = mine ? *reinterpret_cast<const u32x4 *>(xp + k + h * 32) : zero;
#pragma unroll
        for (int i = 0; i < RT; ++i)
          l[i][h] = r0 + i * 16 + fr < R
                        ? *reinterpret_cast<const u32x4 *>(lp + (size_t)i * 16 * K + k + h * 32)
                        : zero;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < RT; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, l[i][h]),
                                                           __builtin_bit_cast(bf16x8, x[h]), acc[i], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) s_part[wave][i][lane] = acc[i];
    __syncthreads();
    // wave i sums the i-th 16 ranks: lane holds row fr's ranks 4 fg .. 4 fg + 3
    if (wave < RT) {
      v4f s = s_part[0][wave][lane];
#pragma unroll
      for (int v = 1; v < WAVES; ++v) s += s_part[v][wave][lane];
      const int r = r0 + wave * 16 + 4 * fg;
      if (mine && r < R) {  // R is a multiple of 8
        const float f = scale[ad];
        *reinterpret_cast<u32x2 *>(H + (size_t)(m0 + fr) * R + r) =
            u32x2{bf16_pair(f * s[0], f * s[1]), bf16_pair(f * s[2], f * s[3])};
      }
    }
    __syncthreads();
  }
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace

extern "C" int lora_shrink_bf16(const void *X, const void *La, const int32_t *ids, const float *scale,
                                void *H, int M, int K, int R, int G, void *stream) {
  if (M < 0 || K < 0 || R < 0 || G < 0) return FP8GEMM_INVALID_ARG;
  if (M == 0 || R == 0 || G == 0) return FP8GEMM_OK;
  if (!ids || !scale || !H || (K > 0 && (!X || !La))) return FP8GEMM_INVALID_ARG;
  if (K % 64 != 0 || R % 8 != 0 || R > 4096 || G > 4096 || (long long)M * R >= (1LL << 30))
    return FP8GEMM_UNSUPPORTED_SHAPE;
  if (!aligned(X, 16) || !aligned(La, 16) || !aligned(H, 16) || !aligned(ids, 4) || !aligned(scale, 4))
    return FP8GEMM_MISALIGNED;
  // Few row tiles: 16 ranks and one adapter a workgroup, so that the adapters'
  // rows stream through many CUs; many: a workgroup takes its rows' adapters
  // one after the other and 64 ranks at once, so X is read once.
  const int tiles = (M + ROWS - 1) / ROWS, r16 = (R + 15) / 16;
  const bool few = tiles < 64;
  const int rt = few ? 1 : std::min(4, r16);
  const int z = few ? ROWS : 1;
  const dim3 grid(tiles, (r16 + rt - 1) / rt, z);
  void *args[] = {&X, &La, &ids, &scale, &H, &M, &K, &R, &G};
  const void *f = rt == 1   ? reinterpret_cast<const void *>(&lora_shrink_kernel<1>)
                  : rt == 2 ? reinterpret_cast<const void *>(&lora_shrink_kernel<2>)
                  : rt == 3 ? reinterpret_cast<const void *>(&lora_shrink_kernel<3>)
                            : reinterpret_cast<const void *>(&lora_shrink_kernel<4>);
  return hipLaunchKernel(f, grid, dim3(WAVES * 64), args, 0, static_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? FP8GEMM_OK
             : FP8GEMM_LAUNCH_FAILED;
}
