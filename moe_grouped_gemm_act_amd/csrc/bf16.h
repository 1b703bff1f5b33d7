// bf16 values as bit patterns, and reductions over a wave, shared by the
// routing kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

static __device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
static __device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// fp32 -> bf16 bits, round to nearest even; NaN -> quiet NaN of its sign
static __device__ __forceinline__ uint32_t bf16_of(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return ((u >> 16) & 0x8000u) | 0x7FC0u;
  u += 0x7FFFu + ((u >> 16) & 1u);
  return u >> 16;
}
static __device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return bf16_of(lo) | (bf16_of(hi) << 16);
}

// x with the lanes of each 16-lane row exchanged: l ^ 1, l ^ 2, and the
// mirrors of 8 and of 16 lanes.  After an operation with each in turn every
// lane of a row holds the row's result.
template <int CTRL>
static __device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
}
constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_HALF_MIRROR = 0x141, DPP_MIRROR = 0x140;

static __device__ __forceinline__ uint32_t lane_of(uint32_t x, int l) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, l);
}

// over each row of 16 lanes, in every lane of it
static __device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, dpp<DPP_XOR1>(x));
  x = max(x, dpp<DPP_XOR2>(x));
  x = max(x, dpp<DPP_HALF_MIRROR>(x));
  return max(x, dpp<DPP_MIRROR>(x));
}
static __device__ __forceinline__ float row_sum(float f) {
  f += __uint_as_float(dpp<DPP_XOR1>(__float_as_uint(f)));
  f += __uint_as_float(dpp<DPP_XOR2>(__float_as_uint(f)));
  f += __uint_as_float(dpp<DPP_HALF_MIRROR>(__float_as_uint(f)));
  return f + __uint_as_float(dpp<DPP_MIRROR>(__float_as_uint(f)));
}

// the greatest of the wave's values (uniform)
static __device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = row_max(x);
  return max(max(lane_of(x, 0), lane_of(x, 16)), max(lane_of(x, 32), lane_of(x, 48)));
}

// the wave's sum, in one fixed order (uniform)
static __device__ __forceinline__ float wave_sum(float f) {
  const uint32_t u = __float_as_uint(row_sum(f));
  return (__uint_as_float(lane_of(u, 0)) + __uint_as_float(lane_of(u, 16))) +
         (__uint_as_float(lane_of(u, 32)) + __uint_as_float(lane_of(u, 48)));
}

// Whether bf16 values seen in pairs are all finite: the greatest magnitude in
// each half, as an integer (infinities and NaN have exponents of all ones).
struct bf16_peak {
  typedef unsigned short us2 __attribute__((ext_vector_type(2)));
  us2 top = {0, 0};
  __device__ __forceinline__ void see(u32x4 v) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      top = __builtin_elementwise_max(top, __builtin_bit_cast(us2, (uint32_t)(v[i] & 0x7FFF7FFFu)));
  }
  __device__ __forceinline__ bool finite() const { return top[0] < 0x7F80 && top[1] < 0x7F80; }
};
