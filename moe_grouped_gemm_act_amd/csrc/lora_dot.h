// One rank of one row of the adapters' first factor: X[m] . La[ad][r] over a
// wave (uniform result).  U 16-byte pieces of each row at a time, 512 elements
// each over the wave; pieces past K read zeros and move nothing.
#pragma once
#include "bf16.h"

template <int U>
static __device__ __forceinline__ float lora_dot(const uint16_t *X, const uint16_t *La, int m, int r, int ad,
                                                 int K, int R, int lane) {
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t *>(X + (size_t)m * K), 0, (int)((uint32_t)K * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t rl = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t *>(La + ((size_t)ad * R + r) * K), 0, (int)((uint32_t)K * 2), 0x00020000);
  float acc[2] = {0.f, 0.f};
  for (uint32_t k = 0; k < (uint32_t)K * 2; k += U * 1024) {
    u32x4 x[U], l[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      x[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, k + u * 1024 + lane * 16, 0, 0));
      l[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rl, k + u * 1024 + lane * 16, 0, 0));
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[0] = __builtin_fmaf(bf16_lo(x[u][e]), bf16_lo(l[u][e]), acc[0]);
        acc[1] = __builtin_fmaf(bf16_hi(x[u][e]), bf16_hi(l[u][e]), acc[1]);
      }
  }
  return wave_sum(acc[0] + acc[1]);
}
