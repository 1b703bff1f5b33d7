// LDS reads for waves that also have direct-to-LDS loads in flight.  The
// compiler lets an LDS read of its own wait for every such load (each might
// write what it reads), which would drain a ring that is filled ahead.  These
// wait for themselves, inside the statement; the caller waits (vmcnt) for the
// loads that fill what it reads.
#pragma once
#include "bf16.h"

static __device__ __forceinline__ uint32_t lds_at(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}
static __device__ __forceinline__ int lds_word(uint32_t at) {
  int v;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(at) : "memory");
  return v;
}
// the words at `at` and 128 bytes on
static __device__ __forceinline__ u32x2 lds_word_pair(uint32_t at) {
  u32x2 v;
  asm volatile("ds_read2_b32 %0, %1 offset0:0 offset1:32\n\ts_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(at) : "memory");
  return v;
}
// 16 bytes each at lo and hi + 2048 i, i < N: the two halves of N operand
// fragments, 16 rows of 128 bytes apart
template <int N>
static __device__ __forceinline__ void lds_fragments(uint32_t lo, uint32_t hi, u32x4 (&f)[N][2]) {
  static_assert(N >= 1 && N <= 4, "fragments at a time");
  if constexpr (N == 1) {
    asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %3\n\ts_waitcnt lgkmcnt(0)"
                 : "=&v"(f[0][0]), "=&v"(f[0][1]) : "v"(lo), "v"(hi) : "memory");
  } else if constexpr (N == 2) {
    asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\t"
                 "ds_read_b128 %2, %4 offset:2048\n\tds_read_b128 %3, %5 offset:2048\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(f[0][0]), "=&v"(f[0][1]), "=&v"(f[1][0]), "=&v"(f[1][1])
                 : "v"(lo), "v"(hi) : "memory");
  } else if constexpr (N == 3) {
    asm volatile("ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\t"
                 "ds_read_b128 %2, %6 offset:2048\n\tds_read_b128 %3, %7 offset:2048\n\t"
                 "ds_read_b128 %4, %6 offset:4096\n\tds_read_b128 %5, %7 offset:4096\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(f[0][0]), "=&v"(f[0][1]), "=&v"(f[1][0]), "=&v"(f[1][1]), "=&v"(f[2][0]), "=&v"(f[2][1])
                 : "v"(lo), "v"(hi) : "memory");
  } else {
    asm volatile("ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\t"
                 "ds_read_b128 %2, %8 offset:2048\n\tds_read_b128 %3, %9 offset:2048\n\t"
                 "ds_read_b128 %4, %8 offset:4096\n\tds_read_b128 %5, %9 offset:4096\n\t"
                 "ds_read_b128 %6, %8 offset:6144\n\tds_read_b128 %7, %9 offset:6144\n\t"
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(f[0][0]), "=&v"(f[0][1]), "=&v"(f[1][0]), "=&v"(f[1][1]), "=&v"(f[2][0]), "=&v"(f[2][1]),
                   "=&v"(f[3][0]), "=&v"(f[3][1])
                 : "v"(lo), "v"(hi) : "memory");
  }
}
