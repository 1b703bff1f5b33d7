// The products with adapters as fp8gemm.hip runs them, given H (the first
// factor's result): used by the calls in lora.hip.
#pragma once
#include <stdint.h>

struct LoraProduct {
  const void *A;
  const float *sa;  // FP8 only
  const void *B;
  const float *sb;
  const void *H, *Lb;
  const int32_t *ids;
  void *D;
  int M, N, K, R, G;
  bool fp8;
  void *stream;
};

// FP8GEMM_OK, an error status, or -1 where the base call alone is the answer
int lora_product_check(const LoraProduct &p);
// after a check that gave FP8GEMM_OK
int lora_product(const LoraProduct &p);
