// Host-side declarations of the 8-bit integer layers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ffn_nvfp4.h"

namespace ffn {

// codes and scales of bf16 rows of k columns (a multiple of 8), row i at i * stride.
cudaError_t launch_int8_quantize(const void* x, int64_t m, int64_t k, int64_t stride, int8_t* codes, float* scales,
                                 cudaStream_t s);

// One projection of int8 rows.  Plain: y bf16 [m, n].  With silu_mul the weight
// holds n / 2 gate rows, then n / 2 up rows, and y is h bf16 [m, n / 2].
struct Int8Product {
  const void* x;  // int8 codes with their scales xs; for launch_int8_gemv also bf16, without
  const float* xs;
  int64_t m;
  const int8_t* w;
  const float* ws;
  const uint16_t* bias;  // bf16 [n] or null
  int64_t n, k;
  uint16_t* y;
  bool silu_mul;
  // The first launch of a call: what is before it in the stream may be writing the
  // weights.  A later one starts when an earlier one of the call has waited for all
  // that, and reads weights ahead of its own wait.
  bool first;
};
cudaError_t launch_int8_product(const Int8Product& p, cudaStream_t s);
// What these two choose for a product of n weight rows (gate and up rows, with silu_mul).
ffn_int8_plan int8_product_plan(int64_t m, int64_t n, int64_t k, bool silu_mul);
ffn_int8_plan int8_gemv_plan(int64_t n, int64_t k, bool silu_mul);
// The same for one row, bf16 as well, whose quantisation is part of it.
bool int8_gemv_serves(int64_t m, int64_t k);
cudaError_t launch_int8_gemv(const Int8Product& p, cudaStream_t s);
// Error bits of these kernels' bounded waits, as read_device_error.
cudaError_t read_int8_device_error(int* flags, bool clear);
cudaError_t read_norm_device_error(int* flags, bool clear);

}  // namespace ffn
