// Quantisation of bf16 rows to int8 with a scale for each row.
#include "int8.cuh"
#include "int8.h"
#include "launch.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using namespace sm100;

// A CTA per row: the row's largest magnitude, then its codes.  CHAINED: the next
// kernel is a product of this call, which waits before it reads the rows, and may
// start.  A quantisation by itself may be that of a weight, which a product reads
// without waiting: it lets nothing start before its end.
template <bool CHAINED>
__global__ void __launch_bounds__(256)
    int8_quantize_kernel(const uint16_t* __restrict__ x, int64_t k, int64_t stride, int8_t* __restrict__ codes,
                         float* __restrict__ scales) {
  griddep_wait();
  if (CHAINED) griddep_launch_dependents();
  __shared__ uint32_t part[8];
  const int64_t row = blockIdx.x;
  const uint4* src = reinterpret_cast<const uint4*>(x + row * stride);
  const int vecs = (int)(k / 8);
  uint32_t top = 0;
  for (int i = threadIdx.x; i < vecs; i += blockDim.x) top = amax8_bf16(top, src[i]);
  const uint32_t mine = __reduce_max_sync(0xffffffffu, amax_of_pair(top));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = mine;
  __syncthreads();
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, part[i]);
  const Int8Row q(a);
  uint2* dst = reinterpret_cast<uint2*>(codes + row * k);
  for (int i = threadIdx.x; i < vecs; i += blockDim.x) dst[i] = int8_encode8(q, src[i]);
  if (threadIdx.x == 0) scales[row] = q.scale;
}

}  // namespace

cudaError_t launch_int8_quantize(const void* x, int64_t m, int64_t k, int64_t stride, int8_t* codes, float* scales,
                                 bool chained, cudaStream_t s) {
  ProfScope prof(s, "int8_quantize");
  return launch_pdl(chained ? int8_quantize_kernel<true> : int8_quantize_kernel<false>, dim3((unsigned)m), dim3(256), 0, s, static_cast<const uint16_t*>(x), k, stride,
                    codes, scales);
}

}  // namespace ffn
