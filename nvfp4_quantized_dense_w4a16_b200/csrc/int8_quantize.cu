// Quantisation of bf16 rows to int8 with a scale for each row.
#include "int8.cuh"
#include "int8.h"
#include "launch.cuh"
#include "moe.h"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using namespace sm100;

// A row stays in registers between its largest magnitude and its codes: a group of
// `threads` threads (a warp or more of a CTA's 256, or the CTA) holds N vectors of 8
// values each; longer rows are read twice.  Bound by memory traffic, 3 bytes a value,
// for many rows; by its latency for few.  x is no __restrict__ pointer: the kernel ahead may be
// writing it while this one starts, which loads of data that never changes do not allow.
template <int N>
__global__ void __launch_bounds__(512)
    int8_quantize_kernel(const uint16_t* x, int64_t m, int64_t k, int64_t stride, int threads,
                         int8_t* codes, float* scales) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ uint32_t part[16];
  const int groups = blockDim.x / threads, g = threadIdx.x / threads, mine = threadIdx.x - g * threads;
  const int warps = threads / 32, first = g * warps;
  const int64_t row = blockIdx.x * (int64_t)groups + g;
  const bool in = row < m;
  const uint4* src = reinterpret_cast<const uint4*>(x + (in ? row : 0) * stride);
  uint2* dst = reinterpret_cast<uint2*>(codes + row * k);
  const int vecs = in ? (int)(k / 8) : 0;
  uint4 v[N];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = mine + i * threads;
    v[i] = at < vecs ? src[at] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) top = amax8_bf16(top, v[i]);
  for (int at = mine + N * threads; at < vecs; at += threads) top = amax8_bf16(top, src[at]);
  uint32_t a = __reduce_max_sync(0xffffffffu, amax_of_pair(top));
  if (warps > 1) {  // (the same for all groups)
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    for (int i = 0; i < warps; ++i) a = max(a, part[first + i]);
  }
  const Int8Row q(a);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = mine + i * threads;
    if (at < vecs) dst[at] = int8_encode8(q, v[i]);
  }
  for (int at = mine + N * threads; at < vecs; at += threads) dst[at] = int8_encode8(q, src[at]);
  if (in && mine == 0) scales[row] = q.scale;
}

template <int N>
cudaError_t launch_one(const void* x, int64_t m, int64_t k, int64_t stride, int threads, int8_t* codes, float* scales,
                       cudaStream_t s) {
  const int block = threads > 256 ? threads : 256 / threads * threads, groups = block / threads;
  return launch_pdl(int8_quantize_kernel<N>, dim3((unsigned)((m + groups - 1) / groups)), dim3(block), 0, s, static_cast<const uint16_t*>(x), m, k,
                    stride, threads, codes, scales);
}

}  // namespace

cudaError_t launch_int8_quantize(const void* x, int64_t m, int64_t k, int64_t stride, int8_t* codes, float* scales,
                                 cudaStream_t s) {
  ProfScope prof(s, "int8_quantize");
  // Few rows: two vectors a thread; many: four, so that a row's cost is shared by as many values.
  const int64_t vecs = k / 8;
  const bool few = m <= 2 * device_sms();
  const int per = few ? 2 : 4;
  const int64_t want = (vecs + 32 * per - 1) / (32 * per) * 32;
  const int threads = (int)(want < 512 ? want : 512);
  if (few && vecs <= 2 * 512) return launch_one<2>(x, m, k, stride, threads, codes, scales, s);
  return launch_one<4>(x, m, k, stride, threads, codes, scales, s);
}

}  // namespace ffn
