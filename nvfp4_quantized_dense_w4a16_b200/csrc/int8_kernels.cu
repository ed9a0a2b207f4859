// Kernels of the 8-bit integer layers: the rows' quantisation and the product.
#include "int8.cuh"
#include "int8.h"
#include "launch.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using namespace sm100;

// A CTA per row: the row's largest magnitude, then its codes.
__global__ void __launch_bounds__(256)
    int8_quantize_kernel(const uint16_t* __restrict__ x, int64_t k, int64_t stride, int8_t* __restrict__ codes,
                         float* __restrict__ scales) {
  griddep_wait();
  griddep_launch_dependents();
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

// 32 rows x 32 columns per CTA; with silu_mul the gate and the up sums of the columns.
constexpr int kRows = 32, kCols = 32, kDepth = 32;

template <bool SILU>
__global__ void __launch_bounds__(256) int8_product_kernel(const Int8Product p) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int xt[kRows][kDepth / 4 + 1], wt[SILU ? 2 * kCols : kCols][kDepth / 4 + 1];
  const int64_t cols = SILU ? p.n / 2 : p.n;
  const int64_t row_tiles = (p.m + kRows - 1) / kRows;
  const int64_t row0 = blockIdx.x % row_tiles * kRows, col0 = blockIdx.x / row_tiles * kCols;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  int acc[4] = {}, up[4] = {};
  for (int64_t k0 = 0; k0 < p.k; k0 += kDepth) {
    {
      const int r = threadIdx.x / 8, c = threadIdx.x % 8;
      xt[r][c] = row0 + r < p.m ? *reinterpret_cast<const int*>(p.x + (row0 + r) * p.k + k0 + 4 * c) : 0;
      wt[r][c] = col0 + r < cols ? *reinterpret_cast<const int*>(p.w + (col0 + r) * p.k + k0 + 4 * c) : 0;
      if (SILU)
        wt[kCols + r][c] = col0 + r < cols ? *reinterpret_cast<const int*>(p.w + (cols + col0 + r) * p.k + k0 + 4 * c) : 0;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kDepth / 4; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] = __dp4a(xt[ty + 8 * i][c], wt[tx][c], acc[i]);
        if (SILU) up[i] = __dp4a(xt[ty + 8 * i][c], wt[kCols + tx][c], up[i]);
      }
    __syncthreads();
  }
  const int64_t col = col0 + tx;
  if (col >= cols) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + ty + 8 * i;
    if (row >= p.m) break;
    float v = int8_scaled(acc[i], p.xs[row], p.ws[col]);
    if (SILU) v = int8_silu_mul(v, int8_scaled(up[i], p.xs[row], p.ws[cols + col]));
    if (!SILU && p.bias) v = __fadd_rn(v, bf16_bits_to_float(p.bias[col]));
    p.y[row * cols + col] = f32_to_bf16_bits(v);
  }
}

}  // namespace

cudaError_t launch_int8_quantize(const void* x, int64_t m, int64_t k, int64_t stride, int8_t* codes, float* scales,
                                 cudaStream_t s) {
  ProfScope prof(s, "int8_quantize");
  return launch_pdl(int8_quantize_kernel, dim3((unsigned)m), dim3(256), 0, s, static_cast<const uint16_t*>(x), k, stride,
                    codes, scales);
}

cudaError_t launch_int8_product(const Int8Product& p, cudaStream_t s) {
  const int64_t cols = p.silu_mul ? p.n / 2 : p.n;
  const dim3 grid((unsigned)(((p.m + kRows - 1) / kRows) * ((cols + kCols - 1) / kCols)));
  ProfScope prof(s, p.silu_mul ? "int8_gate_up" : "int8_product");
  if (p.silu_mul) return launch_pdl(int8_product_kernel<true>, grid, dim3(256), 0, s, p);
  return launch_pdl(int8_product_kernel<false>, grid, dim3(256), 0, s, p);
}

}  // namespace ffn
