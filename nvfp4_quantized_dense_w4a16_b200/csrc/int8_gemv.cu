// Products of the 8-bit integer layers for one row of x, on the CUDA cores.
//
// Bound by the stream of the weights, and, as one token's products are short, by
// what happens before and after it.  So one launch does it all: a thread holds the
// codes of its places in K for every weight row that its CTA takes, which it makes
// itself from a bf16 row (whose largest magnitude is a maximum over the CTA), and the
// first weights are under way before it waits for the kernel ahead that makes the row.
// Four products an instruction; a warp's sum is one reduction of integers.
// In a graph, from a bf16 row (from codes): 4096 x 4096 5.4 us (4.5), 24576 x 4096 18.3
// (17.3, 5.8 TB/s), 4096 x 12288 11.2 (9.0); two rows, quantised and multiplied on the
// tensor cores, take 8.9, 21.0 and 13.9.  Two rows so took 8.3, 23.6 and 16.1, four 12.5,
// 37 and 14.
#include <algorithm>

#include "int8.cuh"
#include "int8.h"
#include "launch.cuh"
#include "moe.h"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using namespace sm100;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBlockRows = 128;  // weight rows between two looks at the sums
constexpr int kVecBytes = 16;

struct GemvArgs {
  const void* x;    // int8 codes with xs, else bf16
  const float* xs;
  const int8_t* w;
  const float* ws;
  const uint16_t* bias;
  uint16_t* y;
  int64_t k, cols;   // cols of y; with silu_mul the weight has 2 * cols rows
  int per_cta;       // columns of y of a CTA
  int lanes;         // threads along K: a power of two from 32 on
  bool first;        // (Int8Product::first)
};

// Past L1, as read-only data: what the kernel ahead of a call's first launch may still write is not read before its end,
// by nobody on this SM (ordinary loads: 4096 x 4096 6.3 us for 5.3, 24576 x 4096 19.4 for 18.1).
__device__ __forceinline__ int4 load_weights(const int8_t* p) {
  int4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// V: vectors of 16 codes of K for a thread; U weight rows are under way at a time.
template <int V, bool SILU>
__global__ void __launch_bounds__(kThreads, 2) int8_gemv_kernel(const GemvArgs a) {
  constexpr int U = V == 1 ? 8 : V == 2 ? 4 : 2;
  __shared__ int part[kBlockRows][kWarps];
  __shared__ uint32_t top_part[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = kThreads / a.lanes;                 // of threads, each with a weight row at a time
  const int g = threadIdx.x / a.lanes, at = threadIdx.x & (a.lanes - 1);
  const int warps = a.lanes / 32, in_group = at >> 5;    // warps of a group
  const int vecs = (int)(a.k / kVecBytes);
  const int64_t col0 = (int64_t)blockIdx.x * a.per_cta;
  const int cols = (int)min((int64_t)a.per_cta, a.cols - col0);
  const int rows = SILU ? 2 * cols : cols;               // weight rows: gate and up of a column in turn
  bool in[V];
#pragma unroll
  for (int v = 0; v < V; ++v) in[v] = at + v * a.lanes < vecs;

  int4 w[U][V];
  auto fetch = [&](int first, int end) {  // weight rows first, first + groups, ...
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = first + u * groups;
      const int64_t row = SILU ? col0 + (r >> 1) + (r & 1 ? a.cols : 0) : col0 + r;
      const int8_t* p = a.w + row * a.k + at * kVecBytes;
#pragma unroll
      for (int v = 0; v < V; ++v)
        w[u][v] = r < end && in[v] ? load_weights(p + v * a.lanes * kVecBytes) : make_int4(0, 0, 0, 0);
    }
  };
  const int blocks = (rows + kBlockRows - 1) / kBlockRows;
  if (a.first) griddep_wait();
  fetch(g, min(rows, kBlockRows));
  griddep_wait();
  griddep_launch_dependents();

  // The codes of x at this thread's places, and its scale.
  int4 x[V];
  float scale;
  if (a.xs) {
    scale = *a.xs;
#pragma unroll
    for (int v = 0; v < V; ++v)
      x[v] = in[v] ? *reinterpret_cast<const int4*>(static_cast<const int8_t*>(a.x) + (at + v * a.lanes) * kVecBytes) : make_int4(0, 0, 0, 0);
  } else {
    // (read twice, the second time from the cache next by: registers hold the first weights)
    auto read = [&](int v, int half) {
      return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + (at + v * a.lanes) * kVecBytes)[half];
    };
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (in[v]) top = amax8_bf16(amax8_bf16(top, read(v, 0)), read(v, 1));
    top = __reduce_max_sync(0xffffffffu, amax_of_pair(top));
    if (lane == 0) top_part[warp] = top;
    __syncthreads();
    const Int8Row q(__reduce_max_sync(0xffffffffu, top_part[lane & (kWarps - 1)]));
    scale = q.scale;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = make_int4(0, 0, 0, 0);
      if (in[v]) {
        const uint2 lo = int8_encode8(q, read(v, 0)), hi = int8_encode8(q, read(v, 1));
        x[v] = make_int4((int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y);
      }
    }
  }

  for (int b = 0; b < blocks; ++b) {
    const int first = b * kBlockRows, end = min(rows, first + kBlockRows);
    for (int r0 = first + g; r0 < end; r0 += U * groups) {
      if (r0 != g) fetch(r0, end);  // (the first are there)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * groups;
        if (r >= end) break;
        int s = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
          s = __dp4a(w[u][v].x, x[v].x, __dp4a(w[u][v].y, x[v].y, __dp4a(w[u][v].z, x[v].z, __dp4a(w[u][v].w, x[v].w, s))));
        s = __reduce_add_sync(0xffffffffu, s);
        if (lane == 0) part[r - first][in_group] = s;
      }
    }
    __syncthreads();
    // An output a thread: the sums of its warps, then what every kernel does to a sum.
    const int outs = SILU ? (end - first) / 2 : end - first;
    for (int o = threadIdx.x; o < outs; o += kThreads) {
      const int64_t col = col0 + (SILU ? first / 2 : first) + o;
      int s = 0, up = 0;
      for (int q = 0; q < warps; ++q) {
        s += part[SILU ? 2 * o : o][q];
        if (SILU) up += part[SILU ? 2 * o + 1 : o][q];
      }
      float v = int8_scaled(s, scale, a.ws[col]);
      if (SILU)
        v = int8_silu_mul(v, int8_scaled(up, scale, a.ws[a.cols + col]));
      else if (a.bias)
        v = __fadd_rn(v, bf16_bits_to_float(a.bias[col]));
      a.y[col] = f32_to_bf16_bits(v);
    }
    __syncthreads();
  }
}

template <int V>
cudaError_t launch_one(const GemvArgs& a, bool silu, int grid, cudaStream_t s) {
  if (silu) return launch_pdl(int8_gemv_kernel<V, true>, dim3(grid), dim3(kThreads), 0, s, a);
  return launch_pdl(int8_gemv_kernel<V, false>, dim3(grid), dim3(kThreads), 0, s, a);
}

constexpr int kMaxVecs = 4;  // of a thread: they stay in registers

struct GemvShape {
  int lanes = 0, vecs = 0, per_cta, grid;  // (GemvArgs); vectors a thread
};
GemvShape gemv_shape(int64_t cols, int64_t k, bool silu_mul) {
  GemvShape g;
  // Threads along K and vectors a thread: the fewest idle places, then the most threads.
  const int vecs = (int)(k / kVecBytes);
  int least = INT32_MAX;
  for (int lanes = kThreads; lanes >= 32; lanes /= 2) {
    const int need = (vecs + lanes - 1) / lanes;
    if (need <= kMaxVecs && lanes * need < least) least = lanes * need, g.lanes = lanes, g.vecs = need;
  }
  // Two CTAs an SM share the columns evenly; each group of threads has a weight row at least.
  const int64_t ctas = 2 * (int64_t)device_sms(), groups = kThreads / g.lanes;
  g.per_cta = (int)std::max((cols + ctas - 1) / ctas, silu_mul ? (groups + 1) / 2 : groups);
  g.grid = (int)((cols + g.per_cta - 1) / g.per_cta);
  return g;
}

}  // namespace

bool int8_gemv_serves(int64_t m, int64_t k) { return m == 1 && k <= kMaxVecs * kThreads * kVecBytes; }

cudaError_t launch_int8_gemv(const Int8Product& p, cudaStream_t s) {
  const int64_t cols = p.silu_mul ? p.n / 2 : p.n;
  const GemvShape g = gemv_shape(cols, p.k, p.silu_mul);
  const GemvArgs a{p.x, p.xs, p.w, p.ws, p.bias, p.y, p.k, cols, g.per_cta, g.lanes, p.first};
  ProfScope prof(s, p.silu_mul ? "int8_gate_up" : "int8_product");
  switch (g.vecs) {
    case 1: return launch_one<1>(a, p.silu_mul, g.grid, s);
    case 2: return launch_one<2>(a, p.silu_mul, g.grid, s);
    case 3: return launch_one<3>(a, p.silu_mul, g.grid, s);
    default: return launch_one<kMaxVecs>(a, p.silu_mul, g.grid, s);
  }
}

ffn_int8_plan int8_gemv_plan(int64_t n, int64_t k, bool silu_mul) {
  const GemvShape g = gemv_shape(silu_mul ? n / 2 : n, k, silu_mul);
  const int rows = silu_mul ? 2 * g.per_cta : g.per_cta;
  return ffn_int8_plan{FFN_INT8_ROW, 1, rows, 1, g.grid, (rows + kBlockRows - 1) / kBlockRows};
}

}  // namespace ffn
