// Products of few rows with the NVFP4 weights of the experts picked for them
// (decode), the plan that sorts the rows by expert, and the weighted sum of
// the experts' outputs.
#include "common.cuh"
#include "launch.cuh"
#include "moe.h"
#include "moe_decode.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using namespace moe;
using sm100::griddep_launch_dependents;
using sm100::griddep_wait;

// ---------------------------------------------------------------- the plan

constexpr int kPlanThreads = 1024;

// One CTA: a histogram of the ids, its prefix sums, and the scatter of the
// pairs.  The order of an expert's rows follows the atomics; no result
// depends on it, as every row is computed by itself.
__global__ void __launch_bounds__(kPlanThreads) moe_plan_kernel(const int32_t* __restrict__ ids, int pairs, int E,
                                                               int tile_rows, MoePlan p) {
  extern __shared__ int plan_smem[];
  int* count = plan_smem;       // [E]
  int* start = plan_smem + E;   // [E]
  int* tile0 = plan_smem + 2 * E;
  griddep_wait();
  griddep_launch_dependents();
  for (int e = threadIdx.x; e < E; e += blockDim.x) count[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int at = 0, tiles = 0;
    for (int e = 0; e < E; ++e) {
      start[e] = at;
      tile0[e] = tiles;
      p.offsets[e] = at;
      at += count[e];
      tiles += (count[e] + tile_rows - 1) / tile_rows;
    }
    p.offsets[E] = at;
    p.tiles[0] = tiles;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int* t = p.tiles + 1 + 3 * tile0[e];
    for (int r = 0; r < count[e]; r += tile_rows, t += 3) {
      t[0] = e;
      t[1] = start[e] + r;
      t[2] = min(tile_rows, count[e] - r);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int e = ids[i];
    if (e >= 0 && e < E) p.order[atomicAdd(&start[e], 1)] = i;
  }
}

// ------------------------------------------------------ products, few rows

constexpr int kRowsWarps = 8;

struct RowsArgs {
  const uint16_t* x;  // [., k] bf16; pair p reads row p / row_div
  int row_div;
  ExpertsView w;
  MoePlan plan;
  void* out;  // row p: bf16 or fp32 [n_out]
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One CTA: 32 weight rows of one expert (16 gate rows and their up rows) times
// up to 8 of its rows, all of K; the warps take 128-element steps of K in turn
// and their sums are added in warp order.  Lane (g, t) = (lane / 4, lane % 4)
// reads 32 consecutive K elements of four weight rows, 32 apart in the tile,
// straight into registers and the same elements of row g of x.  The MMA sums over K in any order, so "k" of the fragments is
// whatever the four lanes of a quad hold, and no data moves between lanes.
template <int MODE>
__global__ void __launch_bounds__(kRowsWarps * 32) experts_rows_kernel(const RowsArgs a) {
  __shared__ float red[kRowsWarps][8][32];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr bool kPair = MODE == (int)ExpertsOut::kSiluMul;
  // tile rows of the four weight rows: r0 + 32 * j, j = 0..3; gate and up: r0 + 32 * (j & 1) of either tile
  const int tile = blockIdx.x / (kPair ? 8 : 4), r8 = 8 * (blockIdx.x & 3), j64 = kPair ? 64 * ((blockIdx.x >> 2) & 1) : 0;
  const int r0 = r8 + g + j64;
  const int ntiles = a.plan.tiles[0];
  const int64_t k = a.w.k;
  const int steps = (a.w.kc + 1) / 2;
  for (int slot = blockIdx.y; slot < ntiles; slot += gridDim.y) {
    const int e = a.plan.tiles[1 + 3 * slot], first = a.plan.tiles[2 + 3 * slot], rows = a.plan.tiles[3 + 3 * slot];
    const size_t tile_bytes = (size_t)a.w.kc * kChunkBytes;
    const uint8_t* wt = a.w.tiles + ((size_t)e * (kPair ? 2 : 1) * a.w.wtiles + tile) * tile_bytes;
    const size_t second = kPair ? a.w.wtiles * tile_bytes : 64 * 16;  // from rows j = 0, 1 to rows j = 2, 3
    const uint16_t* xr = g < rows ? a.x + (size_t)(a.plan.order[first + g] / a.row_div) * k : nullptr;
    float acc[2][4] = {};
    for (int s = warp; s < steps; s += kRowsWarps) {
      const int c = 2 * s + (t >> 1);
      uint4 cw[4], sc = make_uint4(0, 0, 0, 0), xv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) cw[j] = xv[j] = make_uint4(0, 0, 0, 0);
      if (c < a.w.kc) {
        const uint8_t* base = wt + (size_t)c * kChunkBytes;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          cw[j] = __ldg(reinterpret_cast<const uint4*>(base + (t & 1) * 2048 + 16 * (r0 + 32 * (j & 1)) + (j >> 1) * second));
        if (kPair) {  // the scales of rows r8 + g + {0, 32, 64, 96} stand together
          const uint2 s0 = __ldg(reinterpret_cast<const uint2*>(base + 4096 + 16 * (r8 + g) + j64 / 8));
          const uint2 s1 = __ldg(reinterpret_cast<const uint2*>(base + second + 4096 + 16 * (r8 + g) + j64 / 8));
          sc = make_uint4(s0.x, s0.y, s1.x, s1.y);
        } else {
          sc = __ldg(reinterpret_cast<const uint4*>(base + 4096 + 16 * (r8 + g)));
        }
        const int64_t k0 = 128 * (int64_t)s + 32 * t;
        if (xr && k0 < k)
#pragma unroll
          for (int j = 0; j < 4; ++j) xv[j] = *reinterpret_cast<const uint4*>(xr + k0 + 8 * j);
      }
      const uint32_t scw[4] = {sc.x, sc.y, sc.z, sc.w};
      uint32_t s01[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s01[j] = scale_pair((scw[j] >> (16 * (t & 1))) & 0xffffu);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t d[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t word = w == 0 ? cw[j].x : w == 1 ? cw[j].y : w == 2 ? cw[j].z : cw[j].w;
          decode8(word, __byte_perm(s01[j], 0, w < 2 ? 0x1010 : 0x3232), d[j]);
        }
        const uint32_t b[4] = {xv[w].x, xv[w].y, xv[w].z, xv[w].w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_16816(acc[0], d[0][2 * h], d[1][2 * h], d[0][2 * h + 1], d[1][2 * h + 1], b[2 * h], b[2 * h + 1]);
          mma_16816(acc[1], d[2][2 * h], d[3][2 * h], d[2][2 * h + 1], d[3][2 * h + 1], b[2 * h], b[2 * h + 1]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) red[warp][i][lane] = acc[i >> 2][i & 3];
    __syncthreads();
    // accumulator i of lane (g, t): weight row 8a + g + 32 * (i / 2), x row 2t + (i & 1)
    const int og = threadIdx.x & 7, on = (threadIdx.x >> 3) & 7, oj = threadIdx.x >> 6;  // row, token, 32-row group
    if (on < rows && (!kPair || oj < 2)) {
      const int src = 4 * og + (on >> 1), i = 2 * oj + (on & 1);
      const int64_t p = a.plan.order[first + on];
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) v += red[w][i][src];
      if (kPair) {
        float u = 0.0f;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) u += red[w][i + 4][src];
        const int64_t inter = a.w.n / 2, col = kTileRows * (int64_t)tile + r8 + og + j64 + 32 * oj;
        if (col < inter)
          static_cast<uint16_t*>(a.out)[p * inter + col] =
              f32_to_bf16_bits(silu_f32(a.w.gs[2 * e] * kUnscale * v) * (a.w.gs[2 * e + 1] * kUnscale * u));
      } else {
        const int64_t col = kTileRows * (int64_t)tile + r8 + og + 32 * oj;
        if (col < a.w.n) {
          v *= a.w.gs[e] * kUnscale;
          if (MODE == (int)ExpertsOut::kF32)
            static_cast<float*>(a.out)[p * a.w.n + col] = v;
          else
            static_cast<uint16_t*>(a.out)[p * a.w.n + col] = f32_to_bf16_bits(v);
        }
      }
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------- weighted sum

__global__ void __launch_bounds__(256) moe_combine_kernel(const float* __restrict__ y,
                                                          const int32_t* __restrict__ ids,
                                                          const float* __restrict__ weights, int64_t m, int top_k,
                                                          int experts, int64_t hidden, uint16_t* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t quads = hidden / 4;
  const int64_t idx = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if (idx >= m * quads) return;
  const int64_t row = idx / quads, c = 4 * (idx % quads);
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j = 0; j < top_k; ++j) {
    const int64_t p = row * top_k + j;
    const float w = weights[p];
    const int e = ids[p];
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (e >= 0 && e < experts) v = *reinterpret_cast<const float4*>(y + p * hidden + c);
    s.x = fmaf(w, v.x, s.x);
    s.y = fmaf(w, v.y, s.y);
    s.z = fmaf(w, v.z, s.z);
    s.w = fmaf(w, v.w, s.w);
  }
  *reinterpret_cast<uint2*>(out + row * hidden + c) =
      make_uint2((uint32_t)f32_to_bf16_bits(s.x) | ((uint32_t)f32_to_bf16_bits(s.y) << 16),
                 (uint32_t)f32_to_bf16_bits(s.z) | ((uint32_t)f32_to_bf16_bits(s.w) << 16));
}

__global__ void __launch_bounds__(256) experts_zero_kernel(const int32_t* __restrict__ ids, int64_t pairs,
                                                           int experts, int64_t n, uint16_t* __restrict__ y) {
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t p = blockIdx.x; p < pairs; p += gridDim.x) {
    const int e = ids[p];
    if (e >= 0 && e < experts) continue;
    for (int64_t c = threadIdx.x; c < n; c += blockDim.x) y[p * n + c] = 0;
  }
}

}  // namespace

cudaError_t launch_moe_plan(const int32_t* ids, int64_t pairs, int experts, int tile_rows, const MoePlan& p,
                            cudaStream_t s) {
  ProfScope prof(s, "moe_plan");
  return launch_pdl(moe_plan_kernel, dim3(1), dim3(kPlanThreads), 3 * sizeof(int) * experts, s, ids, (int)pairs,
                    experts, tile_rows, p);
}

cudaError_t launch_experts_rows(const void* x, int row_div, const ExpertsView& w, const MoePlan& p, int64_t pairs,
                                ExpertsOut mode, void* out, cudaStream_t s) {
  RowsArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.row_div = row_div;
  a.w = w;
  a.plan = p;
  a.out = out;
  const int64_t tiles = moe_max_tiles(pairs, w.experts, kRowsTile);
  const dim3 grid((unsigned)((w.gate_up ? 8 : 4) * w.wtiles), (unsigned)(tiles < 65535 ? tiles : 65535)), block(kRowsWarps * 32);
  ProfScope prof(s, mode == ExpertsOut::kSiluMul ? "experts_rows_silu" : "experts_rows");
  switch (mode) {
    case ExpertsOut::kSiluMul: return launch_pdl(experts_rows_kernel<(int)ExpertsOut::kSiluMul>, grid, block, 0, s, a);
    case ExpertsOut::kF32: return launch_pdl(experts_rows_kernel<(int)ExpertsOut::kF32>, grid, block, 0, s, a);
    default: return launch_pdl(experts_rows_kernel<(int)ExpertsOut::kBf16>, grid, block, 0, s, a);
  }
}

cudaError_t launch_moe_combine(const float* y, const int32_t* ids, const float* weights, int64_t m, int top_k,
                               int experts, int64_t hidden, void* out, cudaStream_t s) {
  ProfScope prof(s, "moe_combine");
  const int64_t blocks = (m * (hidden / 4) + 255) / 256;
  return launch_pdl(moe_combine_kernel, dim3((unsigned)blocks), dim3(256), 0, s, y, ids, weights, m, top_k, experts,
                    hidden, static_cast<uint16_t*>(out));
}

cudaError_t launch_experts_zero(const int32_t* ids, int64_t pairs, int experts, int64_t n, void* y, cudaStream_t s) {
  ProfScope prof(s, "experts_zero");
  return launch_pdl(experts_zero_kernel, dim3((unsigned)(pairs < 65536 ? pairs : 65536)), dim3(256), 0, s, ids, pairs,
                    experts, n, static_cast<uint16_t*>(y));
}

}  // namespace ffn
