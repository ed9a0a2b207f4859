// Grouped projection of many rows per expert on the tensor cores (prompts):
// one launch computes, for every expert, its rows (sorted by expert) times
// its NVFP4 weight.
//
// A persistent CTA per SM walks the tiles (128 rows of one expert) x (a pair
// of MMA operands of 128 weight rows: gate and up rows of the same columns, or
// 256 consecutive rows of a plain weight).  Per unit of two 64-element K chunks:
//   * one warp streams the weights' chunks (18432 B) by bulk copies
//     and one the rows' chunks (2 x 128 x 128 B, 128-byte swizzle) by TMA;
//   * two warpgroups, one per operand, decode the codes to bf16 and write
//     them to tensor memory, where they are the MMA's A operand (M = 128);
//   * two threads, one per operand, issue tcgen05.mma kind::f16 against
//     the same rows in shared memory (N = 128), each into its own fp32
//     accumulator.  A barrier wait, a fence and a commit cost an issuing thread
//     about 0.1 us each while its MMAs of 64 cycles drain: one thread with
//     one-chunk units kept the tensor pipe busy for half of the time;
//   * two further warpgroups (64 rows each) read a finished tile's
//     accumulators, one into registers and one into shared memory, hand them
//     back and run the epilogue while the next tile's MMAs proceed.
// The pair is what bounds the traffic: a row tile is read from L2 once per 256
// weight rows, 50 KB per unit of 1024 MMA cycles (50 B/clk per SM).
// Tensor memory: accumulators in columns 0..255, two A slots of a unit per
// operand in columns 256..511.  Every wait is bounded; on expiry a device
// error bit is raised and the CTA frees its tensor memory and exits.
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "launch.cuh"
#include "moe.h"
#include "moe_decode.cuh"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using namespace moe;
using namespace sm100;

__device__ int g_moe_device_error = 0;

// SiLU with the fast exponential and quotient: a few steps of fp32, and the
// product is rounded to bf16 right after.
__device__ __forceinline__ float silu_fast(float z) { return __fdividef(z, 1.0f + __expf(-z)); }

constexpr int kThreads = 640;
constexpr int kUnit = 2;  // K chunks per unit
constexpr int kXStages = 3, kWStages = 3, kASlots = 2;
constexpr int kTiles = 4;  // weight tiles of 64 rows per CTA tile: two per MMA operand
constexpr int kWStageBytes = kTiles * kUnit * kChunkBytes;  // [tile][chunk]
constexpr int kXChunkBytes = kTcTile * 128, kXStageBytes = kUnit * kXChunkBytes;
constexpr int kMine = kTcTile / 2;                      // rows of a tile per epilogue warpgroup
constexpr int kOpRows = 2 * kTileRows;                  // weight rows of an MMA operand
constexpr int kParkBytes = kMine * kOpRows * 4;       // one warpgroup's half of an accumulator
constexpr int kSmemW = kXStages * kXStageBytes;
constexpr int kSmemPark = kSmemW + kWStages * kWStageBytes;
constexpr int kSmemBar = kSmemPark + 2 * kParkBytes;
constexpr int kNumBars = 2 * kXStages + 2 * kWStages + 4 * kASlots + 2;
constexpr int kSmemAlloc = kSmemBar + kNumBars * 8 + 16 + 1024;  // slack for 1024-byte alignment
static_assert(kSmemAlloc <= 232448, "shared memory budget");
constexpr int kAColBase = 256;

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

struct TcExpertsArgs {
  ExpertsView w;
  MoePlan plan;
  void* out;
  int pairs_n;  // CTA tiles (two MMA operands) along the weight of an expert
};

struct TileInfo {
  int e, first, rows, wt;
};

__device__ __forceinline__ TileInfo tile_at(const TcExpertsArgs& a, int T) {
  const int tt = T / a.pairs_n;
  const int* p = a.plan.tiles + 1 + 3 * tt;
  return TileInfo{__ldcg(p), __ldcg(p + 1), __ldcg(p + 2), T % a.pairs_n};
}

// Wait that ignores the abort flag (in-flight copies must land before exit).
__device__ __forceinline__ bool drain(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) {
      atomicOr(&g_moe_device_error, 16);
      return false;
    }
  return true;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) experts_tc_kernel(const __grid_constant__ CUtensorMap xmap,
                                                                const TcExpertsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* xs = smem;
  uint8_t* wsm = smem + kSmemW;
  uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + kSmemBar);
  uint64_t* xempty = xfull + kXStages;
  uint64_t* wfull = xempty + kXStages;
  uint64_t* wempty = wfull + kWStages;
  uint64_t* afull = wempty + kWStages;     // [operand][slot]
  uint64_t* aempty = afull + 2 * kASlots;  // likewise
  uint64_t* accfull = aempty + 2 * kASlots;
  uint64_t* accempty = accfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accempty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = &g_moe_device_error;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kc = a.w.kc;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 2);  // one commit per MMA thread
    }
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], 8);
    }
    for (int s = 0; s < 2 * kASlots; ++s) {
      mbar_init(&afull[s], 4);
      mbar_init(&aempty[s], 1);
    }
    mbar_init(accfull, 2);
    mbar_init(accempty, 8);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 1 && lane == 0) tma_prefetch_desc(&xmap);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The kernel before this one (the sorting of the rows, or the gate and up
  // products) lets it start once it has itself waited for the ones before: the
  // plan is in L2.  So only the warp that reads that kernel's rows waits for it,
  // the weights are streamed and decoded ahead (20 experts of 1056 x 672, 111
  // rows: 36.0 -> 33.4 us), and all that is written follows from those rows.
  const int total = __ldcg(a.plan.tiles) * a.pairs_n;

  if (warp == 0) {
    // ------------------------------------------------------ weight producer
    if (lane == 0) {
      int u = 0;
      bool ok = true;
      for (int T = blockIdx.x; ok && T < total; T += gridDim.x) {
        const TileInfo ti = tile_at(a, T);
        const size_t tile_bytes = (size_t)kc * kChunkBytes;
        // Past the last tile, that tile stands in: its sums are not stored.
        const uint8_t* w[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const bool silu = MODE == (int)ExpertsOut::kSiluMul;
          const int tile = min(silu ? 2 * ti.wt + (i & 1) : kTiles * ti.wt + i, a.w.wtiles - 1);
          w[i] = a.w.tiles + ((size_t)(silu ? 2 * ti.e + (i >> 1) : ti.e) * a.w.wtiles + tile) * tile_bytes;
        }
        for (int c = 0; c < kc; c += kUnit, ++u) {
          const int s = u % kWStages;
          if (u >= kWStages && !mbar_wait(&wempty[s], ((u / kWStages) - 1) & 1, abort_flag, err, 1)) {
            ok = false;
            break;
          }
          const uint32_t bytes = min(kUnit, kc - c) * kChunkBytes;
          mbar_arrive_expect_tx(&wfull[s], kTiles * bytes);
#pragma unroll
          for (int i = 0; i < kTiles; ++i)
            bulk_load(wsm + s * kWStageBytes + i * kUnit * kChunkBytes, w[i] + (size_t)c * kChunkBytes, bytes, &wfull[s]);
        }
      }
      for (int r = max(0, u - kWStages); r < u; ++r) drain(&wfull[r % kWStages], (r / kWStages) & 1);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- row producer
    griddep_wait();
    griddep_launch_dependents();
    if (lane == 0) {
      int u = 0;
      bool ok = true;
      for (int T = blockIdx.x; ok && T < total; T += gridDim.x) {
        const TileInfo ti = tile_at(a, T);
        for (int c = 0; c < kc; c += kUnit, ++u) {
          const int s = u % kXStages, nc = min(kUnit, kc - c);
          if (u >= kXStages && !mbar_wait(&xempty[s], ((u / kXStages) - 1) & 1, abort_flag, err, 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&xfull[s], nc * kXChunkBytes);
          for (int j = 0; j < nc; ++j)
            tma_load_2d(xs + s * kXStageBytes + j * kXChunkBytes, &xmap, (c + j) * kChunkK, ti.first, &xfull[s]);
        }
      }
      for (int r = max(0, u - kXStages); r < u; ++r) drain(&xfull[r % kXStages], (r / kXStages) & 1);
    }
  } else if (warp < 4) {
    // ----------------------------------------------------------- MMA issuers
    // (the whole warp walks the loop and one elected lane issues: uniform
    // control flow keeps the descriptors in uniform registers)
    const int half = warp - 2;
    const uint32_t d = tmem + 128 * half;
    int u = 0, i = 0;
    bool ok = true;
    for (int T = blockIdx.x; ok && T < total; T += gridDim.x, ++i) {
      if (i > 0) {
        ok = mbar_wait(accempty, (i - 1) & 1, abort_flag, err, 2);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
      }
      // a tile with few rows needs few columns
      const uint32_t idesc = idesc_bf16_f32(kOpRows, min(kTcTile, (tile_at(a, T).rows + 15) & ~15));
      for (int c = 0; c < kc; c += kUnit, ++u) {
        const int sx = u % kXStages, sa = u % kASlots;
        // (the decode warps have waited for the rows as well)
        ok = mbar_wait(&afull[half * kASlots + sa], (u / kASlots) & 1, abort_flag, err, 2);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint64_t b = smem_desc_sw128(smem_u32(xs + sx * kXStageBytes));
        const uint32_t aslot = tmem + kAColBase + 128 * sa + 64 * half;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kUnit; ++j) {
            if (c + j >= kc) break;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(d, aslot + 32 * j + 8 * kk, b + j * (kXChunkBytes >> 4) + 2 * kk, idesc, (c | j | kk) ? 1u : 0u);
          }
          mma_commit(&aempty[half * kASlots + sa]);
          mma_commit(&xempty[sx]);
          if (c + kUnit >= kc) mma_commit(accfull);
        }
        __syncwarp();
      }
    }
  } else if (warp < 12) {
    // --------------------------------------------------------------- decode
    const int half = (warp - 4) >> 2, q = warp & 3, row = 32 * q + lane;
    const uint32_t col = tmem + ((uint32_t)(32 * q) << 16) + kAColBase + 64 * half;
    int u = 0;
    bool ok = true;
    for (int T = blockIdx.x; ok && T < total; T += gridDim.x) {
      for (int c = 0; c < kc; c += kUnit, ++u) {
        const int sw = u % kWStages, sa = u % kASlots, nc = min(kUnit, kc - c);
        ok = mbar_wait(&wfull[sw], (u / kWStages) & 1, abort_flag, err, 4);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint4 lo[kUnit], hi[kUnit];
        uint32_t sc[kUnit];
        const uint8_t* w = wsm + sw * kWStageBytes + (2 * half + (row >> 6)) * kUnit * kChunkBytes;
        const int r = row & 63;
#pragma unroll
        for (int j = 0; j < kUnit; ++j) {  // (a missing second chunk reads what the stage held before)
          lo[j] = *reinterpret_cast<const uint4*>(w + j * kChunkBytes + code_offset(r, 0, j));
          hi[j] = *reinterpret_cast<const uint4*>(w + j * kChunkBytes + code_offset(r, 1, j));
          sc[j] = *reinterpret_cast<const uint32_t*>(w + j * kChunkBytes + scale_offset(r, j));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&wempty[sw]);
#pragma unroll
        for (int j = 0; j < kUnit; ++j) {
          if (j >= nc) break;
          const uint32_t s2[4] = {scale_twice(sc[j], 0x4040), scale_twice(sc[j], 0x4141), scale_twice(sc[j], 0x4242),
                                  scale_twice(sc[j], 0x4343)};
          const uint32_t words[8] = {lo[j].x, lo[j].y, lo[j].z, lo[j].w, hi[j].x, hi[j].y, hi[j].z, hi[j].w};
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t o[4];
            decode8(words[i], s2[i >> 1], o);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * i + k] = o[k];
          }
          if (j == 0 && u >= kASlots) {  // the MMAs that read this slot two units ago are done
            ok = mbar_wait(&aempty[half * kASlots + sa], ((u / kASlots) - 1) & 1, abort_flag, err, 4);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st32(col + 128 * sa + 32 * j, v);
        }
        if (!ok) break;
        // the unit's rows, on the MMA thread's behalf
        ok = mbar_wait(&xfull[u % kXStages], (u / kXStages) & 1, abort_flag, err, 4);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&afull[half * kASlots + sa]);
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int g = (warp - 12) >> 2, q = warp & 3, row = 32 * q + lane;
    const int et = threadIdx.x - 384 - 128 * g;  // 0..127 within this warpgroup
    float* park = reinterpret_cast<float*>(smem + kSmemPark + g * kParkBytes);  // [kMine][128]
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + kMine * g;
    int i = 0;
    for (int T = blockIdx.x; T < total; T += gridDim.x, ++i) {
      const TileInfo ti = tile_at(a, T);
      const int first = ti.first + kMine * g, mine = min(kMine, ti.rows - kMine * g);  // may be <= 0
      const bool silu = MODE == (int)ExpertsOut::kSiluMul;
      const float gs0 = a.w.gs[silu ? 2 * ti.e : ti.e] * kUnscale;
      const float gs1 = silu ? a.w.gs[2 * ti.e + 1] * kUnscale : gs0;
      int pr[2] = {0, 0};  // the rows' pairs
      if (!silu)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (32 * h + lane < mine) pr[h] = __ldcg(a.plan.order + first + 32 * h + lane);
      bool ok = mbar_wait(accfull, i & 1, abort_flag, err, 8);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      float v[kMine];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t t[32];
        tmem_ld32(lane_addr + 128 + 32 * h, t);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) park[(32 * h + j) * kOpRows + row] = gs1 * __uint_as_float(t[j]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t t[32];
        tmem_ld32(lane_addr + 32 * h, t);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[32 * h + j] = gs0 * __uint_as_float(t[j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(accempty);
      if (silu) {
        // h = silu(g) * u, left as bf16 in the low half of u's own word
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          float* u = park + j * kOpRows + row;
          *reinterpret_cast<uint32_t*>(u) = f32_to_bf16_bits(silu_fast(v[j]) * *u);
        }
        // rows in sorted order, 16 bytes at a time (inter is a multiple of 32)
        named_bar_sync(1 + g, 128);
        const int64_t inter = a.w.n / 2, c0 = kOpRows * (int64_t)ti.wt;
        uint16_t* h = static_cast<uint16_t*>(a.out) + first * inter + c0;
        for (int idx = et; idx < mine * 16; idx += 128) {
          const int j = idx >> 4, ch = idx & 15;
          if (c0 + 8 * ch >= inter) continue;
          const uint4 p0 = *reinterpret_cast<const uint4*>(park + j * kOpRows + 8 * ch);
          const uint4 p1 = *reinterpret_cast<const uint4*>(park + j * kOpRows + 8 * ch + 4);
          *reinterpret_cast<uint4*>(h + j * inter + 8 * ch) =
              make_uint4(p0.x | (p0.y << 16), p0.z | (p0.w << 16), p1.x | (p1.y << 16), p1.z | (p1.w << 16));
        }
        named_bar_sync(1 + g, 128);
      } else {
        const int64_t c0 = 2 * kOpRows * (int64_t)ti.wt + row, c1 = c0 + kOpRows, n = a.w.n;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          if (j >= mine) break;
          const int64_t at = (int64_t)__shfl_sync(0xffffffffu, pr[j >> 5], j & 31) * n;
          if (MODE == (int)ExpertsOut::kF32) {
            float* y = static_cast<float*>(a.out) + at;
            if (c0 < n) y[c0] = v[j];
            if (c1 < n) y[c1] = park[j * kOpRows + row];
          } else {
            uint16_t* y = static_cast<uint16_t*>(a.out) + at;
            if (c0 < n) y[c0] = f32_to_bf16_bits(v[j]);
            if (c1 < n) y[c1] = f32_to_bf16_bits(park[j * kOpRows + row]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// xs[q, :] = x[order[q] / row_div, :] for the sorted positions q, a warp each.
// Behind the last expert's rows: zeros to the rows of y that have no expert.
__global__ void __launch_bounds__(256) moe_gather_kernel(const uint4* __restrict__ x, int row_div, MoePlan p,
                                                         int experts, int64_t pairs, int vecs, uint4* __restrict__ xs,
                                                         uint16_t* __restrict__ y, int64_t n) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t q = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (q >= pairs) return;
  const int64_t pair = p.order[q];
  if (q < p.offsets[experts]) {
    const uint4* src = x + (pair / row_div) * vecs;
    uint4* dst = xs + q * vecs;
    for (int i = lane; i < vecs; i += 32) dst[i] = __ldg(src + i);
  } else if (y) {
    for (int64_t c = lane; c < n; c += 32) y[pair * n + c] = 0;
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

template <int MODE>
cudaError_t launch_one(const CUtensorMap& map, const TcExpertsArgs& a, int grid, cudaStream_t s) {
  auto kern = experts_tc_kernel<MODE>;
  // set on every launch: the attribute belongs to the current device's context
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemAlloc, s, map, a);
}

}  // namespace

cudaError_t launch_moe_gather(const void* x, int row_div, const MoePlan& p, int experts, int64_t pairs, int64_t k,
                              void* xs, void* y, int64_t n, cudaStream_t s) {
  ProfScope prof(s, "moe_gather");
  return launch_pdl(moe_gather_kernel, dim3((unsigned)((pairs + 7) / 8)), dim3(256), 0, s,
                    static_cast<const uint4*>(x), row_div, p, experts, pairs, (int)(k / 8), static_cast<uint4*>(xs),
                    static_cast<uint16_t*>(y), n);
}

cudaError_t launch_experts_tc(const void* xs, const ExpertsView& w, const MoePlan& p, int64_t pairs, ExpertsOut mode,
                              void* out, cudaStream_t s) {
  auto enc = encode_fn();
  if (!enc) return cudaErrorInvalidValue;
  CUtensorMap map;
  // kTcTile rows behind the last pair belong to the buffer: no box leaves it
  cuuint64_t dims[2] = {(cuuint64_t)w.k, (cuuint64_t)(pairs + kTcTile)};
  cuuint64_t strides[1] = {(cuuint64_t)w.k * 2};
  cuuint32_t box[2] = {(cuuint32_t)kChunkK, (cuuint32_t)kTcTile};
  cuuint32_t estr[2] = {1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(xs), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  TcExpertsArgs a;
  a.w = w;
  a.plan = p;
  a.out = out;
  a.pairs_n = mode == ExpertsOut::kSiluMul ? (w.wtiles + 1) / 2 : (w.wtiles + kTiles - 1) / kTiles;
  const int64_t most = moe_max_tiles(pairs, w.experts, kTcTile) * a.pairs_n;
  const int sms = device_sms();
  const int grid = (int)(most < sms ? most : sms);
  ProfScope prof(s, mode == ExpertsOut::kSiluMul ? "experts_tc_silu" : "experts_tc");
  switch (mode) {
    case ExpertsOut::kSiluMul: return launch_one<(int)ExpertsOut::kSiluMul>(map, a, grid, s);
    case ExpertsOut::kF32: return launch_one<(int)ExpertsOut::kF32>(map, a, grid, s);
    default: return launch_one<(int)ExpertsOut::kBf16>(map, a, grid, s);
  }
}

cudaError_t read_moe_device_error(int* flags, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_moe_device_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_moe_device_error, &zero, sizeof(int));
  return e;
}

}  // namespace ffn
