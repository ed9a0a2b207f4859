// Grouped projection of many rows per expert on the tensor cores (prompts):
// one launch computes, for every expert, its rows (sorted by expert) times
// its NVFP4 weight.
//
// A persistent CTA per SM walks the tiles (128 rows of one expert) x (a pair
// of 128-row weight tiles: the gate and up tiles of the same columns, or two
// consecutive tiles of a plain weight).  Per 64-element K chunk:
//   * one warp streams the two weight tiles' chunks (9216 B) by bulk copies
//     and one the rows' chunk (128 x 128 B, 128-byte swizzle) by TMA;
//   * two warpgroups, one per weight tile, decode the codes to bf16 and write
//     them to tensor memory, where they are the MMA's A operand (M = 128);
//   * one thread issues tcgen05.mma kind::f16 of both halves against the same
//     row tile in shared memory (N = 128), into two fp32 accumulators;
//   * two further warpgroups read a finished tile's accumulators (64 rows
//     each), and run the epilogue while the next tile's MMAs proceed.
// The pair is what bounds the traffic: a row tile is read from L2 once per 256
// weight rows, 25 KB per chunk of 512 MMA cycles (50 B/clk per SM).
// Tensor memory: accumulators in columns 0..255, four A slots of both halves
// in columns 256..511.  Every wait is bounded; on expiry a device error bit is
// raised and the CTA frees its tensor memory and exits.
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
constexpr int kXStages = 6, kWStages = 6, kASlots = 4;
constexpr int kWStageBytes = 2 * kChunkBytes;

template <int BN>
struct Cfg {
  static constexpr int kXStageBytes = BN * 128;
  static constexpr int kSmemW = kXStages * kXStageBytes;
  static constexpr int kSmemStage = kSmemW + kWStages * kWStageBytes;  // epilogue staging, two warpgroups
  static constexpr int kStageBytes = (BN / 2) * 256;
  static constexpr int kSmemBar = kSmemStage + 2 * kStageBytes;
  static constexpr int kNumBars = 2 * kXStages + 2 * kWStages + 2 * kASlots + 2;
  static constexpr int kSmemBytes = kSmemBar + kNumBars * 8 + 16;
  static constexpr int kSmemAlloc = kSmemBytes + 1024;
  static_assert(kSmemAlloc <= 232448, "shared memory budget");
};
constexpr int kAColBase = 256;

struct TcExpertsArgs {
  ExpertsView w;
  MoePlan plan;
  void* out;
  int pairs_n;  // weight tile pairs per expert
};

struct TileInfo {
  int e, first, rows, wt;
};

__device__ __forceinline__ TileInfo tile_at(const TcExpertsArgs& a, int T) {
  const int tt = T / a.pairs_n;
  const int* p = a.plan.tiles + 1 + 3 * tt;
  return TileInfo{p[0], p[1], p[2], T % a.pairs_n};
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

template <int BN, int MODE>
__global__ void __launch_bounds__(kThreads, 1) experts_tc_kernel(const __grid_constant__ CUtensorMap xmap,
                                                                const TcExpertsArgs a) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* xs = smem;
  uint8_t* wsm = smem + C::kSmemW;
  uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + C::kSmemBar);
  uint64_t* xempty = xfull + kXStages;
  uint64_t* wfull = xempty + kXStages;
  uint64_t* wempty = wfull + kWStages;
  uint64_t* afull = wempty + kWStages;
  uint64_t* aempty = afull + kASlots;
  uint64_t* accfull = aempty + kASlots;
  uint64_t* accempty = accfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accempty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = &g_moe_device_error;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kc = a.w.kc;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], 8);
    }
    for (int s = 0; s < kASlots; ++s) {
      mbar_init(&afull[s], 8);
      mbar_init(&aempty[s], 1);
    }
    mbar_init(accfull, 1);
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
  griddep_launch_dependents();
  griddep_wait();  // the plan and the rows come from earlier kernels
  const int total = a.plan.tiles[0] * a.pairs_n;

  if (warp == 0) {
    // ------------------------------------------------------ weight producer
    if (lane == 0) {
      int u = 0;
      bool ok = true;
      for (int T = blockIdx.x; ok && T < total; T += gridDim.x) {
        const TileInfo ti = tile_at(a, T);
        const size_t tile_bytes = (size_t)kc * kChunkBytes;
        const uint8_t *w0, *w1;
        if (MODE == (int)ExpertsOut::kSiluMul) {
          w0 = a.w.tiles + ((size_t)ti.e * 2 * a.w.wtiles + ti.wt) * tile_bytes;
          w1 = w0 + a.w.wtiles * tile_bytes;
        } else {
          w0 = a.w.tiles + ((size_t)ti.e * a.w.wtiles + 2 * ti.wt) * tile_bytes;
          // an odd last tile: its chunks stand in for the missing half, whose sums are not stored
          w1 = 2 * ti.wt + 1 < a.w.wtiles ? w0 + tile_bytes : w0;
        }
        for (int c = 0; c < kc; ++c, ++u) {
          const int s = u % kWStages;
          if (u >= kWStages && !mbar_wait(&wempty[s], ((u / kWStages) - 1) & 1, abort_flag, err, 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&wfull[s], kWStageBytes);
          bulk_load(wsm + s * kWStageBytes, w0 + (size_t)c * kChunkBytes, kChunkBytes, &wfull[s]);
          bulk_load(wsm + s * kWStageBytes + kChunkBytes, w1 + (size_t)c * kChunkBytes, kChunkBytes, &wfull[s]);
        }
      }
      for (int r = max(0, u - kWStages); r < u; ++r) drain(&wfull[r % kWStages], (r / kWStages) & 1);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- row producer
    if (lane == 0) {
      int u = 0;
      bool ok = true;
      for (int T = blockIdx.x; ok && T < total; T += gridDim.x) {
        const TileInfo ti = tile_at(a, T);
        for (int c = 0; c < kc; ++c, ++u) {
          const int s = u % kXStages;
          if (u >= kXStages && !mbar_wait(&xempty[s], ((u / kXStages) - 1) & 1, abort_flag, err, 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&xfull[s], C::kXStageBytes);
          tma_load_2d(xs + s * C::kXStageBytes, &xmap, c * kChunkK, ti.first, &xfull[s]);
        }
      }
      for (int r = max(0, u - kXStages); r < u; ++r) drain(&xfull[r % kXStages], (r / kXStages) & 1);
    }
  } else if (warp == 2) {
    // ----------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(kTileRows, BN);
      int u = 0, i = 0;
      bool ok = true;
      for (int T = blockIdx.x; ok && T < total; T += gridDim.x, ++i) {
        if (i > 0 && !mbar_wait(accempty, (i - 1) & 1, abort_flag, err, 2)) break;
        tc_fence_after();
        for (int c = 0; c < kc; ++c, ++u) {
          const int sx = u % kXStages, sa = u % kASlots;
          if (!mbar_wait(&xfull[sx], (u / kXStages) & 1, abort_flag, err, 2) ||
              !mbar_wait(&afull[sa], (u / kASlots) & 1, abort_flag, err, 2)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t b = smem_desc_sw128(smem_u32(xs + sx * C::kXStageBytes));
          const uint32_t aslot = tmem + kAColBase + 64 * sa;
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16_ts(tmem + 128 * half, aslot + 32 * half + 8 * kk, b + 2 * kk, idesc, (c == 0 && kk == 0) ? 0u : 1u);
          mma_commit(&aempty[sa]);
          mma_commit(&xempty[sx]);
        }
        if (ok) mma_commit(accfull);
      }
    }
  } else if (warp >= 4 && warp < 12) {
    // --------------------------------------------------------------- decode
    const int half = (warp - 4) >> 2, q = warp & 3, row = 32 * q + lane;
    const uint32_t col = tmem + ((uint32_t)(32 * q) << 16) + kAColBase + 32 * half;
    int u = 0;
    bool ok = true;
    for (int T = blockIdx.x; ok && T < total; T += gridDim.x) {
      for (int c = 0; c < kc; ++c, ++u) {
        const int sw = u % kWStages, sa = u % kASlots;
        ok = mbar_wait(&wfull[sw], (u / kWStages) & 1, abort_flag, err, 4);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* w = wsm + sw * kWStageBytes + half * kChunkBytes;
        const uint4 lo = *reinterpret_cast<const uint4*>(w + 16 * row);
        const uint4 hi = *reinterpret_cast<const uint4*>(w + 2048 + 16 * row);
        const uint32_t sc = *reinterpret_cast<const uint32_t*>(w + 4096 + 16 * lane + 4 * q);
        __syncwarp();
        if (lane == 0) mbar_arrive(&wempty[sw]);
        const uint32_t s01 = scale_pair(sc & 0xffffu), s23 = scale_pair(sc >> 16);
        const uint32_t words[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t o[4];
          decode8(words[j], __byte_perm(j < 4 ? s01 : s23, 0, (j & 2) ? 0x3232 : 0x1010), o);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * j + i] = o[i];
        }
        if (u >= kASlots) {  // the MMAs that read this slot four chunks ago are done
          ok = mbar_wait(&aempty[sa], ((u / kASlots) - 1) & 1, abort_flag, err, 4);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
        tmem_st32(col + 64 * sa, v);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&afull[sa]);
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------- epilogue
    const int g = (warp - 12) >> 2, q = warp & 3, row = 32 * q + lane;
    const int et = threadIdx.x - 384 - 128 * g;  // 0..127 within this warpgroup
    constexpr int kMine = BN / 2;                // rows of the tile this warpgroup takes
    uint16_t* stage = reinterpret_cast<uint16_t*>(smem + C::kSmemStage + g * C::kStageBytes);  // [kMine][128]
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16);
    int i = 0;
    bool ok = true;
    for (int T = blockIdx.x; ok && T < total; T += gridDim.x, ++i) {
      const TileInfo ti = tile_at(a, T);
      const int j0 = kMine * g;                       // first row of the tile
      const int mine = min(kMine, ti.rows - j0);      // may be <= 0
      float gs0, gs1;
      if (MODE == (int)ExpertsOut::kSiluMul) {
        gs0 = a.w.gs[2 * ti.e] * kUnscale;
        gs1 = a.w.gs[2 * ti.e + 1] * kUnscale;
      } else {
        gs0 = gs1 = a.w.gs[ti.e] * kUnscale;
      }
      ok = mbar_wait(accfull, i & 1, abort_flag, err, 8);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      for (int c = 0; c < kMine; c += 32) {
        uint32_t v0[32], v1[32];
        tmem_ld32(lane_addr + j0 + c, v0);
        tmem_ld32(lane_addr + 128 + j0 + c, v1);
        tmem_ld_wait();
        if (c + 32 >= kMine) {  // the accumulators are read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(accempty);
        }
        if (c >= mine) continue;
        const int n = min(32, mine - c);
        if (MODE == (int)ExpertsOut::kSiluMul) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float z = gs0 * __uint_as_float(v0[j]);
            stage[(c + j) * 128 + row] = f32_to_bf16_bits(silu_fast(z) * (gs1 * __uint_as_float(v1[j])));
          }
        } else if (MODE == (int)ExpertsOut::kF32) {
          float* y = static_cast<float*>(a.out);
          const int p = lane < n ? a.plan.order[ti.first + j0 + c + lane] : 0;
          const int64_t col0 = 256 * (int64_t)ti.wt + row, col1 = col0 + 128;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (j >= n) break;
            float* yr = y + (int64_t)__shfl_sync(0xffffffffu, p, j) * a.w.n;
            if (col0 < a.w.n) yr[col0] = gs0 * __uint_as_float(v0[j]);
            if (col1 < a.w.n) yr[col1] = gs0 * __uint_as_float(v1[j]);
          }
        } else {
          uint16_t* y = static_cast<uint16_t*>(a.out);
          const int p = lane < n ? a.plan.order[ti.first + j0 + c + lane] : 0;
          const int64_t col0 = 256 * (int64_t)ti.wt + row, col1 = col0 + 128;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (j >= n) break;
            uint16_t* yr = y + (int64_t)__shfl_sync(0xffffffffu, p, j) * a.w.n;
            if (col0 < a.w.n) yr[col0] = f32_to_bf16_bits(gs0 * __uint_as_float(v0[j]));
            if (col1 < a.w.n) yr[col1] = f32_to_bf16_bits(gs0 * __uint_as_float(v1[j]));
          }
        }
      }
      if (MODE == (int)ExpertsOut::kSiluMul) {
        // h rows in sorted order, 16 bytes at a time (inter is a multiple of 32)
        named_bar_sync(1 + g, 128);
        const int64_t inter = a.w.n / 2;
        uint16_t* h = static_cast<uint16_t*>(a.out) + (int64_t)(ti.first + j0) * inter + 128 * (int64_t)ti.wt;
        for (int idx = et; idx < mine * 16; idx += 128) {
          const int j = idx >> 4, ch = idx & 15;
          if (128 * (int64_t)ti.wt + 8 * ch < inter)
            *reinterpret_cast<uint4*>(h + j * inter + 8 * ch) =
                *reinterpret_cast<const uint4*>(stage + j * 128 + 8 * ch);
        }
        named_bar_sync(1 + g, 128);
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

// xs[q, :] = x[order[q] / row_div, :] for the sorted positions q.
__global__ void __launch_bounds__(256) moe_gather_kernel(const uint4* __restrict__ x, int row_div, MoePlan p,
                                                         int experts, int64_t pairs, int vecs,
                                                         uint4* __restrict__ xs) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t q = blockIdx.x * (int64_t)(blockDim.x >> 5) + (threadIdx.x >> 5);
  if (q >= p.offsets[experts]) return;
  const uint4* src = x + (int64_t)(p.order[q] / row_div) * vecs;
  uint4* dst = xs + q * vecs;
  for (int i = threadIdx.x & 31; i < vecs; i += 32) dst[i] = __ldg(src + i);
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

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

template <int BN, int MODE>
cudaError_t launch_one(const CUtensorMap& map, const TcExpertsArgs& a, int grid, cudaStream_t s) {
  auto kern = experts_tc_kernel<BN, MODE>;
  // set on every launch: the attribute belongs to the current device's context
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BN>::kSmemAlloc);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), Cfg<BN>::kSmemAlloc, s, map, a);
}

}  // namespace

cudaError_t launch_moe_gather(const void* x, int row_div, const MoePlan& p, int experts, int64_t pairs, int64_t k,
                              void* xs, cudaStream_t s) {
  ProfScope prof(s, "moe_gather");
  return launch_pdl(moe_gather_kernel, dim3((unsigned)((pairs + 7) / 8)), dim3(256), 0, s,
                    static_cast<const uint4*>(x), row_div, p, experts, pairs, (int)(k / 8), static_cast<uint4*>(xs));
}

cudaError_t launch_experts_tc(const void* xs, const ExpertsView& w, const MoePlan& p, int64_t pairs, ExpertsOut mode,
                              void* out, cudaStream_t s) {
  constexpr int BN = kTcTile;
  auto enc = encode_fn();
  if (!enc) return cudaErrorInvalidValue;
  CUtensorMap map;
  // kTcTile rows behind the last pair belong to the buffer: no box leaves it
  cuuint64_t dims[2] = {(cuuint64_t)w.k, (cuuint64_t)(pairs + kTcTile)};
  cuuint64_t strides[1] = {(cuuint64_t)w.k * 2};
  cuuint32_t box[2] = {(cuuint32_t)kChunkK, (cuuint32_t)BN};
  cuuint32_t estr[2] = {1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(xs), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  TcExpertsArgs a;
  a.w = w;
  a.plan = p;
  a.out = out;
  a.pairs_n = mode == ExpertsOut::kSiluMul ? w.wtiles : (w.wtiles + 1) / 2;
  const int64_t most = moe_max_tiles(pairs, w.experts, BN) * a.pairs_n;
  const int sms = sm_count();
  const int grid = (int)(most < sms ? most : sms);
  ProfScope prof(s, mode == ExpertsOut::kSiluMul ? "experts_tc_silu" : "experts_tc");
  switch (mode) {
    case ExpertsOut::kSiluMul: return launch_one<BN, (int)ExpertsOut::kSiluMul>(map, a, grid, s);
    case ExpertsOut::kF32: return launch_one<BN, (int)ExpertsOut::kF32>(map, a, grid, s);
    default: return launch_one<BN, (int)ExpertsOut::kBf16>(map, a, grid, s);
  }
}

cudaError_t read_moe_device_error(int* flags, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_moe_device_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_moe_device_error, &zero, sizeof(int));
  return e;
}

}  // namespace ffn
