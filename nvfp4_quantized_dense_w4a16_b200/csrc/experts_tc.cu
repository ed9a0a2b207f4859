// Grouped projection of many rows per expert on the tensor cores (prompts):
// one launch computes, for every expert, its rows (sorted by expert) times
// its NVFP4 weight.
//
// A persistent cluster of two CTAs (a pair of SMs) walks the tiles: up to 256
// rows of one expert x 256 weight rows, 128 per CTA (64 gate rows and the up
// rows of the same columns, or 128 consecutive rows of a plain weight).  Per
// unit of two 64-element K chunks, in each CTA:
//   * one warp streams its weights' chunks (9216 B) by bulk copies, and one its
//     half of the rows' chunks (2 x 128 x 128 B, 128-byte swizzle) by TMA, which
//     counts on a barrier of CTA 0 for both;
//   * two sets of four warps take the units in turn, decode the codes to bf16
//     and write them to tensor memory, where they are the MMA's A operand;
//   * one warp of CTA 0 issues tcgen05.mma cta_group::2 kind::f16 (M = 256, N =
//     the tile's rows) for both CTAs: each multiplies its weight rows by both
//     halves of the rows, into its own fp32 accumulator;
//   * two warpgroups (128 rows each) take a finished tile's accumulators, half
//     into shared memory and half into registers, hand them back and store the
//     results while the next tile's MMAs proceed.
// What bounds such a loop here is the decode, 670 cycles of the ALU pipe per 256
// weight rows and unit whatever the number of rows, and the traffic from L2.  A
// wide N spreads the decode over 256 rows (512 MMA cycles per 128 of them), and
// the pair halves the rows' traffic: 41 KB per unit of 1024 MMA cycles and CTA.
// One CTA by itself with 256 weight rows and N = 128 (50 KB per unit, the decode
// used once per 128 rows) ran at 1640 cycles per unit: 32768 pairs of 2048 x 1024
// took 478 us and take 433, 1024 pairs of 4096 x 12288 404 and 324 (tensor pipe
// 72% busy).  What is left is the way of a stage of rows: its MMAs' commit, the
// copy, the wait for it, three stages in all.  Four sets of decode warps change
// nothing (346 against 343 us).  What an
// arrival on the other CTA's barrier announces (rows, tensor memory) has been
// waited for before it, so it has no cluster scope, whose fences cost some 1000
// cycles a unit (732 us).
// Tensor memory: accumulators in columns 0..255, four A slots of a unit in
// columns 256..511.  Every wait is bounded; on expiry a device error bit is
// raised and the CTAs free their tensor memory and exit.
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
constexpr int kCtas = 2;  // of a cluster: they share a row tile, each holds half of it
constexpr int kXStages = 3, kWStages = 6, kASlots = 4;
constexpr int kSets = 2;                                // of four decode warps: they take the units in turn
// A wait tells a phase of its barrier from the next one only, so a set has to wait
// for every phase of the barriers that it waits on: a slot belongs to one set.
static_assert(kWStages % kSets == 0 && kASlots % kSets == 0, "stages and slots are the sets' own");
constexpr int kTiles = 2;                               // weight tiles of 64 rows per CTA tile
constexpr int kOpRows = kTiles * kTileRows;             // weight rows of a CTA: M of its half of the MMA
constexpr int kWStageBytes = kTiles * kUnit * kChunkBytes;  // [tile][chunk]
// Rows of a copy come in steps, each with its tensor map: a tile of few rows reads
// few (512 rows over 8 large experts: 342 -> 329 us).  Copies of 32 rows issued
// one after the other cost their issuing thread more than they save (433 us).
constexpr int kBoxStep = 32;
constexpr int kBoxes = kTcTile / kCtas / kBoxStep;
constexpr int kXChunkBytes = kTcTile / kCtas * 128, kXStageBytes = kUnit * kXChunkBytes;
constexpr int kMine = kTcTile / 2;                      // rows of a tile per epilogue warpgroup
constexpr int kHeld = kMine / 2;                        // of them in registers, and as many in shared memory
constexpr int kParkBytes = kHeld * kOpRows * 4;
constexpr int kSmemW = kXStages * kXStageBytes;
constexpr int kSmemPark = kSmemW + kWStages * kWStageBytes;
constexpr int kSmemBar = kSmemPark + 2 * kParkBytes;
constexpr int kNumBars = 2 * kXStages + 2 * kWStages + 2 * kASlots + 2;
constexpr int kSmemAlloc = kSmemBar + kNumBars * 8 + 16 + 1024;  // slack for 1024-byte alignment
static_assert(kSmemAlloc <= 232448, "shared memory budget");
constexpr int kAColBase = 256;

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// ------------------------------------------------- the pair of CTAs of a cluster

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Arrive on CTA 0's barrier that stands where `bar` does.
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// One MMA of both CTAs (256 weight rows): each gives its A, its half of the rows and its accumulator.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on `bar` of both CTAs once this thread's MMAs so far have completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// The address of CTA 0's barrier that stands where `bar` does.
__device__ __forceinline__ uint32_t in_first(uint64_t* bar) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
  return a;
}

// A copy into this CTA's shared memory that counts on a barrier of either CTA.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// Whether `ok` holds for all 128 threads that meet at barrier `id`.
__device__ __forceinline__ bool all_of_group(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(id)
      : "memory");
  return r != 0;
}

struct TcExpertsArgs {
  ExpertsView w;
  MoePlan plan;
  void* out;
  int wide_n;  // cluster tiles along the weight of an expert
};

struct RowMaps {
  CUtensorMap box[kBoxes];  // of kBoxStep, 2 kBoxStep, ... rows
};

struct TileInfo {
  int e, first, rows, wt;
};

__device__ __forceinline__ TileInfo tile_at(const TcExpertsArgs& a, int T, int rank) {
  const int tt = T / a.wide_n;
  const int* p = a.plan.tiles + 1 + 3 * tt;
  return TileInfo{__ldcg(p), __ldcg(p + 1), __ldcg(p + 2), kCtas * (T - tt * a.wide_n) + rank};
}

// Columns of the tile's MMA: a tile with few rows needs few.  Each CTA holds half of them.
__device__ __forceinline__ int tile_columns(int rows) { return min(kTcTile, (rows + 31) & ~31); }

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
__global__ void __cluster_dims__(kCtas) __launch_bounds__(kThreads, 1)
    experts_tc_kernel(const __grid_constant__ RowMaps maps, const TcExpertsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* xs = smem;
  uint8_t* wsm = smem + kSmemW;
  uint64_t* xfull = reinterpret_cast<uint64_t*>(smem + kSmemBar);
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
  const int kc = a.w.kc, rank = (int)cluster_rank();
  const int first_tile = blockIdx.x / kCtas, tile_step = gridDim.x / kCtas;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(&xfull[s], 1);  // (CTA 0's)
      mbar_init(&xempty[s], 1);
    }
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], 4);
    }
    for (int s = 0; s < kASlots; ++s) {
      mbar_init(&afull[s], 4 * kCtas);  // (CTA 0's)
      mbar_init(&aempty[s], 1);
    }
    mbar_init(accfull, 1);
    mbar_init(accempty, 8 * kCtas);  // (CTA 0's)
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_slot, 512);
  }
  if (warp == 1 && lane < kBoxes) tma_prefetch_desc(&maps.box[lane]);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // The kernel before this one (the sorting of the rows, or the gate and up
  // products) lets it start once it has itself waited for the ones before: the
  // plan is in L2.  So only the warp that reads that kernel's rows waits for it,
  // the weights are streamed and decoded ahead (20 experts of 1056 x 672, 203
  // rows: 36.0 -> 33.4 us), and all that is written follows from those rows.
  const int total = __ldcg(a.plan.tiles) * a.wide_n;

  if (warp == 0) {
    // ------------------------------------------------------ weight producer
    if (lane == 0) {
      int u = 0;
      bool ok = true;
      for (int T = first_tile; ok && T < total; T += tile_step) {
        const TileInfo ti = tile_at(a, T, rank);
        const size_t tile_bytes = (size_t)kc * kChunkBytes;
        // Past the last tile, that tile stands in: its sums are not stored.
        const uint8_t* w[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
          const bool silu = MODE == (int)ExpertsOut::kSiluMul;  // gate and up rows of the same 64 columns
          const int tile = min(silu ? ti.wt : kTiles * ti.wt + i, a.w.wtiles - 1);
          w[i] = a.w.tiles + ((size_t)(silu ? 2 * ti.e + i : ti.e) * a.w.wtiles + tile) * tile_bytes;
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
      for (int T = first_tile; ok && T < total; T += tile_step) {
        const TileInfo ti = tile_at(a, T, rank);
        const int half = tile_columns(ti.rows) / kCtas, row = ti.first + rank * half;
        const int box = (half + kBoxStep - 1) / kBoxStep;  // in steps
        for (int c = 0; c < kc; c += kUnit, ++u) {
          const int s = u % kXStages, nc = min(kUnit, kc - c);
          if (u >= kXStages && !mbar_wait(&xempty[s], ((u / kXStages) - 1) & 1, abort_flag, err, 1)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&xfull[s], kCtas * nc * box * kBoxStep * 128);  // both CTAs' copies
          for (int j = 0; j < nc; ++j)
            tma_load_pair(xs + s * kXStageBytes + j * kXChunkBytes, &maps.box[box - 1], (c + j) * kChunkK, row,
                          in_first(&xfull[s]));
        }
      }
      if (rank == 0)  // (CTA 1 leaves after this one)
        for (int r = max(0, u - kXStages); r < u; ++r) drain(&xfull[r % kXStages], (r / kXStages) & 1);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ MMA issuer
    // (CTA 0's, for both; the whole warp walks the loop and one elected lane
    // issues: uniform control flow keeps the descriptors in uniform registers)
    int u = 0, i = 0;
    bool ok = true;
    for (int T = first_tile; rank == 0 && ok && T < total; T += tile_step, ++i) {
      const uint32_t idesc = idesc_bf16_f32(kCtas * kOpRows, tile_columns(tile_at(a, T, rank).rows));
      if (i > 0) {
        ok = mbar_wait(accempty, (i - 1) & 1, abort_flag, err, 2);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
      }
      for (int c = 0; c < kc; c += kUnit, ++u) {
        const int sx = u % kXStages, sa = u % kASlots;
        ok = mbar_wait(&xfull[sx], (u / kXStages) & 1, abort_flag, err, 2) &&
             mbar_wait(&afull[sa], (u / kASlots) & 1, abort_flag, err, 2);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint64_t b = smem_desc_sw128(smem_u32(xs + sx * kXStageBytes));
        const uint32_t aslot = tmem + kAColBase + 32 * kUnit * sa;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kUnit; ++j) {
            if (c + j >= kc) break;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_pair(tmem, aslot + 32 * j + 8 * kk, b + j * (kXChunkBytes >> 4) + 2 * kk, idesc, (c | j | kk) ? 1u : 0u);
          }
          commit_pair(&aempty[sa]);
          commit_pair(&xempty[sx]);
          if (c + kUnit >= kc) commit_pair(accfull);
        }
        __syncwarp();
      }
    }
  } else if (warp >= 4 && warp < 4 + 4 * kSets) {
    // --------------------------------------------------------------- decode
    const int set = (warp - 4) >> 2, q = warp & 3, row = 32 * q + lane, r = row & 63;
    const uint32_t col = tmem + ((uint32_t)(32 * q) << 16) + kAColBase;
    const uint8_t* mine = wsm + (row >> 6) * kUnit * kChunkBytes;
    const int units = (kc + kUnit - 1) / kUnit;
    int base = 0;  // units of the tiles before
    bool ok = true;
    for (int T = first_tile; ok && T < total; T += tile_step, base += units) {
      for (int i = (set - base) & (kSets - 1); i < units; i += kSets) {
        const int u = base + i, sw = u % kWStages, sa = u % kASlots, nc = min(kUnit, kc - kUnit * i);
        ok = mbar_wait(&wfull[sw], (u / kWStages) & 1, abort_flag, err, 4);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint4 lo[kUnit], hi[kUnit];
        uint32_t sc[kUnit];
        const uint8_t* w = mine + sw * kWStageBytes;
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
          for (int k = 0; k < 8; ++k) {
            uint32_t o[4];
            decode8(words[k], s2[k >> 1], o);
#pragma unroll
            for (int z = 0; z < 4; ++z) v[4 * k + z] = o[z];
          }
          if (j == 0 && u >= kASlots) {  // the MMAs that read this slot before are done
            ok = mbar_wait(&aempty[sa], ((u / kASlots) - 1) & 1, abort_flag, err, 4);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st32(col + 32 * (kUnit * sa + j), v);
        }
        if (!ok) break;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&afull[sa]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------- epilogue
    const int g = (warp - 4 - 4 * kSets) >> 2, q = warp & 3, row = 32 * q + lane;
    float* park = reinterpret_cast<float*>(smem + kSmemPark + g * kParkBytes);  // [kHeld][128]
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + kMine * g;
    int i = 0;
    for (int T = first_tile; T < total; T += tile_step, ++i) {
      const TileInfo ti = tile_at(a, T, rank);
      const int first = ti.first + kMine * g, mine = min(kMine, ti.rows - kMine * g);  // may be <= 0
      const bool silu = MODE == (int)ExpertsOut::kSiluMul;
      const float gs0 = a.w.gs[silu ? 2 * ti.e : ti.e] * kUnscale;
      const float gs1 = silu ? a.w.gs[2 * ti.e + 1] * kUnscale : gs0;
      int pr[kMine / 32] = {};  // the rows' pairs
      if (!silu)
#pragma unroll
        for (int h = 0; h < kMine / 32; ++h)
          if (32 * h + lane < mine) pr[h] = __ldcg(a.plan.order + first + 32 * h + lane);
      bool ok = mbar_wait(accfull, i & 1, abort_flag, err, 8);
      ok = __all_sync(0xffffffffu, ok);
      ok = all_of_group(1 + g, ok);  // (the group's warps pass the same barriers)
      if (!ok) break;
      tc_fence_after();
      float v[kHeld];  // rows kHeld .. kMine - 1
#pragma unroll
      for (int h = 0; h < kHeld / 32; ++h) {
        uint32_t t[32];
        tmem_ld32(lane_addr + 32 * h, t);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) park[(32 * h + j) * kOpRows + row] = __uint_as_float(t[j]);
      }
#pragma unroll
      for (int h = 0; h < kHeld / 32; ++h) {
        uint32_t t[32];
        tmem_ld32(lane_addr + kHeld + 32 * h, t);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[32 * h + j] = __uint_as_float(t[j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(accempty);
      // Half of the rows at a time meet in shared memory, so that a warp stores
      // whole rows of the tile's columns (and the gate products of lanes 0..63
      // find the up products of the others).
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (part == 1)
#pragma unroll
          for (int j = 0; j < kHeld; ++j) park[j * kOpRows + row] = v[j];
        named_bar_sync(1 + g, 128);
        const int left = mine - kHeld * part;
        if (silu) {
          const int64_t inter = a.w.n / 2, col = kTileRows * (int64_t)ti.wt + 2 * lane;  // (inter is a multiple of 32)
          uint16_t* h = static_cast<uint16_t*>(a.out) + (first + kHeld * part) * inter + col;
          const int n = col < inter ? min(kHeld, left) : 0;
#pragma unroll 4
          for (int j = q; j < n; j += 4) {
            const float2 z = *reinterpret_cast<const float2*>(park + j * kOpRows + 2 * lane);
            const float2 u = *reinterpret_cast<const float2*>(park + j * kOpRows + kTileRows + 2 * lane);
            const uint32_t h0 = f32_to_bf16_bits(silu_fast(gs0 * z.x) * (gs1 * u.x)),
                           h1 = f32_to_bf16_bits(silu_fast(gs0 * z.y) * (gs1 * u.y));
            *reinterpret_cast<uint32_t*>(h + j * inter) = h0 | (h1 << 16);
          }
        } else {
          const int64_t col = kOpRows * (int64_t)ti.wt + 4 * lane, n = a.w.n;
#pragma unroll
          for (int t = 0; t < kHeld / 4; ++t) {
            const int j = 4 * t + q;
            if (4 * t >= left) break;
            const int64_t at = (int64_t)__shfl_sync(0xffffffffu, pr[2 * part + (t >> 3)], j & 31) * n + col;
            float4 z = *reinterpret_cast<const float4*>(park + j * kOpRows + 4 * lane);
            z.x *= gs0, z.y *= gs0, z.z *= gs0, z.w *= gs0;
            if (j >= left || col >= n) continue;
            if (MODE == (int)ExpertsOut::kF32) {  // (n is a multiple of 32)
              *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = z;
            } else {
              uint16_t* y = static_cast<uint16_t*>(a.out) + at;
              const uint16_t b[4] = {f32_to_bf16_bits(z.x), f32_to_bf16_bits(z.y), f32_to_bf16_bits(z.z),
                                     f32_to_bf16_bits(z.w)};
              if ((n & 3) == 0) {
                *reinterpret_cast<uint2*>(y) = make_uint2(b[0] | ((uint32_t)b[1] << 16), b[2] | ((uint32_t)b[3] << 16));
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (col + i < n) y[i] = b[i];
              }
            }
          }
        }
        named_bar_sync(1 + g, 128);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may arrive on its barriers or read its rows
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
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
cudaError_t launch_one(const RowMaps& maps, const TcExpertsArgs& a, int grid, cudaStream_t s) {
  auto kern = experts_tc_kernel<MODE>;
  // set on every launch: the attribute belongs to the current device's context
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), kSmemAlloc, s, maps, a);
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
  RowMaps maps;
  // kTcTile rows behind the last pair belong to the buffer: no box leaves it
  cuuint64_t dims[2] = {(cuuint64_t)w.k, (cuuint64_t)(pairs + kTcTile)};
  cuuint64_t strides[1] = {(cuuint64_t)w.k * 2};
  cuuint32_t estr[2] = {1, 1};
  for (int i = 0; i < kBoxes; ++i) {
    cuuint32_t box[2] = {(cuuint32_t)kChunkK, (cuuint32_t)(kBoxStep * (i + 1))};
    if (enc(&maps.box[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(xs), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  TcExpertsArgs a;
  a.w = w;
  a.plan = p;
  a.out = out;
  const int tiles = kCtas * (mode == ExpertsOut::kSiluMul ? 1 : kTiles);  // of 64 columns, a cluster
  a.wide_n = (w.wtiles + tiles - 1) / tiles;
  const int64_t most = moe_max_tiles(pairs, w.experts, kTcTile) * a.wide_n;
  const int clusters = device_sms() / kCtas;
  const int grid = kCtas * (int)(most < clusters ? most : clusters);
  ProfScope prof(s, mode == ExpertsOut::kSiluMul ? "experts_tc_silu" : "experts_tc");
  switch (mode) {
    case ExpertsOut::kSiluMul: return launch_one<(int)ExpertsOut::kSiluMul>(maps, a, grid, s);
    case ExpertsOut::kF32: return launch_one<(int)ExpertsOut::kF32>(maps, a, grid, s);
    default: return launch_one<(int)ExpertsOut::kBf16>(maps, a, grid, s);
  }
}

cudaError_t read_moe_device_error(int* flags, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_moe_device_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_moe_device_error, &zero, sizeof(int));
  return e;
}

}  // namespace ffn
