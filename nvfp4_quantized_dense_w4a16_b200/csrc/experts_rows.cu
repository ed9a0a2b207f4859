// Products of few rows with the NVFP4 weights of the experts picked for them
// (decode), the plan that sorts the rows by expert, and the weighted sum of
// the experts' outputs.
#include <cooperative_groups.h>

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

// ---------------------------------------------------------------- the plan

constexpr int kPlanThreads = 1024;
constexpr int kPlanEach = 4;  // ids a thread takes at a time

// One CTA, or a cluster of them that share the pairs: a histogram of the ids,
// its prefix sums over the experts (and over the cluster's CTAs, read from
// their shared memory), and the scatter of the pairs.  Pairs without an expert
// form the bucket behind the last expert.  The order of an expert's rows
// follows the atomics; no result depends on it, as every row is computed by
// itself.
__global__ void __launch_bounds__(kPlanThreads) moe_plan_kernel(const int32_t* __restrict__ ids, int pairs, int E,
                                                               int tile_rows, MoePlan p) {
  namespace cg = cooperative_groups;
  extern __shared__ int plan_smem[];
  int* count = plan_smem;              // [E + 1]
  int* start = plan_smem + E + 1;      // [E + 1]
  __shared__ int2 warp_sums[kPlanThreads / 32];
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  griddep_wait();
  griddep_launch_dependents();
  for (int e = threadIdx.x; e <= E; e += kPlanThreads) count[e] = 0;
  __syncthreads();
  const int each = (pairs + ctas - 1) / ctas, p0 = min(pairs, rank * each), p1 = min(pairs, p0 + each);
  for (int i0 = p0 + threadIdx.x; i0 < p1; i0 += kPlanEach * kPlanThreads) {
    int e[kPlanEach];
#pragma unroll
    for (int j = 0; j < kPlanEach; ++j) e[j] = i0 + j * kPlanThreads < p1 ? ids[i0 + j * kPlanThreads] : -1;
#pragma unroll
    for (int j = 0; j < kPlanEach; ++j)
      if (i0 + j * kPlanThreads < p1) atomicAdd(&count[e[j] >= 0 && e[j] < E ? e[j] : E], 1);
  }
  cluster.sync();
  // thread e: its expert's rows in all CTAs, and in those before this one (E + 1 may exceed the block by one)
  int at = 0, tiles = 0;  // of the chunks of experts before
  for (int e0 = 0; e0 <= E; e0 += kPlanThreads) {
    const int e = e0 + threadIdx.x;
    int all = 0, before = 0;
    if (e <= E)
      for (int c = 0; c < ctas; ++c) {
        const int n = ctas == 1 ? count[e] : *cluster.map_shared_rank(&count[e], c);
        before += c < rank ? n : 0;
        all += n;
      }
    const int mine = e < E ? (all + tile_rows - 1) / tile_rows : 0;
    int2 sum = make_int2(all, mine);  // inclusive scan over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum.x, o), y = __shfl_up_sync(0xffffffffu, sum.y, o);
      if ((threadIdx.x & 31) >= o) sum.x += x, sum.y += y;
    }
    if ((threadIdx.x & 31) == 31) warp_sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
      int2 w = warp_sums[threadIdx.x];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
        if (threadIdx.x >= o) w.x += x, w.y += y;
      }
      warp_sums[threadIdx.x] = w;
    }
    __syncthreads();
    if (threadIdx.x >= 32) {
      const int2 w = warp_sums[(threadIdx.x >> 5) - 1];
      sum.x += w.x, sum.y += w.y;
    }
    if (e <= E) {
      const int first = at + sum.x - all;
      start[e] = first + before;
      if (rank == 0) {
        p.offsets[e] = first;
        int* t = p.tiles + 1 + 3 * (tiles + sum.y - mine);
        // tiles of the tensor cores are of even sizes: one of few rows takes as long as one of many
        const int step = tile_rows == kTcTile && mine > 0 ? ((all + mine - 1) / mine + 31) & ~31 : tile_rows;
        if (e < E)
          for (int r = 0; r < all; r += step, t += 3) {
            t[0] = e;
            t[1] = first + r;
            t[2] = min(step, all - r);
          }
      }
    }
    at += warp_sums[kPlanThreads / 32 - 1].x;
    tiles += warp_sums[kPlanThreads / 32 - 1].y;
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) p.tiles[0] = tiles;
  for (int i0 = p0 + threadIdx.x; i0 < p1; i0 += kPlanEach * kPlanThreads) {
    int e[kPlanEach];
#pragma unroll
    for (int j = 0; j < kPlanEach; ++j) e[j] = i0 + j * kPlanThreads < p1 ? ids[i0 + j * kPlanThreads] : -1;
#pragma unroll
    for (int j = 0; j < kPlanEach; ++j)
      if (i0 + j * kPlanThreads < p1)
        p.order[atomicAdd(&start[e[j] >= 0 && e[j] < E ? e[j] : E], 1)] = i0 + j * kPlanThreads;
  }
  cluster.sync();  // the others may still read this CTA's counts
}

// ------------------------------------------------------ products, few rows

constexpr int kPhases = 4;  // groups of four warps that take the K steps of an item in turn
constexpr int kRowsWarps = 4 * kPhases;           // that compute
constexpr int kRowsThreads = 32 * (kRowsWarps + kPhases);  // and one per group that streams
constexpr int kStepChunks = 2;
constexpr int kTileStep = kStepChunks * kChunkBytes;  // one tile's bytes of a step
constexpr int kXRow = 256 + 16;                       // a row of x's bytes of a step, and 16 that spread the banks

// With few pairs the hidden rows go to the down products as two bf16 parts (the
// rounded value and what it lost), two columns of the MMA that are idle there
// anyway, so that the sum over experts is rounded once.
template <bool SUM>
__host__ __device__ constexpr int parts_of() {
  return SUM ? 2 : 1;
}

template <int NT>
struct RowsCfg {
  static constexpr int kDepth = NT == 1 ? 4 : 3;  // stages of a group
  static constexpr int kStages = kPhases * kDepth;
  static constexpr int kStageBytes = 2 * kTileStep + 8 * NT * kXRow;
  static constexpr int kRedFloats = kRowsWarps * NT * 8 * 32;
  static constexpr int kRed = kStages * kStageBytes;  // two buffers of sums
  static constexpr int kBars = kRed + 2 * kRedFloats * 4;
  static constexpr int kSmem = kBars + 2 * kStages * 8 + 16;
  static_assert(kSmem <= 232448, "shared memory budget");
};

struct RowsArgs {
  const uint16_t* x;  // [., k] bf16; pair p reads row p / row_div
  int row_div;
  ExpertsView w;
  const int32_t* ids;
  MoePlan plan;       // not read with kFewPairs pairs or fewer
  int pairs;
  int splits;         // ranges of K, each with sums of its own (kF32)
  void* out;          // row p: bf16 or fp32 [n_out]
  int* zero;          // words to clear for the kernel that follows, or null
  int zero_count;
  // weighted sum by the CTA that completes its columns (SUM)
  const float* weights;
  uint16_t* sum_out;  // [pairs / top_k, n]
  int* arrived;       // [units], zero on entry
  int top_k;
};

__device__ int g_rows_device_error = 0;

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// out[., col] = bf16(sum_j weights[., j] * y[., j, col]), j ascending and y the
// sum of its splits, for the rows first, first + step, ...: which CTA runs it
// changes no bit.  With few pairs: lane p of every warp holds pair p's weight,
// and in `there` the pairs that have an expert.
__device__ __forceinline__ void rows_sum(const RowsArgs& a, int64_t col, int first, int step, uint32_t there,
                                         float weight) {
  const float* y = static_cast<const float*>(a.out) + min(col, a.w.n - 1);
  const int64_t stride = (int64_t)a.pairs * a.w.n;
  const int rows = a.pairs / a.top_k, terms = a.top_k * a.splits;
  for (int row = first; row < rows; row += step) {
    float sum = 0.0f, v = 0.0f;
    int j = 0, i = 0;  // slot and split of the next term
    for (int f = 0; f < terms; f += 8) {  // eight loads in flight
      float t[8];
      int jj = j, ii = i;
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        const int p = row * a.top_k + jj;
        t[z] = f + z < terms && ((there >> (p & 31)) & 1) ? __ldcg(y + ii * stride + (int64_t)p * a.w.n) : 0.0f;
        if (++ii == a.splits) ii = 0, ++jj;
      }
#pragma unroll
      for (int z = 0; z < 8; ++z) {
        v += t[z];
        if (++i < a.splits) continue;
        const float w = __shfl_sync(0xffffffffu, weight, (row * a.top_k + j) & 31);
        if (j < a.top_k) sum = fmaf(w, v, sum);
        v = 0.0f;
        i = 0;
        ++j;
      }
    }
    if (col < a.w.n) a.sum_out[row * a.w.n + col] = f32_to_bf16_bits(sum);
  }
}

// A tile of rows: its expert, its rows and (in lane i) row i's pair, that of the
// last row in the lanes behind it.
struct RowTile {
  int e, rows, pair;
};

// Where a warp finds the tiles: in the plan; or, with few pairs, by sorting them
// itself, one lane per pair.  Lanes with equal ids form an expert, the lowest of
// them leads, and the leaders' tiles are numbered in lane order.  With one row
// of x every pair is a tile (its ids differ; equal ones are computed twice).
enum : int { kFromPlan = 0, kFromFew = 1, kFromOneRow = 2 };

template <int FROM>
struct Tiles {
  const RowsArgs& a;
  int lane, count;
  int id, mine, upto;  // this lane's id, the tiles it leads, the tiles up to and with them
  uint32_t same;

  __device__ __forceinline__ Tiles(const RowsArgs& args, int l, int tile_rows) : a(args), lane(l) {
    if (FROM == kFromPlan) {
      count = __ldcg(a.plan.tiles);
      return;
    }
    id = lane < a.pairs ? __ldcg(a.ids + lane) : -1;
    if (id < 0 || id >= a.w.experts) id = -1;
    if (FROM == kFromOneRow) {
      const uint32_t there = __ballot_sync(0xffffffffu, id >= 0);
      mine = id >= 0;
      upto = __popc(there & (0xffffffffu >> (31 - lane)));
      count = __popc(there);
      same = 1u << lane;
      return;
    }
    same = __match_any_sync(0xffffffffu, id);
    mine = id >= 0 && __ffs(same) - 1 == lane ? (__popc(same) + tile_rows - 1) / tile_rows : 0;
    upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    count = __shfl_sync(0xffffffffu, upto, 31);
  }

  __device__ __forceinline__ RowTile tile(int slot, int tile_rows) const {
    RowTile r;
    if (FROM == kFromPlan) {
      const int* t = a.plan.tiles + 1 + 3 * slot;
      r.e = __ldcg(t);
      r.rows = __ldcg(t + 2);
      r.pair = __ldcg(a.plan.order + __ldcg(t + 1) + min(lane, r.rows - 1));
      return r;
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, slot < upto && slot >= upto - mine)) - 1;
    r.e = __shfl_sync(0xffffffffu, id, l);
    if (FROM == kFromOneRow) {
      r.rows = 1;
      r.pair = l;
      return r;
    }
    uint32_t rest = __shfl_sync(0xffffffffu, same, l);
    const int skip = tile_rows * (slot - __shfl_sync(0xffffffffu, upto - mine, l));
    r.rows = min(tile_rows, __popc(rest) - skip);
    for (int i = 0; i < skip + min(lane, r.rows - 1); ++i) rest &= rest - 1;
    r.pair = __ffs(rest) - 1;
    return r;
  }
};

// An item's place: tile of rows, unit of weight rows, range of K.
struct Item {
  int slot, unit, split;
  __device__ __forceinline__ Item(int q, int units, int splits) {
    const int su = splits == 1 ? q : q / splits;
    split = q - su * splits;
    slot = su / units;
    unit = su - slot * units;
  }
  __device__ __forceinline__ void next(int units, int splits) {
    if (++split < splits) return;
    split = 0;
    if (++unit < units) return;
    unit = 0;
    ++slot;
  }
};

// An item is 64 gate rows and their up rows of one expert (or 128 rows of a
// plain weight, two tiles) times up to 8 NT of its rows, over all of K or one
// of its ranges.  One CTA per SM takes an equal run of the items.  Four groups
// of four warps take the items' steps (128 elements of K) in turn; a fifth warp
// per group streams its steps of the two tiles and of the rows of x by bulk
// copies into the group's stages, on into the next items while the current one
// is summed (147 KB of weights in flight per SM; issuing the copies takes 0.2 us
// a step, too long for a warp that computes).  Each warp owns 16 rows of either
// tile.  Its lane (g, t) = (lane / 4, lane % 4) reads 32 consecutive K
// elements of rows g and g + 8 of both tiles, and the same elements of rows
// g, g + 8 of x: the MMA sums over K in any order, so "k" of the fragments is
// whatever the four lanes of a quad hold, and no data moves between lanes.  The
// groups' sums are added in a fixed order.
// Bound by the decode: 500 cycles a step and quarter of an SM, of which the ALU
// pipe is busy for 370 (the MMAs for 160).  One row through 2 of 8 experts of
// 4096 x 12288 takes 49 us (170 MB of weights, 26 us at the copy rate), through 8
// of 64 of 2048 x 1024 15.9 us (28 MB, 4.3), 256 pairs of those 71 us (34).
// Tiles of 16 rows (NT = 2) do not fit the 96 registers a thread and spill 28 to
// 68 bytes; those of 8 do.
template <int MODE, int NT, int FROM, bool SUM>
__global__ void __launch_bounds__(kRowsThreads, 1) experts_rows_kernel(const RowsArgs a) {
  using C = RowsCfg<NT>;
  constexpr bool kPair = MODE == (int)ExpertsOut::kSiluMul;
  constexpr int kParts = parts_of<SUM>();         // columns of the MMA per row of x
  constexpr int kRows = 8 * NT / kParts;
  extern __shared__ __align__(128) uint8_t rows_smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(rows_smem + C::kBars);  // [group][stage]
  uint64_t* empty = full + C::kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + C::kStages);
  int* last = reinterpret_cast<int*>(empty + C::kStages) + 1;
  int* err = &g_rows_device_error;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // computing warp 4 * group + own; streaming warp 16 + group
  const bool streams = warp >= kRowsWarps;
  const int phase = streams ? warp - kRowsWarps : warp >> 2, own = warp & 3, g = lane >> 2, t = lane & 3;
  const int k = (int)a.w.k;
  const int steps = (a.w.kc + kStepChunks - 1) / kStepChunks;
  const int units = kPair ? a.w.wtiles : (a.w.wtiles + 1) / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // The next kernel may start once every CTA of this one has waited for the
  // previous one.  So when the down products of few pairs start, whatever wrote
  // the ids has finished, and they stream their first weights while the gate
  // and up products run out.
  if (!SUM) {
    griddep_wait();
    griddep_launch_dependents();
  }
  const Tiles<FROM> tiles(a, lane, kRows);
  const int items = tiles.count * units * a.splits;  // [tile][unit][split]
  const int each = items / (int)gridDim.x, more = items - each * (int)gridDim.x;
  const int q0 = each * (int)blockIdx.x + min((int)blockIdx.x, more), q1 = q0 + each + ((int)blockIdx.x < more);
  uint8_t* ring = rows_smem + phase * C::kDepth * C::kStageBytes;  // the group's stages
  full += phase * C::kDepth;
  empty += phase * C::kDepth;

  if (streams) {
    // ---------------------------------------------- stream of the group's steps
    int n = 0, step0 = 0, slot = -1;
    RowTile rt{0, 0, 0};
    const uint16_t* xrow = nullptr;  // lane i: row (and part) i of x
    bool ok = true, waited = !SUM;
    int held_rows[C::kDepth];        // x's part of the steps whose weights were fetched ahead of the wait
    const uint16_t* held_src[C::kDepth];
    uint32_t held_bytes[C::kDepth];
    auto fetch_x = [&](int s, const uint16_t* src, int rows, uint32_t bytes) {
      if (lane < rows * kParts) bulk_load(ring + s * C::kStageBytes + 2 * kTileStep + lane * kXRow, src, bytes, &full[s]);
    };
    auto wait = [&] {
      griddep_wait();
      griddep_launch_dependents();
      waited = true;
#pragma unroll
      for (int i = 0; i < C::kDepth; ++i)
        if (i < n) fetch_x(i, held_src[i], held_rows[i], held_bytes[i]);
    };
    Item it(q0, units, a.splits);
    for (int q = q0; ok && q < q1; ++q, it.next(units, a.splits)) {
      const int c0 = steps * it.split / a.splits, c1 = steps * (it.split + 1) / a.splits;
      if (it.slot != slot) {
        slot = it.slot;
        rt = tiles.tile(slot, kRows);
        const int p = kParts == 1 ? rt.pair : __shfl_sync(0xffffffffu, rt.pair, lane / kParts);
        xrow = a.x + (size_t)(FROM == kFromOneRow && a.row_div > 1 ? 0 : p / a.row_div * kParts + lane % kParts) * k;
      }
      const size_t tile_bytes = (size_t)a.w.kc * kChunkBytes;
      // a plain weight's missing second tile: the first stands in, its sums are not stored
      const uint8_t* w0 = a.w.tiles + ((size_t)rt.e * (kPair ? 2 : 1) * a.w.wtiles + (kPair ? it.unit : 2 * it.unit)) * tile_bytes;
      const uint8_t* w1 = kPair ? w0 + a.w.wtiles * tile_bytes : 2 * it.unit + 1 < a.w.wtiles ? w0 + tile_bytes : w0;
      for (int c = c0 + ((phase - step0) & (kPhases - 1)); c < c1; c += kPhases, ++n) {
        const int s = n % C::kDepth;
        if (n >= C::kDepth) {
          if (!waited) wait();
          ok = mbar_wait(&empty[s], (n / C::kDepth - 1) & 1, abort_flag, err, 1);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
        }
        const uint32_t bytes = min(kStepChunks, a.w.kc - kStepChunks * c) * kChunkBytes;
        const uint32_t xbytes = 2 * min(128, k - 128 * c);
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[s], 2 * bytes + rt.rows * kParts * xbytes);
          bulk_load(ring + s * C::kStageBytes, w0 + (size_t)c * kTileStep, bytes, &full[s]);
          bulk_load(ring + s * C::kStageBytes + kTileStep, w1 + (size_t)c * kTileStep, bytes, &full[s]);
        }
        __syncwarp();
        if (waited) {
          fetch_x(s, xrow + 128 * c, rt.rows, xbytes);
        } else {
#pragma unroll
          for (int i = 0; i < C::kDepth; ++i)
            if (i == s) held_rows[i] = rt.rows, held_src[i] = xrow + 128 * c, held_bytes[i] = xbytes;
        }
      }
      step0 += c1 - c0;
    }
    if (!waited) wait();
    // No copy into this CTA's shared memory may outlive it; all of them are
    // waited for by the computing warps unless a wait has expired.
    if (lane == 0)
      for (int i = max(0, n - C::kDepth); i < n; ++i) {
        const long long t0 = clock64();
        while (!mbar_try_wait(&full[i % C::kDepth], (i / C::kDepth) & 1) && clock64() - t0 < kWaitLimitCycles) {
        }
      }
    return;
  }
  if (SUM) {
    griddep_wait();
    griddep_launch_dependents();
  }

  uint32_t there = 0;  // for the sum
  float weight = 0.0f;
  if (SUM) {
    there = __ballot_sync(0xffffffffu, tiles.id >= 0);
    weight = lane < a.pairs ? __ldcg(a.weights + lane) : 0.0f;
  }

  // ------------------------------------------------------------------ products
  const int row0 = 16 * own + g, h = t & 1, cc = t >> 1;  // first row, half and chunk of this lane's elements
  // offsets in a stage of this lane's codes (rows row0, row0 + 8), their scales and its elements of x
  const int at0 = cc * kChunkBytes + code_offset(row0, h, cc), at1 = cc * kChunkBytes + code_offset(row0 + 8, h, cc);
  const int at_sc = cc * kChunkBytes + scale_offset(row0, cc), at_x = 2 * kTileStep + g * kXRow + 64 * t;
  const uint32_t pick0 = h ? 0x4242 : 0x4040, pick1 = pick0 + 0x0101;  // this half's two scales
  int n = 0, step0 = 0, slot = -1, buf = 0;  // the group's steps, the items' steps so far
  RowTile rt{0, 0, 0};
  float gs0 = 0.0f, gs1 = 0.0f;
  Item it(q0, units, a.splits);
  for (int q = q0; q < q1; ++q, buf ^= 1, it.next(units, a.splits)) {
    const int unit = it.unit;
    if (it.slot != slot) {
      slot = it.slot;
      rt = tiles.tile(slot, kRows);
      gs0 = a.w.gs[kPair ? 2 * rt.e : rt.e] * kUnscale;
      gs1 = kPair ? a.w.gs[2 * rt.e + 1] * kUnscale : gs0;
    }
    const int c0 = steps * it.split / a.splits, c1 = steps * (it.split + 1) / a.splits;
    float acc[NT][2][4] = {};
    for (int c = c0 + ((phase - step0) & (kPhases - 1)); c < c1; c += kPhases, ++n) {
      const int s = n % C::kDepth;
      const bool ok = mbar_wait(&full[s], (n / C::kDepth) & 1, abort_flag, err, 2);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t* st = ring + s * C::kStageBytes;
      uint4 cw[4];
      uint32_t sc[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        cw[2 * j] = *reinterpret_cast<const uint4*>(st + j * kTileStep + at0);
        cw[2 * j + 1] = *reinterpret_cast<const uint4*>(st + j * kTileStep + at1);
        const uint2 v = *reinterpret_cast<const uint2*>(st + j * kTileStep + at_sc);
        sc[2 * j] = v.x;
        sc[2 * j + 1] = v.y;
      }
      // Columns of the MMA are independent and those behind the last row are
      // not stored: their lanes read whatever the stage holds.
      uint4 xv[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[i][j] = *reinterpret_cast<const uint4*>(st + at_x + i * 8 * kXRow + 16 * j);
      if (128 * c + 128 > k && 128 * c + 32 * t >= k) {  // behind the end of K the stage is stale
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          cw[j] = make_uint4(0, 0, 0, 0);
          sc[j] = 0;
#pragma unroll
          for (int i = 0; i < NT; ++i) xv[i][j] = make_uint4(0, 0, 0, 0);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);  // the step is in registers
      uint32_t s2[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t d[4][4];
        if (w == 0 || w == 2)
#pragma unroll
          for (int j = 0; j < 4; ++j) s2[j] = scale_twice(sc[j], w == 0 ? pick0 : pick1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t word = w == 0 ? cw[j].x : w == 1 ? cw[j].y : w == 2 ? cw[j].z : cw[j].w;
          decode8(word, s2[j], d[j]);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const uint32_t b[4] = {xv[i][w].x, xv[i][w].y, xv[i][w].z, xv[i][w].w};
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            mma_16816(acc[i][0], d[0][2 * z], d[1][2 * z], d[0][2 * z + 1], d[1][2 * z + 1], b[2 * z], b[2 * z + 1]);
            mma_16816(acc[i][1], d[2][2 * z], d[3][2 * z], d[2][2 * z + 1], d[3][2 * z + 1], b[2 * z], b[2 * z + 1]);
          }
        }
      }
    }
    step0 += c1 - c0;
    // The sums of the four groups of these rows: [group][own][n][accumulator][lane].
    float* red = reinterpret_cast<float*>(rows_smem + C::kRed) + buf * C::kRedFloats + own * NT * 256;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) red[phase * 4 * NT * 256 + (i * 8 + j) * 32 + lane] = acc[i][j >> 2][j & 3];
    named_bar_sync(1 + own, 32 * kPhases);
    // (two buffers: this one is written again after the next item's barrier)
    // accumulator i of lane (g, t): tile i / 4, row g + 8 * (i / 2 % 2), x row 2t + (i & 1)
    const int et = 32 * phase + lane, og = et & 7, oh = (et >> 3) & 1, on = et >> 4;
    // (after an expired wait every warp still passes every barrier, and stores nothing)
    const bool live = !*abort_flag;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int row = (8 * i + on) / kParts;  // (of two parts, the first one's threads add both)
      const int64_t p = __shfl_sync(0xffffffffu, rt.pair, row);
      if (row >= rt.rows || on % kParts || !live) continue;
      const float* src = red + (i * 8 + 2 * oh + (on & 1)) * 32 + 4 * og + (on >> 1);
      float v = 0.0f, u = 0.0f;
#pragma unroll
      for (int j = 0; j < kPhases; ++j) {
#pragma unroll
        for (int z = 0; z < kParts; ++z) {
          v += src[j * 4 * NT * 256 + 32 * z];
          u += src[j * 4 * NT * 256 + 4 * 32 + 32 * z];
        }
      }
      const int r = 16 * own + 8 * oh + og;
      if (kPair) {
        const int64_t inter = a.w.n / 2, col = kTileRows * (int64_t)unit + r;
        const float hv = silu_f32(gs0 * v) * (gs1 * u), hi = bf16_round(hv);
        uint16_t* o = static_cast<uint16_t*>(a.out) + p * (FROM == kFromPlan ? 1 : 2) * inter + col;
        if (col < inter) {
          o[0] = f32_to_bf16_bits(hi);
          if (FROM != kFromPlan) o[inter] = f32_to_bf16_bits(isfinite(hi) ? hv - hi : 0.0f);
        }
      } else {
        const int64_t col = 2 * kTileRows * (int64_t)unit + r;
        if (MODE == (int)ExpertsOut::kF32) {
          float* y = static_cast<float*>(a.out) + ((int64_t)it.split * a.pairs + p) * a.w.n + col;
          if (col < a.w.n) y[0] = gs0 * v;
          if (col + kTileRows < a.w.n) y[kTileRows] = gs0 * u;
        } else {
          uint16_t* y = static_cast<uint16_t*>(a.out) + p * a.w.n + col;
          if (col < a.w.n) y[0] = f32_to_bf16_bits(gs0 * v);
          if (col + kTileRows < a.w.n) y[kTileRows] = f32_to_bf16_bits(gs0 * u);
        }
      }
    }
    if (SUM) {
      // The CTA that completes the columns of a unit adds the experts' outputs.
      __threadfence();
      named_bar_sync(5, 32 * kRowsWarps);
      if (threadIdx.x == 0) *last = atomicAdd(&a.arrived[unit], 1) == tiles.count * a.splits - 1;
      named_bar_sync(5, 32 * kRowsWarps);
      if (*last) {
        __threadfence();
        rows_sum(a, 2 * kTileRows * (int64_t)unit + (threadIdx.x & 127), threadIdx.x >> 7, kRowsWarps / 4, there, weight);
      }
    }
  }
  if (MODE == (int)ExpertsOut::kBf16)  // zeros for the pairs without an expert
    for (int64_t p = blockIdx.x; p < a.pairs; p += gridDim.x) {
      const int id = a.ids[p];
      if (id >= 0 && id < a.w.experts) continue;
      for (int64_t c = threadIdx.x; c < a.w.n; c += 32 * kRowsWarps) static_cast<uint16_t*>(a.out)[p * a.w.n + c] = 0;
    }
  if (a.zero && blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.zero_count; i += 32 * kRowsWarps) a.zero[i] = 0;
  if (SUM && tiles.count == 0)  // no row has an expert
    for (int64_t c = 128 * (int64_t)blockIdx.x; c < a.w.n; c += 128 * (int64_t)gridDim.x)
      rows_sum(a, c + (threadIdx.x & 127), threadIdx.x >> 7, kRowsWarps / 4, there, weight);
}

// ----------------------------------------------------------- weighted sum

// Bound by DRAM where a prompt's sums are more than L2 holds: 32768 pairs of 2048
// columns, 268 MB of them written by the down products and 285 MB moved here, 63 us.
// Eight loads in flight per thread, streamed past L2, take 48 us but leave their
// time to the writes still under way: the layer's time is the same.
__global__ void __launch_bounds__(256) moe_combine_kernel(const float* __restrict__ y, int splits,
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
    if (e >= 0 && e < experts) {
      v = *reinterpret_cast<const float4*>(y + p * hidden + c);
      for (int i = 1; i < splits; ++i) {
        const float4 o = *reinterpret_cast<const float4*>(y + (i * m * top_k + p) * hidden + c);
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
      }
    }
    s.x = fmaf(w, v.x, s.x);
    s.y = fmaf(w, v.y, s.y);
    s.z = fmaf(w, v.z, s.z);
    s.w = fmaf(w, v.w, s.w);
  }
  *reinterpret_cast<uint2*>(out + row * hidden + c) =
      make_uint2((uint32_t)f32_to_bf16_bits(s.x) | ((uint32_t)f32_to_bf16_bits(s.y) << 16),
                 (uint32_t)f32_to_bf16_bits(s.z) | ((uint32_t)f32_to_bf16_bits(s.w) << 16));
}

}  // namespace

cudaError_t launch_moe_plan(const int32_t* ids, int64_t pairs, int experts, int tile_rows, const MoePlan& p,
                            cudaStream_t s) {
  ProfScope prof(s, "moe_plan");
  // a CTA takes its ids in one go up to kPlanEach a thread; eight CTAs cut a
  // prompt's 32768 pairs from 35 to 6 us
  const int ctas = pairs <= kPlanEach * kPlanThreads ? 1 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = 2 * sizeof(int) * (experts + 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = profiling() ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, moe_plan_kernel, ids, (int)pairs, experts, tile_rows, p);
}

namespace {

template <int MODE, int NT, int FROM, bool SUM>
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s) {
  auto kern = experts_rows_kernel<MODE, NT, FROM, SUM>;
  constexpr int kSmem = RowsCfg<NT>::kSmem;
  // set on every launch: the attribute belongs to the current device's context
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t most = moe_max_tiles(a.pairs, a.w.experts, 8 * NT / parts_of<SUM>()) * rows_units(a.w) * a.splits;
  if (most > INT32_MAX) return cudaErrorInvalidValue;
  const int sms = device_sms();
  return launch_pdl(kern, dim3((unsigned)(most < sms ? most : sms)), dim3(kRowsThreads), kSmem, s, a);
}

// SUM: of few pairs; from a plan the sum is a launch of its own.
template <int MODE, bool SUM>
cudaError_t launch_rows_from(const RowsArgs& a, cudaStream_t s) {
  constexpr int kNT = 2;
  if (a.pairs > kFewPairs)
    return rows_tile(a.pairs, a.w.experts) == 8 ? launch_rows<MODE, 1, kFromPlan, false>(a, s)
                                                : launch_rows<MODE, kNT, kFromPlan, false>(a, s);
  if (a.pairs == a.top_k) return launch_rows<MODE, 1, kFromOneRow, SUM>(a, s);
  // an expert has at most one row per row of x where a row's ids differ: so few
  // rows fill one tile
  return a.pairs / a.top_k <= 8 / parts_of<SUM>() ? launch_rows<MODE, 1, kFromFew, SUM>(a, s) : launch_rows<MODE, kNT, kFromFew, SUM>(a, s);
}

}  // namespace

int rows_splits(const ExpertsView& w, int64_t tiles, int sms) {
  // Rounds of items over the SMs times the steps of an item, and about four
  // steps' time for an item's sums.  One row through 2 of 8 experts of
  // 4096 x 12288 takes 48.9 us with the two ranges that this gives and 61.5 with one,
  // through 2 of 8 of 1056 x 672 11.5 with six and 12.0 with one.
  const int64_t steps = (w.kc + kStepChunks - 1) / kStepChunks, items = tiles * rows_units(w);
  int64_t best = 0, least = INT64_MAX;
  for (int64_t s = 1; s <= kMaxSplits && s <= steps; ++s) {
    const int64_t cost = ((items * s + sms - 1) / sms) * ((steps + s - 1) / s + 4);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return (int)best;
}

cudaError_t launch_experts_rows(const void* x, int row_div, const ExpertsView& w, const int32_t* ids, const MoePlan& p,
                                int64_t pairs, int top_k, ExpertsOut mode, int splits, void* out, int* zero,
                                int zero_count, const RowsSum* sum, cudaStream_t s) {
  RowsArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.row_div = row_div;
  a.w = w;
  a.ids = ids;
  a.plan = p;
  a.pairs = (int)pairs;
  a.splits = splits;
  a.out = out;
  a.zero = zero;
  a.zero_count = zero_count;
  a.weights = sum ? sum->weights : nullptr;
  a.sum_out = sum ? static_cast<uint16_t*>(sum->out) : nullptr;
  a.arrived = sum ? sum->arrived : nullptr;
  a.top_k = top_k;
  ProfScope prof(s, mode == ExpertsOut::kSiluMul ? "experts_rows_silu" : sum ? "experts_rows_sum" : "experts_rows");
  switch (mode) {
    case ExpertsOut::kSiluMul: return launch_rows_from<(int)ExpertsOut::kSiluMul, false>(a, s);
    case ExpertsOut::kF32: return launch_rows_from<(int)ExpertsOut::kF32, true>(a, s);
    default: return launch_rows_from<(int)ExpertsOut::kBf16, false>(a, s);
  }
}

cudaError_t read_rows_device_error(int* flags, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_rows_device_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_rows_device_error, &zero, sizeof(int));
  return e;
}

cudaError_t launch_moe_combine(const float* y, int splits, const int32_t* ids, const float* weights, int64_t m,
                               int top_k, int experts, int64_t hidden, void* out, cudaStream_t s) {
  ProfScope prof(s, "moe_combine");
  const int64_t blocks = (m * (hidden / 4) + 255) / 256;
  return launch_pdl(moe_combine_kernel, dim3((unsigned)blocks), dim3(256), 0, s, y, splits, ids, weights, m, top_k,
                    experts, hidden, static_cast<uint16_t*>(out));
}

}  // namespace ffn
