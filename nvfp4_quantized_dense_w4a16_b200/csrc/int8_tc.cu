// Products of the 8-bit integer layers on the tensor cores (tcgen05 kind::i8,
// 32-bit sums in tensor memory, operands streamed by TMA as rows of 128 codes).
//
// Many rows: a persistent pair of CTAs (cta_group::2) computes tiles of 256 rows
// of x by up to 256 weight rows.  Per 128 codes of K each CTA loads its 128 rows
// of x and half of the tile's weight rows (with silu_mul: CTA 0 the gate rows,
// CTA 1 the up rows of the same columns), and one warp of CTA 0 issues the MMAs
// of both.  Two accumulators: eight warps scale and store a tile while the next
// one's MMAs run.
//
// Few rows: the weight rows are the MMA's M (a tile of 128; with silu_mul 64 gate
// rows and the 64 up rows of the same columns), x is its N.  Bound by the stream
// of the weights, which all SMs have to share: a cluster of CTAs cuts the K of a
// tile into ranges, and each CTA adds a share of the others' sums, read from their
// shared memory.  Sums are whole numbers: the cut does not change a bit.  More than
// 128 rows go in blocks, each with the weights to itself.
//
// Weights are loaded before the kernel ahead that makes the rows has completed (but
// for the first launch of a call), rows after it.  Every wait is bounded; on expiry a device error bit is raised, the
// CTAs free their tensor memory and exit.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "int8.cuh"
#include "int8.h"
#include "launch.cuh"
#include "moe.h"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using namespace sm100;

__device__ int g_int8_device_error = 0;

constexpr int kChunkK = 128;  // codes of K in a stage: one 128-byte swizzled row

// Instruction descriptor of kind::i8: signed 8-bit A and B (both K-major), 32-bit sums.
__host__ __device__ constexpr uint32_t idesc_s8_s32(int M, int N) {
  return (2u << 4)                      // D format: s32
         | (1u << 7)                    // A format: signed
         | (1u << 10)                   // B format: signed
         | ((uint32_t)(N >> 3) << 17)   // N / 8
         | ((uint32_t)(M >> 4) << 24);  // M / 16
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The shared address of `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

__device__ __forceinline__ int4 load_cluster(uint32_t a) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

// Wait that ignores the abort flag (in-flight copies must land before exit).
__device__ __forceinline__ bool drain(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) {
      atomicOr(&g_int8_device_error, 16);
      return false;
    }
  return true;
}

// ------------------------------------------------------------- many rows

__device__ __forceinline__ void mma_pair_s8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
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

// A copy into this CTA's shared memory that counts on a barrier of either CTA.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

struct PairArgs {
  const float *xs, *ws;
  const uint16_t* bias;
  uint16_t* y;
  int64_t m, cols;  // rows and columns of y
  int kc;           // chunks of K
  int tile_n;       // weight rows of a tile: a multiple of 32 up to 256
  int m_tiles, n_tiles;
  int stages;       // of the ring
  bool first;       // (Int8Product::first)
};

constexpr int kPairRows = 256;
constexpr int kPairThreads = 384;
constexpr int kPairUnit = 2;  // chunks of K in a stage
constexpr int kPairMaxStages = 5;
constexpr int kPairOperand = 128 * kChunkK;  // 128 rows of x, or up to 128 weight rows
constexpr int kPairRing = 6 * 2 * kPairOperand;
constexpr int kPairOut = kPairRing;          // 32 rows x 32 columns of bf16 per epilogue warp
constexpr int kPairScales = kPairOut + 8 * 2048;         // [group][tile parity][scales, biases][256]
constexpr int kPairBar = kPairScales + 2 * 2 * 2 * 256 * 4;
constexpr int kPairSmem = kPairBar + (2 * kPairMaxStages + 4) * 8 + 16 + 1024;  // slack for 1024-byte alignment
static_assert(kPairSmem <= 232448, "shared memory budget");

// Tiles go by groups of this many row tiles, so that those which run at a time
// share rows of x and of the weight in L2.
constexpr int kPairGroup = 8;

__device__ __forceinline__ void tile_place(const PairArgs& a, int t, int* mt, int* nt) {
  const int group = t / (kPairGroup * a.n_tiles), first = group * kPairGroup;
  const int rows = min(kPairGroup, a.m_tiles - first), in = t - first * a.n_tiles;
  *mt = first + in % rows;
  *nt = in / rows;
}

template <bool SILU>
__global__ void __cluster_dims__(2) __launch_bounds__(kPairThreads, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const PairArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairBar);
  uint64_t* empty = full + kPairMaxStages;
  uint64_t* accfull = empty + kPairMaxStages;
  uint64_t* accempty = accfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* err = &g_int8_device_error;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int first = blockIdx.x / 2, step = gridDim.x / 2, total = a.m_tiles * a.n_tiles;
  const int half = a.tile_n / 2;  // weight rows of a CTA
  const int stages = a.stages, chunk_bytes = kPairOperand + half * kChunkK, stage_bytes = kPairUnit * chunk_bytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);  // (CTA 0's)
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 2 * 8);  // (CTA 0's)
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&xmap);
    tma_prefetch_desc(&wmap);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ----------------------------------------------------------- producer
    if (lane == 0) {
      // What to load goes by two cursors, of the weights and of the rows; places of
      // tiles cost divisions, which a cursor pays once a tile (each unit's own took
      // 850 cycles of the 512 that its MMAs take).
      const uint32_t bars = in_cta(full, 0);
      struct Cursor {
        int t, c = 0, s = 0, row = 0;
        bool weights;
        __device__ __forceinline__ void place(const PairArgs& a, int half, int rank) {
          int mt, nt;
          tile_place(a, t, &mt, &nt);
          row = !weights ? mt * kPairRows + rank * 128 : SILU ? (int)(nt * half + rank * a.cols) : nt * a.tile_n + rank * half;
        }
        __device__ __forceinline__ void next(const PairArgs& a, int step, int total, int half, int rank) {
          if (++s == a.stages) s = 0;
          c += kPairUnit;
          if (c < a.kc) return;
          c = 0;
          t += step;
          if (t < total) place(a, half, rank);
        }
      };
      Cursor w{first}, x{first};
      w.weights = true, x.weights = false;
      if (first < total) w.place(a, half, rank), x.place(a, half, rank);
      auto load_weights = [&] {
        const int n = min(kPairUnit, a.kc - w.c);
        if (rank == 0) mbar_arrive_expect_tx(&full[w.s], 2 * n * chunk_bytes);  // of both CTAs
        for (int j = 0; j < n; ++j)
          tma_load_pair(smem + w.s * stage_bytes + j * chunk_bytes + kPairOperand, &wmap, (w.c + j) * kChunkK, w.row, bars + 8 * w.s);
        w.next(a, step, total, half, rank);
      };
      auto load_rows = [&] {
        const int n = min(kPairUnit, a.kc - x.c);
        for (int j = 0; j < n; ++j)
          tma_load_pair(smem + x.s * stage_bytes + j * chunk_bytes, &xmap, (x.c + j) * kChunkK, x.row, bars + 8 * x.s);
        x.next(a, step, total, half, rank);
      };
      int ahead = 0, u = 0;
      if (a.first) griddep_wait();
      for (; ahead < stages && w.t < total; ++ahead) load_weights();
      griddep_wait();
      griddep_launch_dependents();
      for (; u < ahead; ++u) load_rows();
      uint32_t parity = 0;  // of the stage's last use
      for (; w.t < total; ++u) {
        if (!mbar_wait(&empty[w.s], parity, abort_flag, err, 1)) break;
        if (w.s == stages - 1) parity ^= 1;
        load_weights();
        load_rows();
      }
      if (rank == 0)  // (CTA 1 leaves after this one)
        for (int r = max(0, u - stages); r < u; ++r) drain(&full[r % stages], (r / stages) & 1);
    }
  } else if (warp == 1) {
    // --------------------------------------------- MMAs, CTA 0's for both
    // (all roles wait for the kernel ahead: the limits of their waits begin after it)
    const uint32_t idesc = idesc_s8_s32(kPairRows, a.tile_n);
    griddep_wait();
    int s = 0, i = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int t = first; rank == 0 && ok && t < total; t += step, ++i) {
      const int buf = i & 1;
      if (i >= 2) {
        ok = mbar_wait(&accempty[buf], ((i >> 1) - 1) & 1, abort_flag, err, 2);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
      }
      for (int c = 0; c < a.kc; c += kPairUnit) {
        ok = mbar_wait(&full[s], parity, abort_flag, err, 2);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t at = smem_u32(smem + s * stage_bytes);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kPairUnit; ++j) {
            if (c + j >= a.kc) break;
            const uint64_t xd = smem_desc_sw128(at + j * chunk_bytes), wd = smem_desc_sw128(at + j * chunk_bytes + kPairOperand);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_pair_s8(tmem + 256 * buf, xd + 2 * kk, wd + 2 * kk, idesc, (c | j | kk) ? 1u : 0u);
          }
          commit_pair(&empty[s]);
          if (c + kPairUnit >= a.kc) commit_pair(&accfull[buf]);
        }
        __syncwarp();
        if (++s == stages) s = 0, parity ^= 1;
      }
    }
  } else if (warp >= 4) {
    // ----------------------------------------------------------- epilogue
    const int g = (warp - 4) >> 2, q = warp & 3, tid = threadIdx.x & 127;
    uint8_t* out = smem + kPairOut + (warp - 4) * 2048;
    // 16 columns at a time; the two groups share them
    const int outs = SILU ? half : a.tile_n, parts = outs / 16;
    const int part0 = g ? (parts + 1) / 2 : 0, part1 = g ? parts : (parts + 1) / 2;
    const bool wide = a.cols % 8 == 0;
    griddep_wait();
    int i = 0;
    for (int t = first; t < total; t += step, ++i) {
      int mt, nt;
      tile_place(a, t, &mt, &nt);
      const int buf = i & 1;
      const int64_t row0 = (int64_t)mt * kPairRows + rank * 128 + 32 * q, col0 = (int64_t)nt * outs;
      const float xs = row0 + lane < a.m ? a.xs[row0 + lane] : 0.0f;
      float* sc = reinterpret_cast<float*>(smem + kPairScales) + (2 * g + buf) * 512;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = tid + 128 * h;
        if (SILU) {
          const int64_t col = col0 + tid;  // gate scales, then up scales
          if (tid < half) sc[h * 256 + tid] = col < a.cols ? a.ws[h * a.cols + col] : 0.0f;
        } else if (j < outs) {
          const bool in = col0 + j < a.cols;
          sc[j] = in ? a.ws[col0 + j] : 0.0f;
          sc[256 + j] = in && a.bias ? bf16_bits_to_float(a.bias[col0 + j]) : 0.0f;
        }
      }
      __syncwarp();  // (the barriers want whole warps)
      named_bar_sync(1 + g, 128);
      bool ok = mbar_wait(&accfull[buf], (i >> 1) & 1, abort_flag, err, 8);
      ok = __all_sync(0xffffffffu, ok);
      uint32_t any;  // (the group's warps pass the same barriers)
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(any)
          : "r"((uint32_t)ok), "r"(1 + g)
          : "memory");
      if (!any) break;
      tc_fence_after();
      const uint32_t lane_addr = tmem + ((uint32_t)(32 * q) << 16) + 256 * buf;
      for (int p = part0; p < part1; p += 2) {
        const int width = min(2, part1 - p) * 16;  // columns of this step
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (16 * h >= width) break;
          const int c = 16 * (p + h);
          uint32_t v[16], w[16];
          tmem_ld16(lane_addr + c, v);
          if (SILU) tmem_ld16(lane_addr + half + c, w);
          tmem_ld_wait();
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float r[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              r[z] = int8_scaled((int)v[j + z], xs, sc[c + j + z]);
              if (SILU)
                r[z] = int8_silu_mul(r[z], int8_scaled((int)w[j + z], xs, sc[256 + c + j + z]));
              else if (a.bias)
                r[z] = __fadd_rn(r[z], sc[256 + c + j + z]);
            }
            o[j / 2] = f32_to_bf16_bits(r[0]) | ((uint32_t)f32_to_bf16_bits(r[1]) << 16);
          }
#pragma unroll
          for (int z = 0; z < 2; ++z)
            *reinterpret_cast<uint4*>(out + lane * 64 + 16 * ((2 * h + z) ^ ((lane >> 1) & 3))) =
                make_uint4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]);
        }
        __syncwarp();
        const int64_t col = col0 + 16 * p;
        if (wide) {  // four lanes store 64 bytes of a row
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int r = 8 * z + (lane >> 2), c = 8 * (lane & 3);
            if (row0 + r < a.m && c < width && col + c < a.cols)
              *reinterpret_cast<uint4*>(a.y + (row0 + r) * a.cols + col + c) =
                  *reinterpret_cast<const uint4*>(out + r * 64 + 16 * ((lane & 3) ^ ((r >> 1) & 3)));
          }
        } else {  // rows at any two bytes: a warp stores one at a time (6241 x 13289 from K = 128:
          // 157 us, 13296 columns 83; two bytes a lane in 16-byte runs took 391)
          const int rows = (int)min((int64_t)32, a.m - row0);
          for (int r = 0; r < rows; ++r) {
            const uint16_t v = *reinterpret_cast<const uint16_t*>(out + r * 64 + 16 * ((lane >> 3) ^ ((r >> 1) & 3)) + 2 * (lane & 7));
            if (lane < width && col + lane < a.cols) a.y[(row0 + r) * a.cols + col + lane] = v;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_cta(&accempty[buf], 0)) : "memory");
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may arrive on its barriers or read its rows
  if (warp == 2) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// -------------------------------------------------------------- few rows

__device__ __forceinline__ void mma_s8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

struct FewArgs {
  const float *xs, *ws;
  const uint16_t* bias;
  uint16_t* y;
  int64_t cols;
  int64_t m;
  int kc;
  int n;       // the MMA's N: rows of x of a CTA, a multiple of 16
  int stages;  // of the ring
  bool first;  // (Int8Product::first)
};

constexpr int kFewThreads = 192;  // a producer, an issuer, four warps for the sums
constexpr int kFewWeights = 128 * kChunkK;
constexpr int kFewMaxStages = 8, kFewMaxSplits = 8;
constexpr int kFewRing = 100 * 1024;  // two CTAs an SM
constexpr int kFewBar = 0;            // the barriers stand in front of the ring
constexpr int kFewSmem = 1024 + kFewRing + 1024;

template <bool SILU>
__global__ void __launch_bounds__(kFewThreads)
    int8_few_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kFewBar);
  uint64_t* empty = full + kFewMaxStages;
  uint64_t* done = empty + kFewMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* ring = smem + 1024;
  int* err = &g_int8_device_error;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t splits;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(splits));
  const int rank = (int)cluster_rank();
  const int64_t tile = blockIdx.x / splits;
  const int row0 = (int)blockIdx.y * a.n, rows = (int)min((int64_t)a.n, a.m - row0);
  const int c0 = (int)((int64_t)a.kc * rank / splits), c1 = (int)((int64_t)a.kc * (rank + 1) / splits), units = c1 - c0;
  const int stage_bytes = kFewWeights + a.n * kChunkK;
  const uint32_t columns = a.n <= 32 ? 32 : a.n <= 64 ? 64 : 128;  // of tensor memory

  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, columns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  const int64_t col = tile * (SILU ? 64 : 128) + 4 * (SILU ? lane & 15 : lane);  // of y, the first of a lane's four
  float s0[4], s1[4];

  if (warp == 0) {
    if (lane == 0) {
      auto load_weights = [&](int s, int k) {
        uint8_t* at = ring + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        if (SILU) {
          tma_load_2d(at, &wmap, k, (int)(tile * 64), &full[s]);
          tma_load_2d(at + kFewWeights / 2, &wmap, k, (int)(a.cols + tile * 64), &full[s]);
        } else {
          tma_load_2d(at, &wmap, k, (int)(tile * 128), &full[s]);
        }
      };
      auto load_rows = [&](int s, int k) { tma_load_2d(ring + s * stage_bytes + kFewWeights, &xmap, k, row0, &full[s]); };
      const int ahead = min(units, a.stages);
      if (a.first) griddep_wait();
      for (int u = 0; u < ahead; ++u) load_weights(u, (c0 + u) * kChunkK);
      griddep_wait();
      griddep_launch_dependents();
      for (int u = 0; u < ahead; ++u) load_rows(u, (c0 + u) * kChunkK);
      int u = ahead, s = 0;
      uint32_t parity = 0;
      for (; u < units; ++u) {
        if (!mbar_wait(&empty[s], parity, abort_flag, err, 1)) break;
        load_weights(s, (c0 + u) * kChunkK);
        load_rows(s, (c0 + u) * kChunkK);
        if (++s == a.stages) s = 0, parity ^= 1;
      }
      for (int r = max(0, u - a.stages); r < u; ++r) drain(&full[r % a.stages], (r / a.stages) & 1);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_s8_s32(128, a.n);
    griddep_wait();
    int s = 0;
    uint32_t parity = 0;
    for (int u = 0; u < units; ++u) {
      ok = mbar_wait(&full[s], parity, abort_flag, err, 2);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc_fence_after();
      const uint64_t wd = smem_desc_sw128(smem_u32(ring + s * stage_bytes));
      const uint64_t xd = smem_desc_sw128(smem_u32(ring + s * stage_bytes + kFewWeights));
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_s8(tmem, wd + 2 * kk, xd + 2 * kk, idesc, (u | kk) ? 1u : 0u);
        mma_commit(&empty[s]);
        if (u + 1 == units) mma_commit(done);
      }
      __syncwarp();
      if (++s == a.stages) s = 0, parity ^= 1;
    }
  } else {
    griddep_wait();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = col + j < a.cols;
      s0[j] = in ? a.ws[col + j] : 0.0f;
      s1[j] = !in ? 0.0f : SILU ? a.ws[a.cols + col + j] : a.bias ? bf16_bits_to_float(a.bias[col + j]) : 0.0f;
    }
    ok = mbar_wait(done, 0, abort_flag, err, 8);
    ok = __all_sync(0xffffffffu, ok);
  }
  // From here on no copy and no MMA is in flight: the ring holds the sums, [row of x][128].
  __syncwarp();
  ok = __syncthreads_and(ok) != 0;
  int* sums = reinterpret_cast<int*>(ring);
  if (ok && warp >= 2) {
    tc_fence_after();
    const int q = warp & 3;
    for (int c = 0; c < a.n; c += 16) {
      uint32_t v[16];
      tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + c, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) sums[(c + j) * 128 + 32 * q + lane] = (int)v[j];
    }
    tc_fence_before();
  }
  // A CTA whose wait expired has no sums: nobody of its cluster stores.
  if (threadIdx.x == 0) *abort_flag = ok ? 0 : 1;
  __syncthreads();
  cluster_sync();
  int bad = 0;
  if (lane < (int)splits)
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(bad) : "r"(in_cta(const_cast<int*>(abort_flag), lane)));
  if (warp >= 2) {
    // Rows of x by CTA; a warp has 128 sums of a row, four a lane, and kAtOnce such rows under way.
    constexpr int kAtOnce = 2, kPer = SILU ? 2 : 1;  // (with silu_mul half a warp has a row: gate and up sums)
    const int wq = warp - 2, mine = 4 * (SILU ? lane & 15 : lane);
    const int first = (rank * 4 + wq) * kPer + (SILU ? lane >> 4 : 0), step = (int)splits * 4 * kPer;
    ok = __all_sync(0xffffffffu, bad == 0);
    for (int i0 = first; ok && i0 < rows; i0 += kAtOnce * step) {
      int4 g[kAtOnce], u[kAtOnce];
#pragma unroll
      for (int z = 0; z < kAtOnce; ++z) g[z] = u[z] = make_int4(0, 0, 0, 0);
      for (uint32_t r = 0; r < splits; ++r) {
        const uint32_t from = in_cta(sums + mine, r);
        int4 p[kAtOnce], q[kAtOnce];
#pragma unroll
        for (int z = 0; z < kAtOnce; ++z) {
          const int i = min(i0 + z * step, a.n - 1);  // (a row that is not there is read from the last)
          p[z] = load_cluster(from + i * 512);
          if (SILU) q[z] = load_cluster(from + i * 512 + 64 * 4);
        }
#pragma unroll
        for (int z = 0; z < kAtOnce; ++z) {
          g[z].x += p[z].x, g[z].y += p[z].y, g[z].z += p[z].z, g[z].w += p[z].w;
          if (SILU) u[z].x += q[z].x, u[z].y += q[z].y, u[z].z += q[z].z, u[z].w += q[z].w;
        }
      }
#pragma unroll
      for (int z = 0; z < kAtOnce; ++z) {
        const int i = i0 + z * step;
        if (i >= rows) break;
        const float xs = a.xs[row0 + i];
        const int gs[4] = {g[z].x, g[z].y, g[z].z, g[z].w}, us[4] = {u[z].x, u[z].y, u[z].z, u[z].w};
        uint16_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v = int8_scaled(gs[j], xs, s0[j]);
          if (SILU)
            v = int8_silu_mul(v, int8_scaled(us[j], xs, s1[j]));
          else if (a.bias)
            v = __fadd_rn(v, s1[j]);
          b[j] = f32_to_bf16_bits(v);
        }
        uint16_t* y = a.y + (int64_t)(row0 + i) * a.cols + col;
        if (a.cols % 4 == 0) {
          if (col < a.cols)
            *reinterpret_cast<uint2*>(y) = make_uint2(b[0] | ((uint32_t)b[1] << 16), b[2] | ((uint32_t)b[3] << 16));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (col + j < a.cols) y[j] = b[j];
        }
      }
    }
  }
  __syncwarp();    // (half warps leave the loop above on their own; the barrier wants whole warps)
  cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, columns);
  }
}

// ----------------------------------------------------------------- host

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

// Rows of k codes, 128 codes of box_rows rows at a time.
bool encode_rows(CUtensorMap* map, const void* p, int64_t rows, int64_t k, int box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)k};
  cuuint32_t box[2] = {kChunkK, (cuuint32_t)box_rows}, estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// About how long a launch takes, in ns, by what it was fitted to: n x k weights of 512^2 to 16384 x 4096 and 5120 x
// 17408, 2 to 128 rows, codes given, in a graph.
int64_t stream_ns(int64_t cols, int64_t k, bool silu) { return (silu ? 2 : 1) * cols * k / 6200; }  // of the weights

struct PairPlan {
  int tile_n;
  int64_t ns;
};

// The columns of a tile: wide ones take fewer cycles a product, but may leave pairs of SMs idle in the last wave.
// A chunk of K measures 400 cycles for up to 80 columns, and 300 + 1.25 a column from there (64 pairs of SMs at a time; 512
// at 256 columns by the MMAs alone).  512 rows, 5120 x 17408, tiles of 96, 128, 160, 192, 256: 63, 64, 42, 44, 48 us; with 160
// the tensor pipe is 57% busy, and 450 MB come through L2, 10.5 TB/s.
PairPlan pair_plan(int64_t m, int64_t cols, int64_t k, bool silu) {
  const int clusters = device_sms() / 2;
  const int64_t kc = ceil_div(k, kChunkK), m_tiles = ceil_div(m, kPairRows);
  int64_t least = INT64_MAX;
  PairPlan best{};
  for (int n = 256; n >= 64; n -= 32) {
    const int64_t waves = ceil_div(m_tiles * ceil_div(cols, silu ? n / 2 : n), clusters);
    const int64_t cycles = waves * kc * std::max(400, 300 + 5 * n / 4) + 4 * n;
    if (cycles < least) least = cycles, best.tile_n = n;
  }
  const int64_t loop = least * 10 / 19, stream = stream_ns(cols, k, silu);
  best.ns = 2800 + std::max(loop, stream) + std::min(loop, stream) / 2;
  return best;
}

struct FewPlan {
  int splits;
  int blocks, n;  // of rows, n each
  int64_t ns;
};

constexpr int64_t kFewBlock = 128;  // rows of a CTA, at most: their sums are two thirds of the ring

// Clusters of 1, 2, ... CTAs that are resident at a time, an SM each or two an SM (measured on 148 SMs; a cluster stays
// within a part of the GPU; elsewhere the estimate, and with it the cut, is only less good).  The most CTAs that start at once: with one more wave of clusters 5120 x 17408 takes
// 24 us, cut into 8, and 18.0, cut into 6.  Short ranges of K do better with one CTA an SM, beside which the next
// kernel's can start: 4096 x 4096 cut into 4 and 8 6.5 and 7.2 us, 4096 x 12288 13.7 and 12.0.
FewPlan few_plan(int64_t m, int64_t cols, int64_t k, bool silu) {
  constexpr int kOneAnSm[] = {148, 74, 45, 33, 26, 22, 15, 15}, kTwoAnSm[] = {296, 148, 90, 68, 54, 45, 36, 33};
  FewPlan p;
  p.blocks = (int)ceil_div(m, kFewBlock);
  p.n = (int)ceil_div(ceil_div(m, p.blocks), 16) * 16;
  const int64_t tiles = p.blocks * ceil_div(cols, silu ? 64 : 128), kc = ceil_div(k, kChunkK);
  int one = 1, two = 1;
  for (int c = 2; c <= kFewMaxSplits && c <= kc; ++c) {
    if (tiles <= kOneAnSm[c - 1]) one = c;
    if (tiles <= kTwoAnSm[c - 1]) two = c;
  }
  p.splits = ceil_div(kc, one) <= 12 ? one : two;
  const int64_t rounds = ceil_div(tiles, kTwoAnSm[p.splits - 1]), loop = (250 + 13 * p.n / 10) * rounds * ceil_div(kc, p.splits);
  p.ns = 3400 + 200 * p.splits + 40 * p.n + std::max(loop, stream_ns(cols, k, silu));
  return p;
}

template <bool SILU>
cudaError_t launch_pair(const Int8Product& p, cudaStream_t s) {
  const int64_t cols = SILU ? p.n / 2 : p.n;
  const int clusters = device_sms() / 2;
  PairArgs a{p.xs, p.ws, p.bias, p.y, p.m, cols, (int)ceil_div(p.k, kChunkK), 256, (int)ceil_div(p.m, kPairRows), 0, 0, p.first};
  a.tile_n = pair_plan(p.m, cols, p.k, SILU).tile_n;
  a.n_tiles = (int)ceil_div(cols, SILU ? a.tile_n / 2 : a.tile_n);
  a.stages = std::min(kPairMaxStages, kPairRing / (kPairUnit * (kPairOperand + a.tile_n / 2 * kChunkK)));
  CUtensorMap xmap, wmap;
  if (!encode_rows(&xmap, p.x, p.m, p.k, 128) || !encode_rows(&wmap, p.w, p.n, p.k, a.tile_n / 2)) return cudaErrorInvalidValue;
  auto kern = int8_pair_kernel<SILU>;
  // set on every launch: the attribute belongs to the current device's context
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
  return launch_pdl(kern, dim3((unsigned)(2 * (tiles < clusters ? tiles : clusters))), dim3(kPairThreads), kPairSmem, s, xmap,
                    wmap, a);
}

template <bool SILU>
cudaError_t launch_few(const Int8Product& p, cudaStream_t s) {
  const int64_t cols = SILU ? p.n / 2 : p.n, tiles = ceil_div(cols, SILU ? 64 : 128);
  const FewPlan plan = few_plan(p.m, cols, p.k, SILU);
  FewArgs a{p.xs, p.ws, p.bias, p.y, cols, p.m, (int)ceil_div(p.k, kChunkK), plan.n, 0, p.first};
  a.stages = std::min(kFewMaxStages, kFewRing / (kFewWeights + a.n * kChunkK));
  const unsigned splits = (unsigned)plan.splits;
  CUtensorMap xmap, wmap;
  if (!encode_rows(&xmap, p.x, p.m, p.k, a.n) || !encode_rows(&wmap, p.w, p.n, p.k, SILU ? 64 : 128)) return cudaErrorInvalidValue;
  auto kern = int8_few_kernel<SILU>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_clusters(kern, dim3((unsigned)(tiles * splits), (unsigned)plan.blocks), splits, dim3(kFewThreads), kFewSmem, s, xmap, wmap, a);
}

constexpr int64_t kFewRows = 512;

// Few rows of large weights are cut along K; small weights, whose tiles the pairs of SMs take in one wave, are not worth
// a cluster's exchange of sums.  Cut and in pairs, in us: 512 x 512, 2 and 128 rows 3.7, 7.4 and 3.6, 3.9; 2048 x 2048, 2,
// 16, 32, 128 rows 5.3, 6.3, 6.9, 9.8 and 7.2, 6.0, 6.0, 6.1; 4096 x 4096, 16, 64, 128 rows 7.5, 8.5, 11.9 and 13, 10.9,
// 11.1; 5120 x 17408, 128 rows 26 and 34.  In blocks of rows: 225 rows of 576 x 12256 12.2 and 23.8, of 4096 x 4096 13.8
// and 11.4; 512 of 1024 x 8192 14.5 and 17.4, of 5120 x 17408 63 and 43.
bool use_few(int64_t m, int64_t cols, int64_t k, bool silu) {
  return m <= kFewRows && few_plan(m, cols, k, silu).ns < pair_plan(m, cols, k, silu).ns;
}

}  // namespace

ffn_int8_plan int8_product_plan(int64_t m, int64_t n, int64_t k, bool silu_mul) {
  const int64_t cols = silu_mul ? n / 2 : n;
  if (use_few(m, cols, k, silu_mul)) {
    const FewPlan f = few_plan(m, cols, k, silu_mul);
    const int64_t tiles = ceil_div(cols, silu_mul ? 64 : 128);
    return ffn_int8_plan{FFN_INT8_CLUSTERS, f.n, 128, f.splits, (int)(tiles * f.splits * f.blocks), 1};
  }
  const int tile_n = pair_plan(m, cols, k, silu_mul).tile_n;
  const int64_t tiles = ceil_div(m, kPairRows) * ceil_div(cols, silu_mul ? tile_n / 2 : tile_n), pairs = std::min<int64_t>(tiles, device_sms() / 2);
  return ffn_int8_plan{FFN_INT8_PAIRS, kPairRows, tile_n, 1, (int)(2 * pairs), (int)ceil_div(tiles, pairs)};
}

cudaError_t launch_int8_product(const Int8Product& p, cudaStream_t s) {
  ProfScope prof(s, p.silu_mul ? "int8_gate_up" : "int8_product");
  if (use_few(p.m, p.silu_mul ? p.n / 2 : p.n, p.k, p.silu_mul)) return p.silu_mul ? launch_few<true>(p, s) : launch_few<false>(p, s);
  return p.silu_mul ? launch_pair<true>(p, s) : launch_pair<false>(p, s);
}

cudaError_t read_int8_device_error(int* flags, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_int8_device_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_int8_device_error, &zero, sizeof(int));
  return e;
}

}  // namespace ffn
