// Host-side declarations of the mixture-of-experts operators (routing,
// products by expert, the experts' layer).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ffn_nvfp4.h"

namespace ffn {

inline ffn_status moe_status(cudaError_t e) {
  if (e == cudaSuccess) return FFN_OK;
  cudaGetLastError();
  return FFN_ERR_CUDA;
}

// Pick up errors of earlier asynchronous work before enqueuing more.
inline ffn_status moe_precheck() { return moe_status(cudaPeekAtLastError()); }

// SMs of the current device (B200's, where there is none).
inline int device_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

// Stacked experts as the kernels read them: tiles of 64 rows (moe_decode.cuh).
int experts_tiles(int64_t rows);
size_t experts_tile_bytes(int64_t rows, int64_t k);
cudaError_t launch_tile_experts(const void* codes, const void* scales, int64_t weights, int64_t rows, int64_t k,
                                uint8_t* out, cudaStream_t s);
struct ExpertsView {
  const uint8_t* tiles = nullptr;  // [E][wtiles][kc][2304]; gate and up: [E][2][wtiles][kc][2304]
  const float* gs = nullptr;       // [E], or [E][2] (gate, up)
  int experts = 0, kc = 0;
  int wtiles = 0;                  // 64-row tiles of n (gate and up: of inter)
  int64_t n = 0, k = 0;            // logical dims (n = 2 * inter for gate and up)
  bool gate_up = false;
};

// Which rows go to which expert, for pairs p = row * top_k + slot with an id
// in [0, E): device arrays in the caller's workspace.
struct MoePlan {
  int* offsets;  // [E + 1]: expert e owns order[offsets[e] .. offsets[e + 1])
  int* order;    // [pairs]: the pairs, expert by expert, then those without one
  int* tiles;    // [0]: number of tiles; then per tile {expert, first, rows}
};

// Most tiles of `rows` rows that `pairs` pairs over E experts can fill.
inline int64_t moe_max_tiles(int64_t pairs, int64_t experts, int rows) {
  return pairs / rows + (pairs < experts ? pairs : experts);
}

cudaError_t launch_moe_plan(const int32_t* ids, int64_t pairs, int experts, int tile_rows, const MoePlan& p,
                            cudaStream_t s);

enum class ExpertsOut : int {
  kBf16 = 0,     // y[p, :] = bf16(gs * acc)
  kSiluMul = 1,  // h[p, :] = bf16(silu(g) * u), gate and up weights
  kF32 = 2       // y[p, :] = gs * acc, fp32
};

// Up to this many pairs the kernels for few rows read the ids themselves, a lane
// per pair: no plan is needed, and the down products make the sum.  The layer so
// and with a plan, in us: 8 of 64 experts of 2048 x 1024, 1, 2 and 4 rows 15.9,
// 26.9 and 37.9 against 23.0, 32.0 and 40.7; 2 of 8 of 4096 x 12288, 1 row 48.9
// against 56.4.  From about 8 rows the two bf16 parts of h, for which a tile holds
// half the rows, cost more than the plan: 8 and 16 rows of those 168 and 218
// against 150 and 167, 32 rows of one pick each of the small ones 51 against 39.
// The parts are what the layer documents for so few pairs.
constexpr int kFewPairs = 32;
// Rows of a plan's tiles for launch_experts_rows: 8 or 16.  The layer of 64 experts
// of 2048 x 1024 with tiles of 8 and of 16 at 2, 4, 5, 6, 7 and 8 rows an expert,
// in us: 65, 71, 77, 80, 87, 95.5 and 80, 86, 87, 89, 90, 90; 8 of 4096 x 6144 at 4,
// 5, 6, 7, 8: 96, 97, 108, 120, 132 and 117, 117, 118, 119, 119.
inline int64_t last_narrow_pairs(int64_t experts) { return 5 * experts; }
inline int rows_tile(int64_t pairs, int64_t experts) { return pairs <= last_narrow_pairs(experts) ? 8 : 16; }

// How many ranges of K the down products are cut into for `tiles` tiles of
// rows, so that the items fill the SMs evenly; each range leaves its own sums.
constexpr int kMaxSplits = 8;
int rows_splits(const ExpertsView& w, int64_t tiles, int sms);

// The weighted sum over a row's experts, made by the down products themselves
// (kF32, at most kFewPairs pairs): out = bf16(sum_j weights[j] * y[j]).
struct RowsSum {
  const float* weights;
  void* out;
  int* arrived;  // [rows_units(w)] zeroed words
};
inline int rows_units(const ExpertsView& w) { return w.gate_up ? w.wtiles : (w.wtiles + 1) / 2; }

// Products of few rows per expert: row p of the input is x[p / row_div].  With
// at most kFewPairs pairs kSiluMul writes h [pairs, 2, inter], the bf16 value
// and (bf16) what it lost, and a kF32 launch with `sum` reads it so.
// kF32 writes y [splits, pairs, n].  kBf16 also writes zeros for the pairs
// without an expert.  `zero`: words that kSiluMul clears for a later launch.
cudaError_t launch_experts_rows(const void* x, int row_div, const ExpertsView& w, const int32_t* ids, const MoePlan& p,
                                int64_t pairs, int top_k, ExpertsOut mode, int splits, void* out, int* zero,
                                int zero_count, const RowsSum* sum, cudaStream_t s);
// out[i, :] = bf16(sum_j weights[i, j] * y[i * top_k + j, :]), j ascending, y the sum of its splits.
cudaError_t launch_moe_combine(const float* y, int splits, const int32_t* ids, const float* weights, int64_t m,
                               int top_k, int experts, int64_t hidden, void* out, cudaStream_t s);
// Many rows per expert, on the tensor cores (plan with kTcTile rows a tile).
// xs holds the rows sorted by expert, and kTcTile more rows of any content;
// kSiluMul writes h in the same order, the others write row p of the pair.
constexpr int kTcTile = 256;
cudaError_t launch_experts_tc(const void* xs, const ExpertsView& w, const MoePlan& p, int64_t pairs, ExpertsOut mode,
                              void* out, cudaStream_t s);
// xs[q, :] = x[order[q] / row_div, :]; with y, zeros to its rows without an expert.
cudaError_t launch_moe_gather(const void* x, int row_div, const MoePlan& p, int experts, int64_t pairs, int64_t k,
                              void* xs, void* y, int64_t n, cudaStream_t s);
// Error bits of these kernels' bounded waits, as read_device_error.
cudaError_t read_moe_device_error(int* flags, bool clear);
cudaError_t read_rows_device_error(int* flags, bool clear);

}  // namespace ffn
