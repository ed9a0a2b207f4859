// Mixture-of-experts part of the C ABI: the handle of stacked NVFP4 experts,
// argument checks, workspace carving and dispatch of ffn_nvfp4_experts_linear
// and ffn_nvfp4_moe_forward.
#include <algorithm>
#include <new>

#include "ffn_nvfp4.h"
#include "moe.h"

struct ffn_nvfp4_experts {
  int64_t experts = 0, n = 0, k = 0;
  int gate_up = 0;
  int device = 0;
  size_t bytes = 0;
  uint8_t* tiles = nullptr;
  float* gs = nullptr;
  ffn::ExpertsView view() const {
    ffn::ExpertsView v;
    v.tiles = tiles;
    v.gs = gs;
    v.experts = (int)experts;
    v.wtiles = ffn::experts_tiles(n / (gate_up ? 2 : 1));
    v.kc = (int)((k + 63) / 64);
    v.n = n;
    v.k = k;
    v.gate_up = gate_up != 0;
    return v;
  }
};

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool valid_k(int64_t k) { return k > 0 && k % 32 == 0; }

ffn_status check_device(const ffn_nvfp4_experts* w) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return FFN_ERR_CUDA;
  }
  return dev == w->device ? FFN_OK : FFN_ERR_INVALID_ARG;
}

// m * top_k pairs must fit an int, and so must the rows of every product.
bool valid_pairs(int64_t m, int top_k) { return m <= (int64_t)INT32_MAX / 2 / top_k; }

// What a call touches fits 64 bits and the grids' 31 with room to spare: 2^40
// elements of any one buffer are more than a GPU holds.
bool valid_size(int64_t pairs, int64_t columns) {
  return columns <= INT32_MAX / 2 && (pairs == 0 || columns <= ((int64_t)1 << 40) / pairs);
}

struct Carve {
  size_t offsets = 0, order = 0, tiles = 0, arrived = 0, xs = 0, h = 0, y = 0, total = 0;
  bool tc = false;
  int tile_rows = 0;
  int splits = 1;  // of the down products' K
};

// From how many rows an expert (on average) the tensor cores take over.  The
// layer with the few-row kernel and with the tensor cores, in us: 64 experts of
// 2048 x 1024 at 6, 8, 12 rows an expert 90, 96, 112 and 90, 94, 101; 8 of
// 4096 x 6144 at 8, 12, 16 rows 121, 140, 170 and 134, 139, 145; 20 of
// 1056 x 672 at 7, 10, 14 rows 32.2, 32.6, 35.5 and 31.2, 31.7, 32.6.
int64_t last_rows_pairs(int64_t experts) { return std::max((int64_t)ffn::kFewPairs, 8 * experts); }
bool use_tc(int64_t pairs, int64_t experts) { return pairs > last_rows_pairs(experts); }

size_t take(size_t& off, size_t bytes) {
  const size_t at = off;
  off += round_up(bytes, 256);
  return at;
}

// inter = 0: one projection of `hidden` columns and k, whose output is the caller's.
Carve carve(int64_t m, int top_k, int64_t experts, int64_t hidden, int64_t inter, int64_t k, int sms) {
  Carve c;
  const int64_t pairs = m * top_k;
  if (pairs == 0) return c;
  c.tc = use_tc(pairs, experts);
  c.tile_rows = c.tc ? ffn::kTcTile : ffn::rows_tile(pairs, experts);
  const int64_t padded = pairs + ffn::kTcTile;
  size_t off = 0;
  c.offsets = take(off, sizeof(int) * (experts + 1));
  c.order = take(off, sizeof(int) * pairs);
  c.tiles = take(off, sizeof(int) * (1 + 3 * ffn::moe_max_tiles(pairs, experts, c.tile_rows)));
  c.arrived = take(off, sizeof(int) * ((hidden + 127) / 128));
  if (inter > 0 && !c.tc) {
    ffn::ExpertsView down;
    down.wtiles = ffn::experts_tiles(hidden);
    down.kc = (int)((inter + 63) / 64);
    // every pair has an expert of its own with few pairs of one row; a batch spreads over all experts
    c.splits = ffn::rows_splits(down, pairs < experts ? pairs : experts, sms);
  }
  // the sorted rows are read before the down products are written: one buffer
  const size_t xs = c.tc ? (size_t)padded * k * 2 : 0, y = inter > 0 ? (size_t)c.splits * pairs * hidden * 4 : 0;
  c.xs = c.y = take(off, xs > y ? xs : y);
  if (inter > 0) c.h = take(off, (size_t)padded * inter * 2);
  c.total = off;
  return c;
}

// A workspace's size serves every smaller batch as well, though a smaller one may
// need more: its K is cut into more ranges, its tiles have fewer rows, or other
// kernels compute it.  Between such changes the need grows with m: the last
// batches before the changes, and those of fewer pairs than experts, by which K
// is cut, hold the most.
size_t workspace_bytes(int64_t m, int top_k, int64_t experts, int64_t hidden, int64_t inter, int64_t k) {
  const int sms = ffn::device_sms();
  auto need = [&](int64_t rows) { return carve(rows, top_k, experts, hidden, inter, k, sms).total; };
  size_t most = need(m);
  for (const int64_t pairs : {ffn::last_narrow_pairs(experts), last_rows_pairs(experts)})
    if (pairs / top_k < m) most = std::max(most, need(pairs / top_k));
  if (inter > 0 && m * top_k < ffn::kMaxSplits * experts)  // (from there one sum a pair is more)
    for (int64_t rows = std::min(m, experts / top_k); rows > 0; --rows) most = std::max(most, need(rows));
  return most;
}

ffn::MoePlan plan_at(uint8_t* ws, const Carve& c) {
  ffn::MoePlan p;
  p.offsets = reinterpret_cast<int*>(ws + c.offsets);
  p.order = reinterpret_cast<int*>(ws + c.order);
  p.tiles = reinterpret_cast<int*>(ws + c.tiles);
  return p;
}

void free_experts(ffn_nvfp4_experts* w) {
  if (!w) return;
  cudaFree(w->tiles);
  cudaFree(w->gs);
  delete w;
}

}  // namespace

extern "C" {

ffn_status ffn_nvfp4_experts_create(const void* codes, const void* block_scales, const float* global_scales,
                                    int64_t experts, int64_t n, int64_t k, int gate_up, void* stream,
                                    ffn_nvfp4_experts** out) {
  if (!out) return FFN_ERR_INVALID_ARG;
  *out = nullptr;
  if (!codes || !block_scales || !global_scales || (gate_up != 0 && gate_up != 1)) return FFN_ERR_INVALID_ARG;
  if (experts < 1 || n < 1 || !valid_k(k) || (gate_up && n % 2)) return FFN_ERR_SHAPE;
  if (gate_up && (n / 2) % 32) return FFN_ERR_SHAPE;  // inter is the down projection's K
  if (experts > FFN_MOE_MAX_EXPERTS) return FFN_ERR_UNSUPPORTED;
  if (n > INT32_MAX / 2 || k > INT32_MAX / 2) return FFN_ERR_SHAPE;
  if (!aligned16(codes) || !aligned16(block_scales) || !aligned4(global_scales)) return FFN_ERR_ALIGNMENT;
  if (ffn_status st = ffn::moe_precheck()) return st;
  auto* w = new (std::nothrow) ffn_nvfp4_experts;
  if (!w) return FFN_ERR_OOM;
  w->experts = experts;
  w->n = n;
  w->k = k;
  w->gate_up = gate_up;
  const int64_t parts = gate_up ? 2 : 1, rows = n / parts;  // gate and up are tiled apart
  const size_t tile_bytes = ffn::experts_tile_bytes(rows, k);
  const size_t gs_bytes = sizeof(float) * experts * (gate_up ? 2 : 1);
  w->bytes = tile_bytes * parts * experts + gs_bytes;
  if (cudaGetDevice(&w->device) != cudaSuccess) {
    delete w;
    cudaGetLastError();
    return FFN_ERR_CUDA;
  }
  if (cudaMalloc(reinterpret_cast<void**>(&w->tiles), tile_bytes * parts * experts) != cudaSuccess ||
      cudaMalloc(reinterpret_cast<void**>(&w->gs), gs_bytes) != cudaSuccess) {
    cudaGetLastError();
    free_experts(w);
    return FFN_ERR_OOM;
  }
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(w->gs, global_scales, gs_bytes, cudaMemcpyDeviceToDevice, s);
  if (e == cudaSuccess)
    e = ffn::launch_tile_experts(codes, block_scales, experts * parts, rows, k, w->tiles, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    free_experts(w);
    return FFN_ERR_CUDA;
  }
  *out = w;
  return FFN_OK;
}

ffn_status ffn_nvfp4_experts_destroy(ffn_nvfp4_experts* w) {
  if (!w) return FFN_OK;
  const cudaError_t e = cudaDeviceSynchronize();
  free_experts(w);
  return e == cudaSuccess ? FFN_OK : FFN_ERR_CUDA;
}

ffn_status ffn_nvfp4_experts_info(const ffn_nvfp4_experts* w, int64_t* experts, int64_t* n, int64_t* k,
                                  int* is_gate_up, size_t* device_bytes) {
  if (!w) return FFN_ERR_INVALID_ARG;
  if (experts) *experts = w->experts;
  if (n) *n = w->n;
  if (k) *k = w->k;
  if (is_gate_up) *is_gate_up = w->gate_up;
  if (device_bytes) *device_bytes = w->bytes;
  return FFN_OK;
}

ffn_status ffn_nvfp4_experts_workspace_size(int64_t m, int top_k, int64_t experts, int64_t n, int64_t k,
                                            size_t* bytes) {
  if (!bytes || m < 0 || top_k < 1 || experts < 1 || n < 1) return FFN_ERR_INVALID_ARG;
  if (experts > FFN_MOE_MAX_EXPERTS) return FFN_ERR_UNSUPPORTED;
  if (!valid_k(k) || !valid_pairs(m, top_k) || !valid_size(m * top_k, n) || !valid_size(m * top_k, k)) return FFN_ERR_SHAPE;
  *bytes = workspace_bytes(m, top_k, experts, n, 0, k);
  return FFN_OK;
}

ffn_status ffn_nvfp4_experts_linear(const void* x, int64_t m, const ffn_nvfp4_experts* w, const int32_t* ids,
                                    int top_k, void* y, void* workspace, size_t workspace_bytes, void* stream) {
  if (m < 0 || !w || top_k < 1) return FFN_ERR_INVALID_ARG;
  if (w->gate_up) return FFN_ERR_UNSUPPORTED;
  if (!valid_pairs(m, top_k) || !valid_size(m * top_k, w->n) || !valid_size(m * top_k, w->k)) return FFN_ERR_SHAPE;
  if (m == 0) return FFN_OK;
  if (!x || !ids || !y) return FFN_ERR_INVALID_ARG;
  if (ffn_status st = check_device(w)) return st;
  const Carve c = carve(m, top_k, w->experts, w->n, 0, w->k, ffn::device_sms());
  if (!workspace || workspace_bytes < c.total) return FFN_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(y) || !aligned16(workspace) || !aligned4(ids)) return FFN_ERR_ALIGNMENT;
  if (ffn_status st = ffn::moe_precheck()) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const ffn::ExpertsView v = w->view();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const ffn::MoePlan p = plan_at(ws, c);
  const int64_t pairs = m * top_k;
  cudaError_t e = cudaSuccess;
  if (pairs > ffn::kFewPairs)
    e = ffn::launch_moe_plan(ids, pairs, v.experts, c.tile_rows, p, s);
  if (c.tc) {
    if (e == cudaSuccess) e = ffn::launch_moe_gather(x, top_k, p, v.experts, pairs, v.k, ws + c.xs, y, v.n, s);
    if (e == cudaSuccess) e = ffn::launch_experts_tc(ws + c.xs, v, p, pairs, ffn::ExpertsOut::kBf16, y, s);
  } else if (e == cudaSuccess) {
    e = ffn::launch_experts_rows(x, top_k, v, ids, p, pairs, top_k, ffn::ExpertsOut::kBf16, 1, y, nullptr, 0, nullptr, s);
  }
  return ffn::moe_status(e);
}

ffn_status ffn_nvfp4_moe_workspace_size(int64_t m, int top_k, int64_t experts, int64_t hidden, int64_t inter,
                                        size_t* bytes) {
  if (!bytes || m < 0 || top_k < 1 || experts < 1) return FFN_ERR_INVALID_ARG;
  if (experts > FFN_MOE_MAX_EXPERTS) return FFN_ERR_UNSUPPORTED;
  if (!valid_k(hidden) || !valid_k(inter) || !valid_pairs(m, top_k) || !valid_size(m * top_k, hidden) ||
      !valid_size(m * top_k, inter))
    return FFN_ERR_SHAPE;
  *bytes = workspace_bytes(m, top_k, experts, hidden, inter, hidden);
  return FFN_OK;
}

ffn_status ffn_nvfp4_moe_forward(const void* x, int64_t m, int64_t hidden, int64_t inter,
                                 const ffn_nvfp4_experts* gate_up, const ffn_nvfp4_experts* down,
                                 const int32_t* ids, const float* weights, int top_k, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (m < 0 || !gate_up || !down || top_k < 1) return FFN_ERR_INVALID_ARG;
  if (!valid_k(hidden) || !valid_k(inter)) return FFN_ERR_SHAPE;
  if (!gate_up->gate_up || down->gate_up) return FFN_ERR_INVALID_ARG;
  if (gate_up->n != 2 * inter || gate_up->k != hidden || down->n != hidden || down->k != inter ||
      gate_up->experts != down->experts || !valid_pairs(m, top_k) || !valid_size(m * top_k, hidden) ||
      !valid_size(m * top_k, inter))
    return FFN_ERR_SHAPE;
  if (m == 0) return FFN_OK;
  if (!x || !ids || !weights || !out) return FFN_ERR_INVALID_ARG;
  if (ffn_status st = check_device(gate_up)) return st;
  if (ffn_status st = check_device(down)) return st;
  const Carve c = carve(m, top_k, down->experts, hidden, inter, hidden, ffn::device_sms());
  if (!workspace || workspace_bytes < c.total) return FFN_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(out) || !aligned16(workspace) || !aligned4(ids) || !aligned4(weights))
    return FFN_ERR_ALIGNMENT;
  if (ffn_status st = ffn::moe_precheck()) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const ffn::ExpertsView gu = gate_up->view(), dn = down->view();
  const ffn::MoePlan p = plan_at(ws, c);
  const int64_t pairs = m * top_k;
  const ffn::ExpertsOut kSilu = ffn::ExpertsOut::kSiluMul, kF32 = ffn::ExpertsOut::kF32;
  float* y = reinterpret_cast<float*>(ws + c.y);
  cudaError_t e = cudaSuccess;
  if (pairs <= ffn::kFewPairs) {
    const ffn::RowsSum sum{weights, out, reinterpret_cast<int*>(ws + c.arrived)};
    e = ffn::launch_experts_rows(x, top_k, gu, ids, p, pairs, top_k, kSilu, 1, ws + c.h, sum.arrived, ffn::rows_units(dn),
                                 nullptr, s);
    if (e == cudaSuccess) e = ffn::launch_experts_rows(ws + c.h, 1, dn, ids, p, pairs, top_k, kF32, c.splits, y, nullptr, 0, &sum, s);
    return ffn::moe_status(e);
  }
  e = ffn::launch_moe_plan(ids, pairs, dn.experts, c.tile_rows, p, s);
  if (c.tc) {
    if (e == cudaSuccess) e = ffn::launch_moe_gather(x, top_k, p, dn.experts, pairs, hidden, ws + c.xs, nullptr, 0, s);
    if (e == cudaSuccess) e = ffn::launch_experts_tc(ws + c.xs, gu, p, pairs, kSilu, ws + c.h, s);
    if (e == cudaSuccess) e = ffn::launch_experts_tc(ws + c.h, dn, p, pairs, kF32, y, s);
  } else {
    if (e == cudaSuccess)
      e = ffn::launch_experts_rows(x, top_k, gu, ids, p, pairs, top_k, kSilu, 1, ws + c.h, nullptr, 0, nullptr, s);
    if (e == cudaSuccess)
      e = ffn::launch_experts_rows(ws + c.h, 1, dn, ids, p, pairs, top_k, kF32, c.splits, y, nullptr, 0, nullptr, s);
  }
  if (e == cudaSuccess) e = ffn::launch_moe_combine(y, c.splits, ids, weights, m, top_k, dn.experts, hidden, out, s);
  return ffn::moe_status(e);
}

}  // extern "C"
