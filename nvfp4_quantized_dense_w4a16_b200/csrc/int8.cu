// 8-bit integer part of the C ABI: argument checks, workspace carving and
// dispatch of ffn_int8_quantize, ffn_int8_linear and ffn_int8_forward.
#include "int8.h"

#include "ffn_nvfp4.h"
#include "moe.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1u)) == 0; }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool valid_k(int64_t k) { return k > 0 && k % 32 == 0; }

// Rows and columns fit the grids' 31 bits, and a buffer's elements 2^40.
bool valid_size(int64_t rows, int64_t columns) {
  return rows <= INT32_MAX / 2 && columns <= INT32_MAX / 2 && (rows == 0 || columns <= ((int64_t)1 << 40) / rows);
}

struct Carve {
  size_t xq = 0, xs = 0, h = 0, hq = 0, hs = 0, total = 0;
};

size_t take(size_t& off, size_t bytes) {
  const size_t at = off;
  off += round_up(bytes, 256);
  return at;
}

// inter = 0: one projection.
Carve carve(int64_t m, int64_t k, int64_t inter) {
  Carve c;
  c.xq = take(c.total, (size_t)m * k);
  c.xs = take(c.total, sizeof(float) * m);
  if (inter > 0) {
    c.h = take(c.total, (size_t)m * inter * 2);
    c.hq = take(c.total, (size_t)m * inter);
    c.hs = take(c.total, sizeof(float) * m);
  }
  return c;
}

// A product whose rows are quantised first, into `codes` and `scales`, if they have no scales.
cudaError_t product(ffn::Int8Product p, uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  if (ffn::int8_gemv_serves(p.m, p.k)) return ffn::launch_int8_gemv(p, s);
  if (!p.xs) {
    int8_t* xq = reinterpret_cast<int8_t*>(codes);
    float* xs = reinterpret_cast<float*>(scales);
    const cudaError_t e = ffn::launch_int8_quantize(p.x, p.m, p.k, p.k, xq, xs, s);
    if (e != cudaSuccess) return e;
    p.x = xq;
    p.xs = xs;
    p.first = false;
  }
  return ffn::launch_int8_product(p, s);
}

ffn_status check_linear(int64_t m, int64_t n, int64_t k) {
  if (m < 0) return FFN_ERR_INVALID_ARG;
  if (n <= 0 || !valid_k(k)) return FFN_ERR_SHAPE;
  if (k > FFN_INT8_MAX_K) return FFN_ERR_UNSUPPORTED;
  return valid_size(m, k) && valid_size(m, n) && valid_size(n, k) ? FFN_OK : FFN_ERR_SHAPE;
}

ffn_status check_layer(int64_t m, int64_t hidden, int64_t inter) {
  if (m < 0) return FFN_ERR_INVALID_ARG;
  if (!valid_k(hidden) || !valid_k(inter)) return FFN_ERR_SHAPE;
  if (hidden > FFN_INT8_MAX_K || inter > FFN_INT8_MAX_K) return FFN_ERR_UNSUPPORTED;
  return valid_size(m, hidden) && valid_size(m, inter) ? FFN_OK : FFN_ERR_SHAPE;
}

}  // namespace

extern "C" {

ffn_status ffn_int8_quantize(const void* x_bf16, int64_t m, int64_t k, int64_t row_stride, int8_t* codes,
                             float* scales, void* stream) {
  if (m < 0) return FFN_ERR_INVALID_ARG;
  if (!valid_k(k)) return FFN_ERR_SHAPE;
  if (row_stride < k) return FFN_ERR_INVALID_ARG;
  if (!valid_size(m, row_stride)) return FFN_ERR_SHAPE;
  if (m == 0) return FFN_OK;
  if (!x_bf16 || !codes || !scales) return FFN_ERR_INVALID_ARG;
  if (!aligned16(x_bf16) || row_stride % 8 || !aligned16(codes) || !aligned(scales, 4)) return FFN_ERR_ALIGNMENT;
  if (ffn_status st = ffn::moe_precheck()) return st;
  return ffn::moe_status(
      ffn::launch_int8_quantize(x_bf16, m, k, row_stride, codes, scales, reinterpret_cast<cudaStream_t>(stream)));
}

ffn_status ffn_int8_linear_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes) return FFN_ERR_INVALID_ARG;
  if (ffn_status st = check_linear(m, n, k)) return st;
  *bytes = carve(m, k, 0).total;
  return FFN_OK;
}

ffn_status ffn_int8_linear(const void* x, const float* x_scales, int64_t m, const int8_t* w, const float* w_scales,
                           const void* bias, int64_t n, int64_t k, void* y, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (ffn_status st = check_linear(m, n, k)) return st;
  if (m == 0) return FFN_OK;
  if (!x || !w || !w_scales || !y) return FFN_ERR_INVALID_ARG;
  const Carve c = carve(m, k, 0);
  if (!x_scales && (!workspace || workspace_bytes < c.total)) return FFN_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned(x_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(bias, 2) || (!x_scales && !aligned16(workspace)))
    return FFN_ERR_ALIGNMENT;
  if (ffn_status st = ffn::moe_precheck()) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const ffn::Int8Product p{x, x_scales, m, w, w_scales, static_cast<const uint16_t*>(bias), n, k, static_cast<uint16_t*>(y), false, true};
  return ffn::moe_status(product(p, ws + c.xq, ws + c.xs, s));
}

ffn_status ffn_int8_projection_plan(int64_t m, int64_t n, int64_t k, int role, ffn_int8_plan* out) {
  if (!out || role < FFN_ROLE_LINEAR || role > FFN_ROLE_DOWN) return FFN_ERR_INVALID_ARG;
  if (ffn_status st = check_linear(m, n, k)) return st;
  const bool gate_up = role == FFN_ROLE_GATE_UP;
  if (gate_up && n % 2) return FFN_ERR_SHAPE;
  *out = ffn_int8_plan{};
  if (m > 0) *out = ffn::int8_gemv_serves(m, k) ? ffn::int8_gemv_plan(n, k, gate_up) : ffn::int8_product_plan(m, n, k, gate_up);
  return FFN_OK;
}

ffn_status ffn_int8_workspace_size(int64_t m, int64_t hidden, int64_t inter, size_t* bytes) {
  if (!bytes) return FFN_ERR_INVALID_ARG;
  if (ffn_status st = check_layer(m, hidden, inter)) return st;
  *bytes = carve(m, hidden, inter).total;
  return FFN_OK;
}

ffn_status ffn_int8_forward(const void* x, const float* x_scales, int64_t m, int64_t hidden, int64_t inter,
                            const int8_t* gate_up, const float* gate_up_scales, const int8_t* down,
                            const float* down_scales, void* out, void* workspace, size_t workspace_bytes,
                            void* stream) {
  if (ffn_status st = check_layer(m, hidden, inter)) return st;
  if (m == 0) return FFN_OK;
  if (!x || !gate_up || !gate_up_scales || !down || !down_scales || !out) return FFN_ERR_INVALID_ARG;
  const Carve c = carve(m, hidden, inter);
  if (!workspace || workspace_bytes < c.total) return FFN_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(gate_up) || !aligned16(down) || !aligned16(out) || !aligned16(workspace) ||
      !aligned(x_scales, 4) || !aligned(gate_up_scales, 4) || !aligned(down_scales, 4))
    return FFN_ERR_ALIGNMENT;
  if (ffn_status st = ffn::moe_precheck()) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + c.h);
  cudaError_t e = product(ffn::Int8Product{x, x_scales, m, gate_up, gate_up_scales, nullptr, 2 * inter, hidden, h, true, true},
                          ws + c.xq, ws + c.xs, s);
  if (e == cudaSuccess)
    e = product(ffn::Int8Product{h, nullptr, m, down, down_scales, nullptr, hidden, inter, static_cast<uint16_t*>(out), false, false},
                ws + c.hq, ws + c.hs, s);
  return ffn::moe_status(e);
}

}  // extern "C"
