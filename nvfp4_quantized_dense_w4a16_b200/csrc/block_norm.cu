// What stands between two layers in one pass over the rows: the norm after a
// layer, gate and residual, the norm before the next layer and, if asked, its
// quantisation to int8 (ffn_block_norm).
//
// A row stays in registers from its loads to its stores: a warp holds a short
// row, a CTA a longer one.  Each norm is then one sum over the row (two for a
// layer norm: the mean, and the squares of what differs from it).  It is bound by
// its memory traffic.
#include "ffn_nvfp4.h"
#include "int8.cuh"
#include "launch.cuh"
#include "moe.h"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using namespace sm100;

struct NormArgs {
  const void *weight, *bias;
  float eps, offset;
  bool on, layer, bf16;
};

struct BlockArgs {
  int64_t m;
  int hidden;
  const uint16_t* y;
  const void *gate, *residual;
  void *residual_out, *out;
  float* out_scales;
  int64_t y_stride, gate_row_stride, residual_stride, residual_out_stride, out_stride;
  float residual_scale, branch_scale;
  int gate_activation;
  bool gate_bf16, gate_cols;  // (one gate for each column, or for the row)
  NormArgs post, pre;
};

// V consecutive values of a tensor as fp32.
template <int V>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&o)[V]) {
  if (V == 8) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      o[2 * i] = __uint_as_float(w[i] << 16);
      o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    o[0] = bf16_bits_to_float(*p);
  }
}

template <int V>
__device__ __forceinline__ void load_f32(const float* p, float (&o)[V]) {
  if (V == 8) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 t = reinterpret_cast<const float4*>(p)[i];
      o[4 * i] = t.x, o[4 * i + 1] = t.y, o[4 * i + 2] = t.z, o[4 * i + 3] = t.w;
    }
  } else {
    o[0] = *p;
  }
}

template <int V>
__device__ __forceinline__ void load_any(const void* p, bool bf16, int64_t at, float (&o)[V]) {
  if (bf16)
    load_bf16<V>(static_cast<const uint16_t*>(p) + at, o);
  else
    load_f32<V>(static_cast<const float*>(p) + at, o);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}

template <int V>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&v)[V]) {
  if (V == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1 % V]), pack_bf16(v[2 % V], v[3 % V]),
                                              pack_bf16(v[4 % V], v[5 % V]), pack_bf16(v[6 % V], v[7 % V]));
  else
    *p = f32_to_bf16_bits(v[0]);
}

// Sums and maxima over the threads that hold a row: a warp, or the CTA, whose
// warps leave their parts in one of two sets of words in turn, so that one
// barrier is enough.
template <bool WARP>
struct Row {
  uint32_t* parts;
  int turn = 0;
  template <typename T, typename F>
  __device__ __forceinline__ T over(T v, F f) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (WARP) return v;
    T* p = reinterpret_cast<T*>(parts + 32 * turn);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
    __syncthreads();
    v = p[0];
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) v = f(v, p[w]);
    return v;
  }
  __device__ __forceinline__ float sum(float v) {
    return over(v, [](float a, float b) { return a + b; });
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    return over(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
  }
};

// v = norm(v) of a row's N sets of V values, set i of this thread at column at(i).
// The squares of values beyond 2^64 would pass fp32's range: such a row is
// scaled by 2^-75 and gone over once more.
template <bool WARP, int V, int N, typename At>
__device__ __forceinline__ void norm_row(Row<WARP>& row, const NormArgs& a, int hidden, float (&v)[N][V], At at) {
  const float share = 1.0f / (float)hidden;
  float c = 1.0f, mean, squares;
  for (;;) {
    mean = 0.0f;
    if (a.layer) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (at(i) < hidden)
#pragma unroll
          for (int j = 0; j < V; ++j) s = fmaf(v[i][j], c, s);
      mean = row.sum(s) * share;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < hidden)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = fmaf(v[i][j], c, -mean);
          s = fmaf(d, d, s);
        }
    squares = row.sum(s);
    if (squares < __uint_as_float(0x7f800000u) || c != 1.0f) break;
    c = 2.6469780e-23f;  // 2^-75
  }
  const float inv = rsqrtf(fmaf(squares, share, a.eps * (c * c)));
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at(i) < hidden) {
      float w[V], b[V];
      if (a.weight) load_any<V>(a.weight, a.bf16, at(i), w);
      if (a.bias) load_any<V>(a.bias, a.bf16, at(i), b);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float t = fmaf(v[i][j], c, -mean) * inv;
        if (a.weight) t *= a.offset + w[j];
        if (a.bias) t += b[j];
        v[i][j] = t;
      }
    }
}

__device__ __forceinline__ float gate_value(float g, int activation) {
  if (activation == FFN_GATE_SIGMOID) return 1.0f / (1.0f + expf(-g));
  if (activation == FFN_GATE_TANH) return tanhf(g);
  return g;
}

// R: the residual is bf16; WARP: a warp for each row, else the CTA; V: values of an
// access (8, or 1 where a tensor's rows are not whole 16 bytes); N: accesses a thread.
template <bool R, bool WARP, int V, int N, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_kernel(const BlockArgs a) {
  __shared__ uint32_t parts[64];
  Row<WARP> row{parts};
  const int threads = WARP ? 32 : blockDim.x, mine = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int per_cta = WARP ? blockDim.x >> 5 : 1;
  auto at = [&](int i) { return V * (mine + i * threads); };
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t r = blockIdx.x * (int64_t)per_cta + (WARP ? threadIdx.x >> 5 : 0); r < a.m;
       r += (int64_t)gridDim.x * per_cta) {
    float res[N][V], z[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < a.hidden) {
        if (a.y) load_bf16<V>(a.y + r * a.y_stride + at(i), z[i]);
        load_any<V>(a.residual, R, r * a.residual_stride + at(i), res[i]);
      }
    if (a.y) {
      if (a.post.on) norm_row<WARP, V, N>(row, a.post, a.hidden, z, at);
      float g1[1] = {1.0f};
      if (a.gate && !a.gate_cols) {
        load_any<1>(a.gate, a.gate_bf16, r * a.gate_row_stride, g1);
        g1[0] = gate_value(g1[0], a.gate_activation);
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (at(i) < a.hidden) {
          float g[V];
          if (a.gate && a.gate_cols) load_any<V>(a.gate, a.gate_bf16, r * a.gate_row_stride + at(i), g);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float gate = a.gate && a.gate_cols ? gate_value(g[j], a.gate_activation) : g1[0];
            const float s = fmaf(a.residual_scale, res[i][j], a.branch_scale * (gate * z[i][j]));
            res[i][j] = R ? bf16_round(s) : s;
          }
          if (a.residual_out) {
            if (R) {
              store_bf16<V>(static_cast<uint16_t*>(a.residual_out) + r * a.residual_out_stride + at(i), res[i]);
            } else {
              float* o = static_cast<float*>(a.residual_out) + r * a.residual_out_stride + at(i);
              if (V == 8) {
#pragma unroll
                for (int q = 0; q < V / 4; ++q)
                  reinterpret_cast<float4*>(o)[q] =
                      make_float4(res[i][(4 * q) % V], res[i][(4 * q + 1) % V], res[i][(4 * q + 2) % V], res[i][(4 * q + 3) % V]);
              } else {
                *o = res[i][0];
              }
            }
          }
        }
    }
    if (!a.pre.on) continue;
    norm_row<WARP, V, N>(row, a.pre, a.hidden, res, at);
    if (!a.out_scales) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (at(i) < a.hidden) store_bf16<V>(static_cast<uint16_t*>(a.out) + r * a.out_stride + at(i), res[i]);
      continue;
    }
    // The codes are those of the row as it would be stored in bf16.
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < a.hidden)
#pragma unroll
        for (int j = 0; j < V; ++j) top = max(top, (uint32_t)(f32_to_bf16_bits(res[i][j]) & 0x7fffu));
    const Int8Row q(row.max(top));
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < a.hidden) {
        int8_t* o = static_cast<int8_t*>(a.out) + r * a.out_stride + at(i);
        if (V == 8)
          *reinterpret_cast<uint2*>(o) =
              int8_encode8(q, make_uint4(pack_bf16(res[i][0], res[i][1 % V]), pack_bf16(res[i][2 % V], res[i][3 % V]),
                                         pack_bf16(res[i][4 % V], res[i][5 % V]), pack_bf16(res[i][6 % V], res[i][7 % V])));
        else
          *o = (int8_t)q.code(bf16_round(res[i][0]));
      }
    if (mine == 0) a.out_scales[r] = q.scale;
  }
}

template <bool R, bool WARP, int V, int N, int THREADS>
cudaError_t launch_one(const BlockArgs& a, int threads, cudaStream_t s) {
  const int64_t per_cta = WARP ? threads / 32 : 1;
  const int64_t ctas = (a.m + per_cta - 1) / per_cta, most = (int64_t)device_sms() * (2048 / threads);
  ProfScope prof(s, "block_norm");
  return launch_pdl(block_norm_kernel<R, WARP, V, N, THREADS>, dim3((unsigned)(ctas < most ? ctas : most)), dim3(threads),
                    0, s, a);
}

int round_up_32(int v) { return (v + 31) / 32 * 32; }

// Threads and accesses for a row: as few accesses as keep a CTA to 512 threads.
template <bool R>
cudaError_t launch_rows(const BlockArgs& a, bool vec, cudaStream_t s) {
  const int h = a.hidden;
  if (!vec) {
    if (h <= 256) return launch_one<R, true, 1, 8, 256>(a, 256, s);
    if (h <= 4096) return launch_one<R, false, 1, 8, 512>(a, round_up_32((h + 7) / 8), s);
    return launch_one<R, false, 1, 32, 1024>(a, round_up_32((h + 31) / 32), s);
  }
  if (h <= 256) return launch_one<R, true, 8, 1, 256>(a, 256, s);
  if (h <= 512) return launch_one<R, true, 8, 2, 256>(a, 256, s);
  if (h <= 1024) return launch_one<R, true, 8, 4, 256>(a, 256, s);
  if (h <= 8192) return launch_one<R, false, 8, 2, 512>(a, round_up_32((h + 15) / 16), s);
  if (h <= 16384) return launch_one<R, false, 8, 4, 512>(a, round_up_32((h + 31) / 32), s);
  return launch_one<R, false, 8, 4, 1024>(a, round_up_32((h + 31) / 32), s);
}

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1u)) == 0; }
bool valid_type(int t) { return t == FFN_VALUE_F32 || t == FFN_VALUE_BF16; }
unsigned size_of(int type) { return type == FFN_VALUE_BF16 ? 2 : 4; }
bool finite(float v) { return v - v == 0.0f; }

ffn_status check_norm(const ffn_norm* n) {
  if (!n) return FFN_OK;
  if ((n->kind != FFN_NORM_RMS && n->kind != FFN_NORM_LAYER) || !valid_type(n->type) || !finite(n->eps) || !(n->eps > 0.0f) ||
      !finite(n->offset))
    return FFN_ERR_INVALID_ARG;
  return FFN_OK;
}

NormArgs norm_args(const ffn_norm* n) {
  NormArgs a = {};
  if (!n) return a;
  a.on = true;
  a.weight = n->weight;
  a.bias = n->bias;
  a.eps = n->eps;
  a.offset = n->offset;
  a.layer = n->kind == FFN_NORM_LAYER;
  a.bf16 = n->type == FFN_VALUE_BF16;
  return a;
}

// Whether 8 values at a time can be accessed: rows of whole 16 bytes.
bool whole(const void* p, int64_t stride) { return !p || (aligned(p, 16) && stride % 8 == 0); }

}  // namespace
}  // namespace ffn

extern "C" ffn_status ffn_block_norm(const ffn_block_norm_args* b, int64_t m, int64_t hidden, void* stream) {
  using namespace ffn;
  if (!b || m < 0 || hidden < 1) return FFN_ERR_INVALID_ARG;
  if (!valid_type(b->residual_type) || !finite(b->residual_scale) || !finite(b->branch_scale)) return FFN_ERR_INVALID_ARG;
  if (ffn_status st = check_norm(b->post)) return st;
  if (ffn_status st = check_norm(b->pre)) return st;
  if (b->gate && (!valid_type(b->gate_type) || b->gate_activation < FFN_GATE_NONE || b->gate_activation > FFN_GATE_TANH ||
                  (b->gate_col_stride != 0 && b->gate_col_stride != 1) || b->gate_row_stride < 0 ||
                  (b->gate_col_stride == 1 && b->gate_row_stride != 0 && b->gate_row_stride < hidden)))
    return FFN_ERR_INVALID_ARG;
  if (hidden > FFN_NORM_MAX_HIDDEN) return FFN_ERR_UNSUPPORTED;
  if (m == 0) return FFN_OK;  // (empty tensors have no addresses)
  if (!b->y && (b->post || b->gate || b->residual_out || b->residual_scale != 1.0f || b->branch_scale != 1.0f))
    return FFN_ERR_INVALID_ARG;
  if (!b->pre && (b->out || b->out_scales || !b->y)) return FFN_ERR_INVALID_ARG;
  if (b->residual_stride < hidden || (b->y && b->y_stride < hidden) || (b->residual_out && b->residual_out_stride < hidden) ||
      (b->pre && b->out_stride < hidden))
    return FFN_ERR_INVALID_ARG;
  if (b->out_scales && (hidden % 32 || b->out_stride != hidden)) return FFN_ERR_SHAPE;
  const int64_t most = ((int64_t)1 << 40) / m;
  if (b->residual_stride > most || (b->y && b->y_stride > most) || (b->residual_out && b->residual_out_stride > most) ||
      (b->pre && b->out_stride > most) || (b->gate && b->gate_row_stride > most))
    return FFN_ERR_SHAPE;
  if (!b->residual || (b->pre && !b->out) || (b->y && !b->residual_out && !b->pre)) return FFN_ERR_INVALID_ARG;
  const unsigned rs = size_of(b->residual_type);
  if (!aligned(b->y, 2) || !aligned(b->residual, rs) || !aligned(b->residual_out, rs) || !aligned(b->out_scales, 4) ||
      (b->out && !aligned(b->out, b->out_scales ? 8 : 2)) || (b->gate && !aligned(b->gate, size_of(b->gate_type))))
    return FFN_ERR_ALIGNMENT;
  bool vec = hidden % 8 == 0 && whole(b->y, b->y_stride) && whole(b->residual, b->residual_stride) &&
             whole(b->residual_out, b->residual_out_stride) && whole(b->out, b->out_stride) &&
             (!b->gate || b->gate_col_stride == 0 || whole(b->gate, b->gate_row_stride));
  for (const ffn_norm* n : {b->post, b->pre})
    if (n) {
      if (!aligned(n->weight, size_of(n->type)) || !aligned(n->bias, size_of(n->type))) return FFN_ERR_ALIGNMENT;
      vec = vec && aligned(n->weight, 16) && aligned(n->bias, 16);
    }
  if (ffn_status st = moe_precheck()) return st;
  BlockArgs a = {};
  a.m = m;
  a.hidden = (int)hidden;
  a.y = static_cast<const uint16_t*>(b->y);
  a.gate = b->gate;
  a.residual = b->residual;
  a.residual_out = b->residual_out;
  a.out = b->out;
  a.out_scales = b->out_scales;
  a.y_stride = b->y_stride;
  a.gate_row_stride = b->gate_row_stride;
  a.residual_stride = b->residual_stride;
  a.residual_out_stride = b->residual_out_stride;
  a.out_stride = b->out_stride;
  a.residual_scale = b->residual_scale;
  a.branch_scale = b->branch_scale;
  a.gate_activation = b->gate_activation;
  a.gate_bf16 = b->gate_type == FFN_VALUE_BF16;
  a.gate_cols = b->gate_col_stride == 1;
  a.post = norm_args(b->post);
  a.pre = norm_args(b->pre);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return moe_status(b->residual_type == FFN_VALUE_BF16 ? launch_rows<true>(a, vec, s) : launch_rows<false>(a, vec, s));
}
