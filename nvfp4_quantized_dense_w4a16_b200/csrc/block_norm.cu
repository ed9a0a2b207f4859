// What stands between two layers in one pass over the rows: the norm after a
// layer, gate and residual, the norm before the next layer and, if asked, its
// quantisation to int8 (ffn_block_norm).
//
// A row stays in registers from its first norm to its stores: a warp holds a short
// row, a CTA a longer one, some warps of a CTA one of many.  Each norm is then one
// sum over the row (two for a layer norm: the mean, and the squares of what differs
// from it).
//
// Few rows are a matter of latency: all loads of a row are under way before its first
// sum (one row of 4096, both norms: 5.2 -> 3.8 us in a graph).  Many are bound by their
// memory traffic if the instructions allow: 4096 rows of 5120, fp32 residual, both
// norms, a gate for each channel (252 MB) take 47 us, 5.3 TB/s, 81% of the measured copy
// rate; 16384 rows of 2048 with tanh gates of their own (336 MB) 67 us, 77% (47
// instructions a value, 38 in the former).  With a CTA a row and plain loads those
// took 142 and 177 us (one or two rows under way in an SM); rows prefetched into a ring
// 93 and 139; 32 values a thread and packed fp32 arithmetic 59 and 79; groups of one CTA
// that share the columns' coefficients 47 and 77; the hardware's exponential and quotient
// in tanh 69; no registers spilled, as RMS norms are compiled apart, 67.
#include <algorithm>

#include "ffn_nvfp4.h"
#include "int8.cuh"
#include "int8.h"
#include "launch.cuh"
#include "moe.h"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using namespace sm100;

__device__ int g_norm_device_error = 0;

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

__device__ __host__ __forceinline__ bool finite(float v) { return v - v == 0.0f; }

__device__ __forceinline__ float load_one(const void* p, bool bf16, int64_t at) {
  return bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
}

// 8 consecutive values as fp32.
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&o)[8]) {
  const uint4 t = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(w[i] << 16);
    o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// The same in two steps, so that a load can stand far before its use: the words as
// they are, and their values.  WIDE: they may be fp32, else they are bf16.
template <bool WIDE>
struct Raw {
  uint32_t w[WIDE ? 8 : 4];
  __device__ __forceinline__ void load(const void* p, bool bf16, int64_t at) {
    if (!WIDE || bf16) {
      const uint4 t = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
      w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 t = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at)[i];
        w[(4 * i) % (WIDE ? 8 : 4)] = t.x, w[(4 * i + 1) % (WIDE ? 8 : 4)] = t.y;
        w[(4 * i + 2) % (WIDE ? 8 : 4)] = t.z, w[(4 * i + 3) % (WIDE ? 8 : 4)] = t.w;
      }
    }
  }
  __device__ __forceinline__ void get(bool bf16, float (&o)[8]) const {
    if (WIDE && !bf16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(w[i % (WIDE ? 8 : 4)]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(i % 2 == 0 ? w[i / 2] << 16 : w[i / 2] & 0xffff0000u);
    }
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return f32_to_bf16_bits(lo) | ((uint32_t)f32_to_bf16_bits(hi) << 16);
}

__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

__device__ __forceinline__ float from_bits(uint32_t w, float) { return __uint_as_float(w); }
__device__ __forceinline__ uint32_t from_bits(uint32_t w, uint32_t) { return w; }
__device__ __forceinline__ uint32_t to_bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t to_bits(uint32_t v) { return v; }

// Sums and maxima over the threads that hold a row: a warp, or the CTA, whose
// warps leave their parts in one of two sets of 32 words in turn, so that one
// barrier is enough.  Words behind the last warp's are zeros.
template <bool WARP>
struct Row {
  uint32_t* parts;  // (one word more, of the row's first value)
  int turn = 0;
  // The first thread's v.
  __device__ __forceinline__ float first(float v) {
    if (WARP) return __shfl_sync(0xffffffffu, v, 0);
    if (threadIdx.x == 0) parts[64] = __float_as_uint(v);
    __syncthreads();
    return __uint_as_float(parts[64]);
  }
  template <typename T, typename F>
  __device__ __forceinline__ T over(T v, F f) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (WARP) return v;
    uint32_t* p = parts + 32 * turn;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = to_bits(v);
    __syncthreads();
    v = T(0);
    for (int w = 0; w < (int)(blockDim.x >> 5); w += 4) {
      const uint4 t = *reinterpret_cast<const uint4*>(p + w);
      v = f(v, f(f(from_bits(t.x, v), from_bits(t.y, v)), f(from_bits(t.z, v), from_bits(t.w, v))));
    }
    return v;
  }
  __device__ __forceinline__ float sum(float v) {
    return over(v, [](float a, float b) { return a + b; });
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    return over(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
  }
};

// A norm of a row's N sets of 8 values, set i of this thread at column at(i), is
// v * factor + shift before its weight and bias.
struct NormFactors {
  float factor, shift;
};

// A layer norm is taken of (v - c) / 2, c the row's first value.  Of values that hardly differ, a mean of v would be off
// by more than they differ (and of equal ones the norm would be that of the mean's rounding), or there is no number
// near enough; their v - c is exact, and other rows' off by 2^-24 of a difference that is in the row.  Halves, as v - c
// may pass fp32's range.
__device__ __forceinline__ float layer_eps(float eps) { return fmaxf(0.25f * eps, 1.4012985e-45f); }

// Squares of values beyond 2^64 pass fp32's range: such a row is scaled by 2^-75 and summed once more (eps by its
// square, of which nothing is left but that a row without variance does not divide by zero).
struct Resum {
  float eps, by = 1.0f;
  bool scaled = false;
  __device__ __forceinline__ bool wanted(float squares) {
    if (squares < __uint_as_float(0x7f800000u) || scaled) return false;
    scaled = true;
    by = 2.6469780e-23f;                        // 2^-75
    eps = fmaxf(eps * by * by, 1.1754944e-38f);  // 2^-126
    return true;
  }
};

template <bool WARP, int N, typename At>
__device__ __forceinline__ float row_squares(Row<WARP>& row, bool layer, int hidden, const float (&v)[N][8], At at, float* mean) {
  *mean = 0.0f;
  float s = 0.0f;
  if (layer) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < hidden)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[i][j];
    *mean = row.sum(s) * (1.0f / (float)hidden);
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < hidden)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = v[i][j] - *mean;
          s = fmaf(d, d, s);
        }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < hidden)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(v[i][j], v[i][j], s);
  }
  return row.sum(s);
}

template <bool LAYER, bool WARP, int N, typename At>
__device__ __forceinline__ NormFactors norm_factors(Row<WARP>& row, const NormArgs& a, int hidden, float (&v)[N][8], At at) {
  const float share = 1.0f / (float)hidden;
  float mean, squares;
  if (LAYER && a.layer) {
    const float c = -0.5f * row.first(v[0][0]);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = fmaf(0.5f, v[i][j], c);
  }
  Resum re{a.layer ? layer_eps(a.eps) : a.eps};
  while (re.wanted(squares = row_squares<WARP, N>(row, LAYER && a.layer, hidden, v, at, &mean)))
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= re.by;
  const float factor = rsqrtf(fmaf(squares, share, re.eps));
  return NormFactors{factor, -mean * factor};
}

// A norm's weights (and biases) at this thread's columns, loaded before the sums that they follow.
template <int N>
struct Weights {
  Raw<true> weight[N], bias[N];
  template <typename At>
  __device__ __forceinline__ void load(const NormArgs& a, int hidden, At at) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < hidden) {
        if (a.weight) weight[i].load(a.weight, a.bf16, at(i));
        if (a.bias) bias[i].load(a.bias, a.bf16, at(i));
      }
  }
  __device__ __forceinline__ void apply(const NormArgs& a, const NormFactors& f, int i, float (&v)[8]) const {
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = fmaf(v[j], f.factor, f.shift);
    if (a.weight) {
      weight[i].get(a.bf16, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= a.offset + t[j];
    }
    if (a.bias) {
      bias[i].get(a.bf16, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += t[j];
    }
  }
};

// tanh by its power series up to 1/2 (the first term left out is below 2^-26 of it) and by
// 1 - 2 / (exp(2 |g|) + 1) from there, where little cancels.
__device__ __forceinline__ float tanh_fast(float g) {
  const float a = fabsf(g), x = g * g;
  float s = fmaf(x, -929569.0f / 638512875.0f, 21844.0f / 6081075.0f);
  s = fmaf(x, s, -1382.0f / 155925.0f);
  s = fmaf(x, s, 62.0f / 2835.0f);
  s = fmaf(x, s, -17.0f / 315.0f);
  s = fmaf(x, s, 2.0f / 15.0f);
  s = fmaf(x, s, -1.0f / 3.0f);
  const float small = fmaf(g * x, s, g);
  const float large = copysignf(fmaf(-2.0f, rcp_approx(exp_approx(2.0f * a) + 1.0f), 1.0f), g);
  return a < 0.5f ? small : large;
}

__device__ __forceinline__ float gate_value(float g, int activation) {
  if (activation == FFN_GATE_SIGMOID) return rcp_approx(1.0f + expf(-g));
  if (activation == FFN_GATE_TANH) return tanh_fast(g);
  return g;
}

// The new residual of row r from v, the values of y, stored and left in v: each N sets of
// 8 values at columns at(i), the residual's and (with gate_cols) the gates' by load_res and load_gate.
template <bool R, bool LAYER, bool WARP, int N, typename LoadRes, typename LoadGate, typename At>
__device__ __forceinline__ void residual_row(Row<WARP>& row, const BlockArgs& a, int64_t r, float (&v)[N][8], LoadRes load_res,
                                             LoadGate load_gate, At at) {
  if (!a.y) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < a.hidden) load_res(i, v[i]);
    return;
  }
  NormFactors f = {};
  Weights<N> w;
  if (a.post.on) {
    w.load(a.post, a.hidden, at);
    f = norm_factors<LAYER, WARP, N>(row, a.post, a.hidden, v, at);
  }
  float scale = a.branch_scale;  // with the row's gate
  if (a.gate && !a.gate_cols) scale *= gate_value(load_one(a.gate, a.gate_bf16, r * a.gate_row_stride), a.gate_activation);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at(i) < a.hidden) {
      float t[8];
      if (a.post.on) w.apply(a.post, f, i, v[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= scale;
      if (a.gate && a.gate_cols) {
        load_gate(i, t);
        if (a.gate_activation != FFN_GATE_NONE)
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] = gate_value(t[j], a.gate_activation);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= t[j];
      }
      load_res(i, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = fmaf(a.residual_scale, t[j], v[i][j]);
        v[i][j] = R ? bf16_round(x) : x;
      }
      if (a.residual_out) {
        if (R) {
          store_bf16(static_cast<uint16_t*>(a.residual_out) + r * a.residual_out_stride + at(i), v[i]);
        } else {
          float* o = static_cast<float*>(a.residual_out) + r * a.residual_out_stride + at(i);
#pragma unroll
          for (int q = 0; q < 2; ++q)
            reinterpret_cast<float4*>(o)[q] = make_float4(v[i][4 * q], v[i][4 * q + 1], v[i][4 * q + 2], v[i][4 * q + 3]);
        }
      }
    }
}

// The norm of the new residual, and its stores.
template <bool LAYER, bool WARP, int N, typename At>
__device__ __forceinline__ void output_row(Row<WARP>& row, const BlockArgs& a, int64_t r, int mine, float (&res)[N][8], At at) {
  if (!a.pre.on) return;
  Weights<N> w;
  w.load(a.pre, a.hidden, at);
  const NormFactors f = norm_factors<LAYER, WARP, N>(row, a.pre, a.hidden, res, at);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at(i) < a.hidden) w.apply(a.pre, f, i, res[i]);
  if (!a.out_scales) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < a.hidden) store_bf16(static_cast<uint16_t*>(a.out) + r * a.out_stride + at(i), res[i]);
    return;
  }
  // The codes are those of the row as it would be stored in bf16.
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at(i) < a.hidden)
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, (uint32_t)(f32_to_bf16_bits(res[i][j]) & 0x7fffu));
  const Int8Row q(row.max(top));
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at(i) < a.hidden) {
      int8_t* o = static_cast<int8_t*>(a.out) + r * a.out_stride + at(i);
      *reinterpret_cast<uint2*>(o) =
          int8_encode8(q, make_uint4(pack_bf16(res[i][0], res[i][1]), pack_bf16(res[i][2], res[i][3]),
                                     pack_bf16(res[i][4], res[i][5]), pack_bf16(res[i][6], res[i][7])));
    }
  if (mine == 0) a.out_scales[r] = q.scale;
}

// R: the residual is bf16; LAYER: a norm may be a layer norm; WARP: a warp for each
// row, else the CTA; N: accesses of 8 values a thread.
template <bool R, bool LAYER, bool WARP, int N, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) block_norm_kernel(const BlockArgs a) {
  __shared__ __align__(16) uint32_t parts[65];
  Row<WARP> row{parts};
  const int threads = WARP ? 32 : blockDim.x, mine = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int per_cta = WARP ? blockDim.x >> 5 : 1;
  auto at = [&](int i) { return 8 * (mine + i * threads); };
  if (!WARP) {
    if (threadIdx.x < 64) parts[threadIdx.x] = 0;
    if (blockDim.x < 64 && threadIdx.x < 32) parts[threadIdx.x + 32] = 0;
    __syncthreads();
  }
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t r = blockIdx.x * (int64_t)per_cta + (WARP ? threadIdx.x >> 5 : 0); r < a.m;
       r += (int64_t)gridDim.x * per_cta) {
    // all loads first: a row's latency counts here
    float v[N][8];
    Raw<!R> res[N];
    Raw<true> g[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < a.hidden) {
        if (a.y) load_bf16(a.y + r * a.y_stride + at(i), v[i]);
        res[i].load(a.residual, R, r * a.residual_stride + at(i));
        if (a.gate && a.gate_cols) g[i].load(a.gate, a.gate_bf16, r * a.gate_row_stride + at(i));
      }
    residual_row<R, LAYER, WARP, N>(
        row, a, r, v, [&](int i, float(&t)[8]) { res[i].get(R, t); }, [&](int i, float(&t)[8]) { g[i].get(a.gate_bf16, t); }, at);
    output_row<LAYER, WARP, N>(row, a, r, mine, v, at);
  }
}

// ----------------------------------------- rows that are not whole 16 bytes

// A CTA a row, values one by one; the row is in shared memory, where a thread only touches its own.
// Loops of few instructions: with a row unrolled in registers (8 values a thread, each with its types
// and gates) the code was long and 203 rows of 1037, layer norm, took 5.9 to 9.6 us; so they take 4.8.
template <bool R>
__device__ __forceinline__ void any_rows(const BlockArgs& a, float* v, uint32_t* parts) {
  Row<false> row{parts};
  constexpr int kAtOnce = 4;  // values of a thread under way
  const int mine = threadIdx.x, threads = blockDim.x, h = a.hidden;
  const float share = 1.0f / (float)h;
  // A norm of the row, (v - c) * factor + shift before its weight and bias.  v stays as it is, so that differences beyond
  // fp32's range are found by their sums, and the row is scaled.
  struct Normed {
    float c, factor, shift;
    __device__ __forceinline__ float operator()(float v) const { return fmaf(v - c, factor, shift); }
  };
  auto factors = [&](const NormArgs& n) {
    float c = n.layer ? row.first(mine == 0 ? v[0] : 0.0f) : 0.0f;
    for (Resum re{n.eps};;) {
      float mean = 0.0f, s = 0.0f;
      if (n.layer) {
        for (int i = mine; i < h; i += threads) s += v[i] - c;
        mean = row.sum(s) * share;
        s = 0.0f;
      }
      for (int i = mine; i < h; i += threads) {
        const float d = (v[i] - c) - mean;
        s = fmaf(d, d, s);
      }
      const float squares = row.sum(s);
      if (!re.wanted(squares)) {
        const float factor = rsqrtf(fmaf(squares, share, re.eps));
        return Normed{c, factor, -mean * factor};
      }
      for (int i = mine; i < h; i += threads) v[i] *= re.by;
      c *= re.by;
    }
  };
  for (int64_t r = blockIdx.x; r < a.m; r += gridDim.x) {
    const uint16_t* y = a.y + r * a.y_stride;
    for (int i0 = mine; i0 < h; i0 += kAtOnce * threads) {
      float t[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * threads;
        if (i < h) t[j] = a.y ? bf16_bits_to_float(y[i]) : load_one(a.residual, R, r * a.residual_stride + i);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (i0 + j * threads < h) v[i0 + j * threads] = t[j];
    }
    if (a.y) {
      Normed f{0.0f, 1.0f, 0.0f};
      if (a.post.on) f = factors(a.post);
      for (int i0 = mine; i0 < h; i0 += kAtOnce * threads) {
        float x[kAtOnce], g[kAtOnce], w[kAtOnce], b[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int i = i0 + j * threads;
          g[j] = w[j] = 1.0f, b[j] = 0.0f;
          if (i >= h) continue;
          x[j] = load_one(a.residual, R, r * a.residual_stride + i);
          if (a.gate) g[j] = load_one(a.gate, a.gate_bf16, r * a.gate_row_stride + (a.gate_cols ? i : 0));
          if (a.post.weight) w[j] = a.post.offset + load_one(a.post.weight, a.post.bf16, i);
          if (a.post.bias) b[j] = load_one(a.post.bias, a.post.bf16, i);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int i = i0 + j * threads;
          if (i >= h) break;
          const float z = fmaf(f(v[i]), w[j], b[j]);
          float s = fmaf(a.residual_scale, x[j], a.branch_scale * z * gate_value(g[j], a.gate ? a.gate_activation : 0));
          if (R) s = bf16_round(s);
          v[i] = s;
          if (!a.residual_out) continue;
          if (R)
            static_cast<uint16_t*>(a.residual_out)[r * a.residual_out_stride + i] = f32_to_bf16_bits(s);
          else
            static_cast<float*>(a.residual_out)[r * a.residual_out_stride + i] = s;
        }
      }
    }
    if (!a.pre.on) continue;
    const Normed f = factors(a.pre);
    uint32_t top = 0;
    for (int i0 = mine; i0 < h; i0 += kAtOnce * threads) {
      float w[kAtOnce], b[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * threads;
        w[j] = 1.0f, b[j] = 0.0f;
        if (i < h && a.pre.weight) w[j] = a.pre.offset + load_one(a.pre.weight, a.pre.bf16, i);
        if (i < h && a.pre.bias) b[j] = load_one(a.pre.bias, a.pre.bf16, i);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * threads;
        if (i >= h) break;
        const uint16_t x = f32_to_bf16_bits(fmaf(f(v[i]), w[j], b[j]));
        if (a.out_scales)
          top = max(top, x & 0x7fffu), v[i] = bf16_bits_to_float(x);
        else
          static_cast<uint16_t*>(a.out)[r * a.out_stride + i] = x;
      }
    }
    if (!a.out_scales) continue;
    // The codes are those of the row as it would be stored in bf16.
    const Int8Row q(row.max(top));
    for (int i = mine; i < h; i += threads) static_cast<int8_t*>(a.out)[r * a.out_stride + i] = (int8_t)q.code(v[i]);
    if (mine == 0) a.out_scales[r] = q.scale;
  }
}

template <bool R, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) block_norm_any_kernel(const BlockArgs a) {
  extern __shared__ float v[];
  __shared__ __align__(16) uint32_t parts[65];
  for (int i = threadIdx.x; i < 64; i += blockDim.x) parts[i] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  any_rows<R>(a, v, parts);
}

// ------------------------------------------------- many rows of whole 16 bytes

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 of_pair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)), "l"(pair_of(c)));
  return of_pair(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)));
  return of_pair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)));
  return of_pair(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// U (8 or 4) consecutive values in pairs.
template <int U>
__device__ __forceinline__ void load_u(const void* p, bool bf16, int64_t at, float2 (&o)[U / 2]) {
  if (bf16) {
    uint32_t w[U / 2];
    if (U == 8) {
      const uint4 t = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
      w[0] = t.x, w[1] = t.y, w[2 % (U / 2)] = t.z, w[3 % (U / 2)] = t.w;
    } else {
      const uint2 t = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
      w[0] = t.x, w[1] = t.y;
    }
#pragma unroll
    for (int j = 0; j < U / 2; ++j) o[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
  } else {
#pragma unroll
    for (int j = 0; j < U / 4; ++j) {
      const float4 t = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at)[j];
      o[2 * j] = make_float2(t.x, t.y), o[2 * j + 1] = make_float2(t.z, t.w);
    }
  }
}
template <int U>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[U / 2]) {
  if (U == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2 % (U / 2)], w[3 % (U / 2)]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
// tanh_fast of two values.
__device__ __forceinline__ float2 tanh2(float2 g) {
  const float2 x = mul2(g, g);
  float2 s = fma2(x, both(-929569.0f / 638512875.0f), both(21844.0f / 6081075.0f));
  s = fma2(x, s, both(-1382.0f / 155925.0f));
  s = fma2(x, s, both(62.0f / 2835.0f));
  s = fma2(x, s, both(-17.0f / 315.0f));
  s = fma2(x, s, both(2.0f / 15.0f));
  s = fma2(x, s, both(-1.0f / 3.0f));
  const float2 small = fma2(mul2(g, x), s, g);
  const float2 e = add2(make_float2(exp_approx(2.0f * fabsf(g.x)), exp_approx(2.0f * fabsf(g.y))), both(1.0f));
  const float2 large = fma2(both(-2.0f), make_float2(rcp_approx(e.x), rcp_approx(e.y)), both(1.0f));
  return make_float2(fabsf(g.x) < 0.5f ? small.x : copysignf(large.x, g.x), fabsf(g.y) < 0.5f ? small.y : copysignf(large.y, g.y));
}
template <int U>
__device__ __forceinline__ void gate_values(float2 (&g)[U / 2], int activation) {
  if (activation == FFN_GATE_TANH) {
#pragma unroll
    for (int j = 0; j < U / 2; ++j) g[j] = tanh2(g[j]);
  } else if (activation == FFN_GATE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < U / 2; ++j) g[j] = make_float2(gate_value(g[j].x, FFN_GATE_SIGMOID), gate_value(g[j].y, FFN_GATE_SIGMOID));
  }
}
__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Sums and maxima of a group's row stand in sets of words of their own, in the order in which a row meets them: a set is
// written again a row later only, behind other barriers.
constexpr int kMeanSet = 0, kSquaresSet = 1, kMaxSet = 4, kSets = 5;  // (of the post norm; of the pre norm 2 more)
constexpr int kSetWords = 72;  // 24 warps, each group's from a multiple of 4 on

// The threads of a CTA that hold a row: some of its warps, with a named barrier.
struct Group {
  uint32_t* parts;  // the group's words of the first set, zeros behind the last warp's
  int id, threads, warp;
  __device__ __forceinline__ void sync() {
    __syncwarp();  // (the barrier wants whole warps)
    named_bar_sync(id, threads);
  }
  __device__ __forceinline__ float sum(float v, int set) {
    v = warp_sum(v);
    uint32_t* p = parts + kSetWords * set;
    if ((threadIdx.x & 31) == 0) p[warp] = __float_as_uint(v);
    sync();
    float s[4] = {};
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (4 * w < threads / 32) {
        const float4 t = *reinterpret_cast<const float4*>(p + 4 * w);
        s[w] = (t.x + t.y) + (t.z + t.w);
      }
    return (s[0] + s[1]) + (s[2] + s[3]);
  }
  __device__ __forceinline__ uint32_t max(uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    uint32_t* p = parts + kSetWords * kMaxSet;
    if ((threadIdx.x & 31) == 0) p[warp] = v;
    sync();
    v = 0;
    for (int w = 0; w < threads / 32; ++w) v = ::max(v, p[w]);
    return v;
  }
  __device__ __forceinline__ bool all(bool ok) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
  }
};

// The factors of a norm for N sets of U values, the row's first value c; columns behind the row are zeros.
template <bool LAYER, int WHICH, int U, int N>
__device__ __forceinline__ NormFactors norm_factors2(Group& row, const NormArgs& a, float share, float2 (&v)[N][U / 2],
                                                     const bool (&in)[N], float c) {
  float mean = 0.0f, squares;
  if (LAYER && a.layer) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (in[i])
#pragma unroll
        for (int j = 0; j < U / 2; ++j) v[i][j] = fma2(both(0.5f), v[i][j], both(-0.5f * c));
  }
  for (Resum re{a.layer ? layer_eps(a.eps) : a.eps};;) {
    float2 s[2] = {both(0.0f), both(0.0f)};
    if (LAYER && a.layer) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < U / 2; ++j) s[j & 1] = add2(s[j & 1], v[i][j]);
      s[0] = add2(s[0], s[1]);
      mean = row.sum(s[0].x + s[0].y, kMeanSet + 2 * WHICH) * share;
      s[0] = s[1] = both(0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (in[i])
#pragma unroll
          for (int j = 0; j < U / 2; ++j) {
            const float2 d = add2(v[i][j], both(-mean));
            s[j & 1] = fma2(d, d, s[j & 1]);
          }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < U / 2; ++j) s[j & 1] = fma2(v[i][j], v[i][j], s[j & 1]);
    }
    s[0] = add2(s[0], s[1]);
    squares = row.sum(s[0].x + s[0].y, kSquaresSet + 2 * WHICH);
    if (!re.wanted(squares)) {
      const float factor = rsqrtf(fmaf(squares, share, re.eps));
      return NormFactors{factor, -mean * factor};
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (in[i])
#pragma unroll
        for (int j = 0; j < U / 2; ++j) v[i][j] = mul2(v[i][j], both(re.by));
    row.sync();  // (the sets once more)
  }
}

// Coefficients of the columns in shared memory, fp32: 16 bytes at a time, those of a set of 8 in two planes.
template <int U>
__device__ __forceinline__ void load_plane(const float4* c, int vecs, int vec, float2 (&o)[U / 2]) {
#pragma unroll
  for (int j = 0; j < U / 4; ++j) {
    const float4 t = c[j * vecs + vec];
    o[2 * j] = make_float2(t.x, t.y), o[2 * j + 1] = make_float2(t.z, t.w);
  }
}
template <int U>
__device__ __forceinline__ void store_plane(float4* c, int vecs, int vec, const float2 (&v)[U / 2]) {
#pragma unroll
  for (int j = 0; j < U / 4; ++j) c[j * vecs + vec] = make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
}

struct StreamPlan {
  int threads, groups, slots;  // threads of a group; groups of a CTA, one CTA an SM; slots of a group
  int slot_bytes;
  float share;                 // 1 / hidden
  bool shift;                  // a norm has a mean or a bias (SHIFT of the kernel)
};

constexpr int kStreamValues = 32;    // of a thread
constexpr int kStreamThreads = 768;  // of a CTA, at most

// any_rows in a kernel whose registers it should not take.
template <bool R>
__device__ __noinline__ void rows_apart(const BlockArgs& a, float* v, uint32_t* parts) {
  any_rows<R>(a, v, parts);
}

// One persistent CTA an SM, groups of whose warps work on a row each: as many rows
// are under way as their inputs find room for in shared memory (bulk copies, the next
// row's as soon as all have read the last one's).  What belongs to the columns for all
// rows is made once, in shared memory: the norms' weights, with a gate of the channels
// and the branch's scale in the first.  A thread has N sets of U values, 32 in all: what a row
// costs apart from its values (two sums over the group) is shared by as many.  U: 8, or 4
// where the residual is fp32, so that neighbouring lanes access neighbouring 16 bytes.  SHIFT: a norm has a mean or a
// bias; what others do not need would cost them registers (4096 x 5120, bf16, gates by row: 39.6 us with six values
// spilled, 35.7 without).
template <bool R, bool SHIFT>
__global__ void __launch_bounds__(kStreamThreads, 1) block_norm_stream_kernel(const __grid_constant__ BlockArgs a, const __grid_constant__ StreamPlan p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) uint32_t parts[kSets * kSetWords];
  __shared__ uint64_t full[32];
  __shared__ int abort_word;
  __shared__ float first_value[15];  // of each group's new residual
  volatile int* abort_flag = &abort_word;
  const int g = threadIdx.x / p.threads, mine = threadIdx.x - g * p.threads;
  Group row{parts + (p.threads / 32 + 3) / 4 * 4 * g, 1 + g, p.threads, mine >> 5};
  constexpr int U = R ? 8 : 4, N = kStreamValues / U;
  const int vecs = a.hidden / U;
  auto vec = [&](int i) { return mine + i * p.threads; };
  bool in[N];
#pragma unroll
  for (int i = 0; i < N; ++i) in[i] = vec(i) < vecs;
  float4* w1 = reinterpret_cast<float4*>(smem);
  float4* w2 = w1 + a.hidden / 4;
  float4* b1 = w2 + a.hidden / 4;  // (with shift)
  float4* b2 = b1 + a.hidden / 4;
  uint8_t* ring = reinterpret_cast<uint8_t*>(SHIFT ? b2 + a.hidden / 4 : b1) + g * p.slots * p.slot_bytes;
  uint64_t* bar = full + g * p.slots;
  // A slot: y, the residual, the gates if each row has its own.
  const bool own_gates = a.gate && a.gate_cols && a.gate_row_stride != 0, channel_gates = a.gate && a.gate_cols && !own_gates;
  const int y_bytes = a.y ? 2 * a.hidden : 0, r_bytes = (R ? 2 : 4) * a.hidden;
  const int g_bytes = own_gates ? (a.gate_bf16 ? 2 : 4) * a.hidden : 0;
  for (int i = threadIdx.x; i < kSets * kSetWords; i += blockDim.x) parts[i] = 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.groups * p.slots; ++s) mbar_init(&full[s], 1);
    abort_word = 0;
    fence_mbar_init();
  }
  __syncthreads();
  auto copy = [&](int64_t r, int s) {
    uint8_t* to = ring + s * p.slot_bytes;
    mbar_arrive_expect_tx(&bar[s], y_bytes + r_bytes + g_bytes);
    if (y_bytes) bulk_load(to, a.y + r * a.y_stride, y_bytes, &bar[s]);
    bulk_load(to + y_bytes, static_cast<const uint8_t*>(a.residual) + r * a.residual_stride * (R ? 2 : 4), r_bytes, &bar[s]);
    if (g_bytes)
      bulk_load(to + y_bytes + r_bytes, static_cast<const uint8_t*>(a.gate) + r * a.gate_row_stride * (a.gate_bf16 ? 2 : 4),
                g_bytes, &bar[s]);
  };
  // A copy of a row that is given up lands before the CTA leaves.
  auto landed = [&](int s, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait(&bar[s], parity) && clock64() - t0 < kWaitLimitCycles) {
    }
  };
  // (rows in 32 bits: of 80 registers none is left, and what is spilled comes back from L2)
  const int m = (int)a.m, first = blockIdx.x + g * gridDim.x, step = gridDim.x * p.groups;
  griddep_wait();
  griddep_launch_dependents();
  if (mine == 0)
    for (int s = 0; s < p.slots && first + s * step < m; ++s) copy(first + s * step, s);
  bool ok = true;  // the first coefficients are finite
  for (int i = threadIdx.x; i < vecs; i += blockDim.x) {
    float2 w[U / 2], t[U / 2];
    for (int j = 0; j < U / 2; ++j) w[j] = both(a.branch_scale);
    if (channel_gates) {
      load_u<U>(a.gate, a.gate_bf16, U * i, t);
      gate_values<U>(t, a.gate_activation);
      for (int j = 0; j < U / 2; ++j)
        w[j] = mul2(w[j], t[j]);
    }
    if (SHIFT) {
      for (int j = 0; j < U / 2; ++j) t[j] = both(0.0f);
      if (a.post.bias) load_u<U>(a.post.bias, a.post.bf16, U * i, t);
      for (int j = 0; j < U / 2; ++j) t[j] = mul2(t[j], w[j]), ok = ok && finite(t[j].x) && finite(t[j].y);
      store_plane<U>(b1, vecs, i, t);
    }
    if (a.post.weight) {
      load_u<U>(a.post.weight, a.post.bf16, U * i, t);
      for (int j = 0; j < U / 2; ++j) w[j] = mul2(add2(t[j], both(a.post.offset)), w[j]);
    }
    for (int j = 0; j < U / 2; ++j) ok = ok && finite(w[j].x) && finite(w[j].y);
    store_plane<U>(w1, vecs, i, w);
    for (int j = 0; j < U / 2; ++j) w[j] = both(1.0f), t[j] = both(0.0f);
    if (SHIFT) {
      if (a.pre.bias) load_u<U>(a.pre.bias, a.pre.bf16, U * i, t);
      store_plane<U>(b2, vecs, i, t);
    }
    if (a.pre.weight) {
      load_u<U>(a.pre.weight, a.pre.bf16, U * i, t);
      for (int j = 0; j < U / 2; ++j) w[j] = add2(t[j], both(a.pre.offset));
    }
    store_plane<U>(w2, vecs, i, w);
  }
  if (!__syncthreads_and(ok) && channel_gates) {
    // A gate of channels is part of coefficients that are not finite (an infinity, of which 0 * inf would come where a
    // value is 0): these rows are computed in the order of their definition, once the copies have landed.
    if (mine == 0)
      for (int s = 0; s < p.slots && first + s * step < m; ++s)
        if (!mbar_wait(&bar[s], 0, abort_flag, &g_norm_device_error, 1)) landed(s, 0);
    if (__syncthreads_and(*abort_flag == 0)) rows_apart<R>(a, reinterpret_cast<float*>(smem), parts);
    return;
  }
  const float share = p.share;
  int s = 0;
  uint32_t parity = 0;
  for (int r = first; r < m; r += step) {
    float g1 = 1.0f;  // the row's gate
    if (a.gate && !a.gate_cols) {
      g1 = gate_value(load_one(a.gate, a.gate_bf16, (int64_t)r * a.gate_row_stride), a.gate_activation);
    }
    // The group agrees that the row's copy has landed before it uses any of it: a row that is given up is not stored.
    if (!row.all(mbar_wait(&bar[s], parity, abort_flag, &g_norm_device_error, 1))) {
      if (mine == 0)
        for (int q = r; q < m && q < r + p.slots * step; q += step) {
          landed(s, parity);
          if (++s == p.slots) s = 0, parity ^= 1;
        }
      return;
    }
    const uint8_t* from = ring + s * p.slot_bytes;
    float2 v[N][U / 2];
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int j = 0; j < U / 2; ++j) v[i][j] = both(0.0f);
      if (in[i]) load_u<U>(a.y ? from : from + y_bytes, a.y ? true : R, U * vec(i), v[i]);
    }
    if (a.y) {
      NormFactors f{1.0f, 0.0f};
      if (a.post.on) f = norm_factors2<SHIFT, 0, U, N>(row, a.post, share, v, in, bf16_bits_to_float(*reinterpret_cast<const uint16_t*>(from)));
      if (!SHIFT) {  // (a row's gate, then, is part of its factor, or takes its place where that would be beyond fp32)
        if (finite(g1) && !finite(f.factor * g1)) {
#pragma unroll
          for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < U / 2; ++j) v[i][j] = mul2(v[i][j], both(f.factor));
          f.factor = 1.0f;
        }
        f.factor *= g1;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (!in[i]) continue;
        float2 t[U / 2];
        if (SHIFT) {
#pragma unroll
          for (int j = 0; j < U / 2; ++j) v[i][j] = fma2(v[i][j], both(f.factor), both(f.shift));
        } else {
#pragma unroll
          for (int j = 0; j < U / 2; ++j) v[i][j] = mul2(v[i][j], both(f.factor));
        }
        load_plane<U>(w1, vecs, vec(i), t);
#pragma unroll
        for (int j = 0; j < U / 2; ++j) v[i][j] = mul2(v[i][j], t[j]);
        if (SHIFT) {
          load_plane<U>(b1, vecs, vec(i), t);
#pragma unroll
          for (int j = 0; j < U / 2; ++j) v[i][j] = add2(v[i][j], t[j]);
        }
        if (SHIFT && a.gate && !a.gate_cols) {
#pragma unroll
          for (int j = 0; j < U / 2; ++j) v[i][j] = mul2(v[i][j], both(g1));
        }
        if (own_gates) {
          load_u<U>(from + y_bytes + r_bytes, a.gate_bf16, U * vec(i), t);
          gate_values<U>(t, a.gate_activation);
#pragma unroll
          for (int j = 0; j < U / 2; ++j) v[i][j] = mul2(v[i][j], t[j]);
        }
        load_u<U>(from + y_bytes, R, U * vec(i), t);
#pragma unroll
        for (int j = 0; j < U / 2; ++j) v[i][j] = fma2(both(a.residual_scale), t[j], v[i][j]);
        if (R) {
          uint32_t q[U / 2];
#pragma unroll
          for (int j = 0; j < U / 2; ++j) q[j] = pack2(v[i][j]), v[i][j] = unpack2(q[j]);
          if (a.residual_out)
            store_words<U>(static_cast<uint16_t*>(a.residual_out) + (int64_t)r * a.residual_out_stride + U * vec(i), q);
        } else if (a.residual_out) {
          float* o = static_cast<float*>(a.residual_out) + (int64_t)r * a.residual_out_stride + U * vec(i);
#pragma unroll
          for (int j = 0; j < U / 4; ++j)
            reinterpret_cast<float4*>(o)[j] = make_float4(v[i][2 * j].x, v[i][2 * j].y, v[i][2 * j + 1].x, v[i][2 * j + 1].y);
        }
      }
    }
    if (SHIFT && mine == 0) first_value[g] = v[0][0].x;
    row.sync();  // all have read the slot
    const int next = r + p.slots * step;
    if (mine == 0 && next < m) copy(next, s);
    if (++s == p.slots) s = 0, parity ^= 1;
    if (!a.pre.on) continue;
    const NormFactors f = norm_factors2<SHIFT, 1, U, N>(row, a.pre, share, v, in, first_value[g]);
    uint32_t q[N][U / 2];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!in[i]) continue;
      float2 t[U / 2];
      load_plane<U>(w2, vecs, vec(i), t);
      if (SHIFT) {
        float2 u[U / 2];
        load_plane<U>(b2, vecs, vec(i), u);
#pragma unroll
        for (int j = 0; j < U / 2; ++j) v[i][j] = fma2(fma2(v[i][j], both(f.factor), both(f.shift)), t[j], u[j]);
      } else {
#pragma unroll
        for (int j = 0; j < U / 2; ++j) v[i][j] = mul2(mul2(v[i][j], both(f.factor)), t[j]);
      }
#pragma unroll
      for (int j = 0; j < U / 2; ++j) q[i][j] = pack2(v[i][j]);
      if (!a.out_scales) store_words<U>(static_cast<uint16_t*>(a.out) + (int64_t)r * a.out_stride + U * vec(i), q[i]);
    }
    if (!a.out_scales) continue;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (in[i])
#pragma unroll
        for (int j = 0; j < U / 2; ++j) top = amax_bf16x2(top, q[i][j]);
    const Int8Row codes(row.max(amax_of_pair(top)));
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (in[i]) {
        int8_t* o = static_cast<int8_t*>(a.out) + (int64_t)r * a.out_stride + U * vec(i);
        const uint2 c = int8_encode8(codes, make_uint4(q[i][0], q[i][1], U == 8 ? q[i][2 % (U / 2)] : 0u, U == 8 ? q[i][3 % (U / 2)] : 0u));
        if (U == 8)
          *reinterpret_cast<uint2*>(o) = c;
        else
          *reinterpret_cast<uint32_t*>(o) = c.x;
      }
    if (mine == 0) a.out_scales[r] = codes.scale;
  }
}

template <bool R, bool WARP, int N, int THREADS>
cudaError_t launch_one(const BlockArgs& a, int threads, cudaStream_t s) {
  const int64_t per_cta = WARP ? threads / 32 : 1;
  const int64_t ctas = (a.m + per_cta - 1) / per_cta, most = (int64_t)device_sms() * (2048 / threads);
  ProfScope prof(s, "block_norm");
  auto kern = a.post.layer || a.pre.layer ? block_norm_kernel<R, true, WARP, N, THREADS> : block_norm_kernel<R, false, WARP, N, THREADS>;
  return launch_pdl(kern, dim3((unsigned)(ctas < most ? ctas : most)), dim3(threads),
                    0, s, a);
}

int round_up_32(int v) { return (v + 31) / 32 * 32; }

constexpr int kStreamBytes = 224 * 1024;  // of shared memory

// Set on every launch, as the attribute belongs to the current device's context, and to the most that any launch of the
// kernel takes: with its own size a call would refuse that of another thread, between the two steps of its launch.
template <typename Kernel>
cudaError_t allow_shared(Kernel kern, int bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

int stream_coefs(const BlockArgs& a, bool shift) { return (shift ? 4 : 2) * 4 * a.hidden; }

// As many groups as fit (15 named barriers, kStreamThreads), and a second slot for each where there is room;
// no groups where even two rows do not fit.
StreamPlan plan_stream(const BlockArgs& a, bool bf16) {
  StreamPlan p = {};
  const int own_gate = a.gate && a.gate_cols && a.gate_row_stride != 0 ? (a.gate_bf16 ? 2 : 4) : 0;
  p.shift = a.post.layer || a.post.bias || a.pre.layer || a.pre.bias;
  p.share = 1.0f / (float)a.hidden;
  p.threads = round_up_32((a.hidden + kStreamValues - 1) / kStreamValues);
  p.slot_bytes = a.hidden * ((a.y ? 2 : 0) + (bf16 ? 2 : 4) + own_gate);
  const int slots = (kStreamBytes - stream_coefs(a, p.shift)) / p.slot_bytes, most = kStreamThreads / p.threads < 15 ? kStreamThreads / p.threads : 15;
  if (slots < 2 || p.threads > 512) return p;
  p.groups = slots < most ? slots : most;
  p.slots = slots >= 2 * p.groups ? 2 : 1;
  return p;
}

// Threads and accesses for a row: as few accesses as keep a CTA to 512 threads.
template <bool R>
cudaError_t launch_rows(const BlockArgs& a, bool vec, cudaStream_t s) {
  const int h = a.hidden;
  if (!vec) {
    // 4 values a thread while all rows are under way at once; then 8, and registers for 3 CTAs of 512 threads on an SM
    // (2074 rows of 2797, layer norms before and after, 107 and 61 us; 476 rows of 497 7.0 and 11.4).
    const int four = std::min(1024, round_up_32((h + 3) / 4));
    const bool few = a.m <= (int64_t)device_sms() * (1024 / four) || h > 8192;
    auto kern = few ? block_norm_any_kernel<R, 1024, 1> : block_norm_any_kernel<R, 512, 3>;
    const int threads = few ? four : std::min(512, round_up_32((h + 7) / 8)), bytes = 4 * h;
    if (few) {
      const cudaError_t e = allow_shared(kern, 4 * FFN_NORM_MAX_HIDDEN);
      if (e != cudaSuccess) return e;
    }
    const int64_t most = 8 * (int64_t)device_sms();  // (the longest rows' CTAs wait for room)
    ProfScope prof(s, "block_norm");
    return launch_pdl(kern, dim3((unsigned)(a.m < most ? a.m : most)), dim3(threads), bytes, s, a);
  }
  // The streaming kernel, for more rows than the kernels by rows have under way at once (8 warps or 512 threads an SM):
  // their second wave costs as much as the first, the streaming kernel's start (the columns' coefficients) less.  Both
  // norms, by rows and streaming, in us, bf16 residual: 450 and 600 rows of 2048 4.8, 7.1 and 5.2, 5.4; 150, 200 and
  // 300 of 4096, 5120 and 4096 4.8, 8.2, 7.5 and 5.2, 5.4, 5.4; 140 and 149 of 8192 5.4, 8.8 and 5.9, 6.2; 1184 of 512 4.1 and
  // 4.8, 1190 of 384 6.2 and 4.7; 2400 of 4096 20.2 and 12.7.  Rows of four accesses a lane are slow by a warp each: 640 of
  // 1024 6.4 and 5.3 (fp32 6.6 and 6.5).  Of 256 (an access a lane) 600 rows take 3.2 and 4.4, 9600 10.2 and 11.9.
  const int64_t at_once = (int64_t)device_sms() * (h <= 1024 ? 8 : std::max(1, 512 / round_up_32((h + 15) / 16)));
  if (h > 256 && (a.m > at_once || (h > 512 && h <= 1024 && a.m * h >= 600000)) && a.m <= INT32_MAX / 2) {
    const StreamPlan p = plan_stream(a, R);
    if (p.groups > 0) {
      auto kern = p.shift ? block_norm_stream_kernel<R, true> : block_norm_stream_kernel<R, false>;
      const int bytes = stream_coefs(a, p.shift) + p.groups * p.slots * p.slot_bytes;
      const cudaError_t e = allow_shared(kern, kStreamBytes);
      if (e != cudaSuccess) return e;
      ProfScope prof(s, "block_norm");
      return launch_pdl(kern, dim3(device_sms()), dim3(p.threads * p.groups), bytes, s, a, p);
    }
  }
  if (h <= 256) return launch_one<R, true, 1, 256>(a, 256, s);
  if (h <= 512) return launch_one<R, true, 2, 256>(a, 256, s);
  if (h <= 1024) return launch_one<R, true, 4, 256>(a, 256, s);
  if (h <= 8192) return launch_one<R, false, 2, 512>(a, round_up_32((h + 15) / 16), s);
  if (h <= 16384) return launch_one<R, false, 4, 512>(a, round_up_32((h + 31) / 32), s);
  return launch_one<R, false, 4, 1024>(a, round_up_32((h + 31) / 32), s);
}

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1u)) == 0; }
bool valid_type(int t) { return t == FFN_VALUE_F32 || t == FFN_VALUE_BF16; }
unsigned size_of(int type) { return type == FFN_VALUE_BF16 ? 2 : 4; }
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
cudaError_t read_norm_device_error(int* flags, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_norm_device_error, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && clear) e = cudaMemcpyToSymbol(g_norm_device_error, &zero, sizeof(int));
  return e;
}

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
      !aligned(b->out, b->out_scales ? 1 : 2) || (b->gate && !aligned(b->gate, size_of(b->gate_type))))
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
