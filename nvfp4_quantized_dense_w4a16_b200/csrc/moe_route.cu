// Routing of rows to experts: scores of E experts per row -> the top_k experts
// and their weights (ffn_nvfp4_moe_route).
//
// With s = softmax(l) or sigmoid(l) of a row's logits, the choice goes by the
// keys c = s + bias (optionally only inside the best groups of experts) and
// the weights by s alone, renormalised over the chosen experts on request.
//
// One warp owns one row; lane l holds experts l, l + 32, ... in registers.
#include <math.h>

#include "common.cuh"
#include "ffn_nvfp4.h"
#include "launch.cuh"
#include "moe.h"
#include "profile.h"
#include "sm100.cuh"

namespace ffn {
namespace {

using sm100::griddep_launch_dependents;
using sm100::griddep_wait;

constexpr int kRouteWarps = 4;

struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;  // or null
  int32_t* ids;
  float* weights;
  int64_t m;
  int experts, top_k, groups, top_groups, scoring, group_score, renormalize;
  float scale;
};

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// log(sigmoid(l)), finite for every finite l.
__device__ __forceinline__ double log_sigmoid(double l) {
  return l < 0.0 ? l - log1p(exp(l)) : -log1p(exp(-l));
}

template <int EPL, bool BF16>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const RouteArgs a) {
  extern __shared__ double route_smem[];  // [warps][experts] keys, only with groups
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (row >= a.m) return;
  const int E = a.experts;
  const bool softmax = a.scoring == FFN_MOE_SOFTMAX;

  float l[EPL];
  double key[EPL];
  bool bad = false;
  double mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    l[i] = -INFINITY;
    if (e < E) {
      l[i] = BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.logits)[row * a.ld + e])
                  : static_cast<const float*>(a.logits)[row * a.ld + e];
      bad |= isnan(l[i]) || (softmax && l[i] == INFINITY);
    }
    if (!isnan(l[i])) mx = fmax(mx, (double)l[i]);
  }
  bad = __any_sync(0xffffffffu, bad);
  mx = warp_max(mx);
  double lse = 0.0;
  if (softmax) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (l[i] > -INFINITY) sum += exp((double)l[i] - mx);
    lse = mx + log(warp_sum64(sum));
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = -INFINITY;
    if (e < E && l[i] > -INFINITY) {
      double c = softmax ? (l[i] == INFINITY ? 1.0 : exp((double)l[i] - lse)) : 1.0 / (1.0 + exp(-(double)l[i]));
      if (isnan(c)) c = 0.0;  // another expert's +inf: the row's weights are NaN, its ids go by the keys all the same
      if (a.bias) c += (double)a.bias[e];
      if (c > -INFINITY) key[i] = c;
    }
  }

  if (a.groups > 1) {
    double* keys = route_smem + (size_t)warp * E;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 32 * i < E) keys[lane + 32 * i] = key[i];
    __syncwarp();
    const int size = E / a.groups;
    double best = -INFINITY, second = -INFINITY;
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) {
        const double c = keys[lane * size + i];
        second = fmax(second, fmin(best, c));
        best = fmax(best, c);
      }
    if (a.group_score == FFN_MOE_GROUP_TOP2 && second > -INFINITY) best += second;
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl_sync(0xffffffffu, best, g);
      rank += o > best || (o == best && g < lane);
    }
    const uint32_t open = __ballot_sync(0xffffffffu, lane < a.groups && rank < a.top_groups);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !((open >> (e / size)) & 1u)) key[i] = -INFINITY;
    }
  }

  // top_k rounds of a warp-wide maximum; lane j keeps the j-th choice
  int my_id = -1;
  float my_l = -INFINITY;
  for (int j = 0; j < a.top_k; ++j) {
    double best = -INFINITY;
    int at = 0x7fffffff;
    float bl = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = lane + 32 * i;
        bl = l[i];
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      const float ol = __shfl_xor_sync(0xffffffffu, bl, o);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
        bl = ol;
      }
    }
    if (best == -INFINITY) break;  // nothing is left
    if (lane == j) {
      my_id = at;
      my_l = bl;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (at == lane + 32 * i) key[i] = -INFINITY;
  }

  // Renormalised weights go through the logarithms, so that scores that
  // underflow still have their ratio.
  double log_s = -INFINITY, w = 0.0;
  if (my_id >= 0) log_s = softmax ? (double)my_l - lse : log_sigmoid((double)my_l);
  if (a.renormalize) {
    const double top = warp_max(log_s);
    const double s = my_id >= 0 ? exp(log_s - top) : 0.0;
    const double sum = warp_sum64(s);
    if (my_id >= 0) w = s / sum;
  } else if (my_id >= 0) {
    w = exp(log_s);
  }
  if (lane < a.top_k) {
    a.ids[row * a.top_k + lane] = my_id;
    a.weights[row * a.top_k + lane] = bad ? NAN : (float)(w * (double)a.scale);
  }
}

template <bool BF16>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.m + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
  const size_t smem = a.groups > 1 ? sizeof(double) * kRouteWarps * a.experts : 0;
  ProfScope prof(s, "moe_route");
  if (a.experts <= 64) return launch_pdl(moe_route_kernel<2, BF16>, grid, block, smem, s, a);
  if (a.experts <= 256) return launch_pdl(moe_route_kernel<8, BF16>, grid, block, smem, s, a);
  return launch_pdl(moe_route_kernel<32, BF16>, grid, block, smem, s, a);
}

}  // namespace
}  // namespace ffn

extern "C" ffn_status ffn_nvfp4_moe_route(const void* logits, ffn_logits_type type, int64_t m, int64_t experts,
                                          int64_t row_stride, const float* bias, const ffn_moe_router* router,
                                          int32_t* ids, float* weights, void* stream) {
  if (m < 0 || !router) return FFN_ERR_INVALID_ARG;
  if (type != FFN_LOGITS_F32 && type != FFN_LOGITS_BF16) return FFN_ERR_INVALID_ARG;
  const ffn_moe_router& r = *router;
  if (r.scoring != FFN_MOE_SOFTMAX && r.scoring != FFN_MOE_SIGMOID) return FFN_ERR_INVALID_ARG;
  if (r.group_score != FFN_MOE_GROUP_MAX && r.group_score != FFN_MOE_GROUP_TOP2) return FFN_ERR_INVALID_ARG;
  if (!(fabsf(r.scale) < INFINITY)) return FFN_ERR_INVALID_ARG;
  if (experts < 1 || r.top_k < 1 || r.groups < 1 || r.top_groups < 1 || r.top_groups > r.groups || row_stride < experts)
    return FFN_ERR_INVALID_ARG;
  if (experts % r.groups || r.top_k > experts / r.groups * r.top_groups) return FFN_ERR_SHAPE;
  if (experts > FFN_MOE_MAX_EXPERTS || r.top_k > FFN_MOE_MAX_TOP_K || r.groups > FFN_MOE_MAX_GROUPS)
    return FFN_ERR_UNSUPPORTED;
  if (m == 0) return FFN_OK;
  if (!logits || !ids || !weights) return FFN_ERR_INVALID_ARG;
  if (m > INT32_MAX / r.top_k || m > INT64_MAX / 4 / row_stride) return FFN_ERR_SHAPE;
  const uintptr_t mask = type == FFN_LOGITS_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(logits) & mask) || (reinterpret_cast<uintptr_t>(ids) & 3u) ||
      (reinterpret_cast<uintptr_t>(weights) & 3u) || (reinterpret_cast<uintptr_t>(bias) & 3u))
    return FFN_ERR_ALIGNMENT;
  if (ffn_status st = ffn::moe_precheck()) return st;
  ffn::RouteArgs a;
  a.logits = logits;
  a.ld = row_stride;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.m = m;
  a.experts = (int)experts;
  a.top_k = r.top_k;
  a.groups = r.groups;
  a.top_groups = r.top_groups;
  a.scoring = r.scoring;
  a.group_score = r.group_score;
  a.renormalize = r.renormalize != 0;
  a.scale = r.scale;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      type == FFN_LOGITS_BF16 ? ffn::launch_route<true>(a, s) : ffn::launch_route<false>(a, s);
  return ffn::moe_status(e);
}
