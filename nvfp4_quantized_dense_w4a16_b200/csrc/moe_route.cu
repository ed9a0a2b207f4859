// Routing of rows to experts: scores of E experts per row -> the top_k experts
// and their weights (ffn_nvfp4_moe_route).
//
// With s = softmax(l) or sigmoid(l) of a row's logits, the choice goes by the
// keys c = s + bias (optionally only inside the best groups of experts) and
// the weights by s alone, renormalised over the chosen experts on request.
//
// One warp owns one row; lane l holds experts l * EPL .. l * EPL + EPL - 1 in
// registers.  Finite keys that 64 bits do not tell apart (scores that saturate or
// underflow) go by their logits, so that of experts of equal biases the logits
// alone decide.  Without a bias (and with group scores that are maxima) they are
// compared as they are: exact, and the order that a bias of zeros gives.  Else the
// keys are computed in fp32, and the row is computed again in 64 bits where two
// keys whose order matters are closer than their errors: the choice is always
// that of 64-bit arithmetic, and few rows in a thousand pay for it.  A key's
// error goes by its score, which its bias may cancel: a key that seems to stand
// far behind may belong in front.  So distances are held against the largest
// error of the row first, and where that is too much against each key's own.
//
// Bound by instructions: the logits and results of 16384 rows of 128 experts are
// 0.8 us of memory traffic, and 8 choices of each take 10.3 us at 520 instructions
// a row (67% of the issue slots): half of them the rounds of a warp-wide maximum,
// whose lanes hold their keys sorted, half the softmax.  fp32 keys need a vote and
// two shuffles a round to find the winner; bf16 keys carry their id in the word
// (12.9 -> 10.7 us).  509 rows of 256 with groups and a bias, one row a warp and
// four warps an SM, take 6.1 us: the latency of one row, of one that 64 bits settle
// (5.5 without such rows).
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

__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// exp(a - b) for a <= b, to about two fp32 steps: the difference's rounding
// error multiplies the result.  Zero for a far below b.
__device__ __forceinline__ float exp_diff(float a, float b) {
  const float d = a - b, bb = a - d;  // a - b = d + lo, lo = (a - (d + bb)) + (bb - b)
  const float lo = (a - (d + bb)) + (bb - b);
  return d > -200.0f ? expf(d) * (1.0f + lo) : 0.0f;
}

// sigmoid to about three fp32 steps.
__device__ __forceinline__ float sigmoid_f32(float l) {
  const float e = expf(-fabsf(l));
  return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// The experts of the row that may be chosen after the groups: keys of the
// others become -inf.  Key is float or double.  Returns how near the worst
// group kept and the best one left out are (infinity: no matter).  Equal finite
// maxima go by the logits l of the experts that they belong to (double: fp32 is
// never left to decide between near scores).
template <int EPL, typename Key>
__device__ __forceinline__ Key keep_best_groups(const RouteArgs& a, Key (&key)[EPL], const float (&l)[EPL], int lane,
                                                Key* smem) {
  const int size = a.experts / a.groups;
  const bool top2 = a.group_score == FFN_MOE_GROUP_TOP2;
  Key best = -INFINITY, second = -INFINITY;  // of group `lane` (or of the lane's group)
  auto take = [&](Key c) {
    second = fmax(second, fmin(best, c));
    best = fmax(best, c);
  };
  const int span = size / EPL;  // lanes of a group, where it is whole lanes
  const bool whole = size % EPL == 0 && (span & (span - 1)) == 0;
  if (whole) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) take(key[i]);
    for (int o = 1; o < span; o <<= 1) {
      const Key ob = __shfl_xor_sync(0xffffffffu, best, o), os = __shfl_xor_sync(0xffffffffu, second, o);
      second = fmax(fmax(second, os), fmin(best, ob));
      best = fmax(best, ob);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane * EPL + i < a.experts) smem[lane * EPL + i] = key[i];
    __syncwarp();
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) take(smem[lane * size + i]);
    __syncwarp();
  }
  constexpr bool kTies = sizeof(Key) == 8;
  float tie = 0.0f;
  if (kTies && !top2) {
    tie = -INFINITY;
    if (whole) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (key[i] == best) tie = fmaxf(tie, l[i]);
      for (int o = 1; o < span; o <<= 1) tie = fmaxf(tie, __shfl_xor_sync(0xffffffffu, tie, o));
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        const Key its = __shfl_sync(0xffffffffu, best, min(e / size, 31));
        if (e < a.experts) smem[e] = key[i] == its ? (Key)l[i] : (Key)-INFINITY;
      }
      __syncwarp();
      if (lane < a.groups)
        for (int i = 0; i < size; ++i) tie = fmaxf(tie, (float)smem[lane * size + i]);
      __syncwarp();
    }
    if (!(best < INFINITY)) tie = 0.0f;
  }
  if (top2 && second > -INFINITY) best += second;
  // rank among the groups: ties to the lower one
  const int step = whole ? span : 1, mine = whole ? lane / span : lane;
  int rank = 0;
  for (int g = 0; g < a.groups; ++g) {
    const Key o = __shfl_sync(0xffffffffu, best, g * step);
    bool first = g < mine;
    if constexpr (kTies) {
      const float ot = __shfl_sync(0xffffffffu, tie, g * step);
      first = (ot > tie) | ((ot == tie) & first);
    }
    rank += o > best || (o == best && first);
  }
  const bool in = mine < a.groups, kept = in && rank < a.top_groups;
  Key low = kept ? best : (Key)INFINITY, high = in && !kept ? best : (Key)-INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    low = fmin(low, __shfl_xor_sync(0xffffffffu, low, o));
    high = fmax(high, __shfl_xor_sync(0xffffffffu, high, o));
  }
  const uint32_t open = __ballot_sync(0xffffffffu, kept);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int g = whole ? lane : min((lane * EPL + i) / size, 31);
    if (!((open >> g) & 1u)) key[i] = -INFINITY;
  }
  return high > -INFINITY && low < INFINITY ? low - high : (Key)INFINITY;
}

// Batcher's odd-even merge sort of EPL registers: order(x, y) for x < y puts the
// better one at x.
template <int EPL, typename Order>
__device__ __forceinline__ void merge_sort(Order order) {
#pragma unroll
  for (int p = 1; p < EPL; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j <= EPL - 1 - k; j += 2 * k)
#pragma unroll
        for (int i = 0; i <= (k - 1 < EPL - j - k - 1 ? k - 1 : EPL - j - k - 1); ++i)
          if ((i + j) / (p * 2) == (i + j + k) / (p * 2)) order(i + j, i + j + k);
}

// The row's choice in 64 bits: lane j gets the j-th id (-1: none).
template <int EPL>
__device__ __noinline__ int choose_64(const RouteArgs& a, const float (&l)[EPL], int lane, double* smem) {
  const bool softmax = a.scoring == FFN_MOE_SOFTMAX;
  double key[EPL];
  float tie[EPL];
  double top = -INFINITY, sum = 0.0;
  if (softmax) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = fmax(top, (double)l[i]);
    top = warp_max(top);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (l[i] > -INFINITY) sum += exp((double)l[i] - top);
    sum = warp_sum64(sum);
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    key[i] = -INFINITY;
    if (l[i] > -INFINITY) {
      double c = softmax ? (l[i] == INFINITY ? 1.0 : exp((double)l[i] - top) / sum) : 1.0 / (1.0 + exp(-(double)l[i]));
      if (isnan(c)) c = 0.0;  // beside a logit of +inf
      if (a.bias) c += (double)a.bias[lane * EPL + i];
      if (c > -INFINITY) key[i] = c;
    }
    tie[i] = key[i] < INFINITY ? l[i] : 0.0f;  // what equal keys go by, before the id
  }
  if (a.groups > 1) keep_best_groups<EPL, double>(a, key, l, lane, smem);
  int mine = -1;
  for (int j = 0; j < a.top_k; ++j) {
    double best = -INFINITY;
    float best_tie = -INFINITY;
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool take = (key[i] > best) | ((key[i] == best) & (key[i] > -INFINITY) & (tie[i] > best_tie));
      best = take ? key[i] : best;
      best_tie = take ? tie[i] : best_tie;
      at = take ? lane * EPL + i : at;
    }
    // the warp's best by maxima of words in the numbers' order: the key's two
    // halves, the logit; of equal ones the lowest lane
    const long long bits = __double_as_longlong(best + 0.0);  // (one zero)
    const unsigned long long up = bits ^ ((bits >> 63) | (long long)0x8000000000000000ull);
    const uint32_t hi = (uint32_t)(up >> 32), lo = (uint32_t)up;
    const int tbits = __float_as_int(best_tie + 0.0f);
    const uint32_t top_hi = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t top_lo = __reduce_max_sync(0xffffffffu, hi == top_hi ? lo : 0u);
    const bool equal = hi == top_hi && lo == top_lo;
    const uint32_t order = equal ? tbits ^ ((tbits >> 31) | 0x80000000u) : 0u;
    const uint32_t top_order = __reduce_max_sync(0xffffffffu, order);
    const int w = __ffs(__ballot_sync(0xffffffffu, equal && order == top_order)) - 1;
    best = __shfl_sync(0xffffffffu, best, w);
    at = __shfl_sync(0xffffffffu, at, w);
    if (best == -INFINITY) break;  // nothing is left
    if (lane == j) mine = at;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (at == lane * EPL + i) key[i] = -INFINITY;
  }
  return mine;
}

// EPL logits of the row from expert lane * EPL on; -inf past the last expert.
template <int EPL, bool BF16, bool WIDE>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t row, int lane, float (&l)[EPL]) {
  constexpr int kBytes = EPL * (BF16 ? 2 : 4);
  const char* p = static_cast<const char*>(a.logits) + (row * a.ld + lane * EPL) * (BF16 ? 2 : 4);
  if (WIDE && lane * EPL < a.experts) {  // E is a multiple of EPL and every lane's logits are aligned
    uint32_t w[(kBytes + 3) / 4];
    if (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = kBytes == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      l[i] = BF16 ? bf16_bits_to_float((w[i / 2] >> (16 * (i & 1))) & 0xffffu) : __uint_as_float(w[i]);
    return;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    l[i] = -INFINITY;
    if (!WIDE && lane * EPL + i < a.experts)
      l[i] = BF16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
  }
}

// The choice by bf16 keys: a word holds a key, in an order that unsigned numbers
// have, above the id's complement, so that one maximum over the warp gives the
// best key and of equal ones the lowest id.  Lane j gets the j-th id (-1: none)
// and its logit.
template <int EPL>
__device__ __forceinline__ void choose_words(const float (&key)[EPL], int lane, int top_k, int& my_id, float& my_l) {
  uint32_t w[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const uint32_t b = __float_as_uint(key[i] + 0.0f);  // (one zero)
    const uint32_t up = (b ^ ((uint32_t)((int)b >> 31) | 0x80000000u)) & 0xffff0000u;
    w[i] = key[i] > -INFINITY ? up | (0xffffu - (lane * EPL + i)) : 0u;
  }
  constexpr bool kSorted = EPL <= 8;
  auto order = [&](int x, int y) {
    const uint32_t hi = max(w[x], w[y]), lo = min(w[x], w[y]);
    w[x] = hi, w[y] = lo;
  };
  if (kSorted) merge_sort<EPL>(order);
  uint32_t head = w[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i)
    if (!kSorted) head = max(head, w[i]);
  uint32_t mine = 0;
  for (int j = 0; j < top_k; ++j) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, head);
    if (best == 0) break;  // nothing is left
    if (lane == j) mine = best;
    if (head == best) {
      if (kSorted) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) w[i] = i + 1 < EPL ? w[i + 1] : 0u;
        head = w[0];
      } else {
        head = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) head = max(head, w[i] < best ? w[i] : 0u);
      }
    }
  }
  if (mine) {
    my_id = 0xffff - (int)(mine & 0xffffu);
    const uint32_t b = mine & 0xffff0000u;
    my_l = __uint_as_float(b & 0x80000000u ? b ^ 0x80000000u : ~b & 0xffff0000u);
  }
}

// Ten CTAs an SM for up to 128 experts: 48 registers (16384 x 128: 10.3 us, 10.4
// with the 52 to 56 that the compiler takes by itself).
template <int EPL, bool BF16, bool WIDE>
__global__ void __launch_bounds__(kRouteWarps * 32, EPL <= 4 ? 10 : 0) moe_route_kernel(const RouteArgs a) {
  extern __shared__ double route_smem[];  // [warps][experts], only with groups that are not whole lanes
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (row >= a.m) return;
  const bool softmax = a.scoring == FFN_MOE_SOFTMAX;
  // do the keys need more than the logits' order, does anything need the sum?
  const bool scored = a.bias || (a.groups > 1 && a.group_score == FFN_MOE_GROUP_TOP2);
  const bool summed = softmax && (scored || !a.renormalize);

  float l[EPL], key[EPL];
  load_logits<EPL, BF16, WIDE>(a, row, lane, l);
  bool bad = false;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    bad |= isnan(l[i]) || (softmax && l[i] == INFINITY);
    if (isnan(l[i])) l[i] = -INFINITY;
    top = fmaxf(top, l[i]);
  }
  bad = __any_sync(0xffffffffu, bad);
  float sum = 0.0f;
  if (summed) {
    top = redux_max(top);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = l[i] == INFINITY ? 1.0f : l[i] > -INFINITY ? exp_diff(l[i], top) : 0.0f;
      sum += key[i];
    }
    sum = warp_sum(sum);
  }
  // An upper bound of a score's relative error: softmax has EPL + 5 additions
  // and about ten steps of the exponentials and the quotient, sigmoid three;
  // a key's adds a step of its size.  Below the normal range errors are steps of
  // 2^-149: keys that are all this small are always close.
  constexpr float kStep = 1.1920929e-7f, kTiny = 1e-37f;
  const float err = (softmax ? EPL + 16 : 4) * kStep;
  auto key_error = [&](float score, float c) { return err * score + 2.0f * kStep * (fabsf(c) + score) + kTiny; };
  float most = 0.0f;  // the largest score or key of the row, those of groups that get closed as well
  if (scored) {
    const float inv = summed ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float score = softmax ? key[i] * inv : sigmoid_f32(l[i]);
      float c = score;
      if (a.bias && l[i] > -INFINITY) c += a.bias[lane * EPL + i];
      key[i] = l[i] > -INFINITY && c > -INFINITY ? c : -INFINITY;
      if (key[i] > -INFINITY) most = fmaxf(most, fmaxf(score, fabsf(c)));
    }
    most = redux_max(most);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = l[i];
  }
  bool close = false;
  if (a.groups > 1) {
    const float gap =
        keep_best_groups<EPL, float>(a, key, l, lane, reinterpret_cast<float*>(route_smem + (size_t)warp * a.experts));
    // (up to four scores, each at most one; two large keys may cancel in their sum)
    close = scored && gap <= 4.0f * err + 8.0f * kStep * most + kTiny;
  }

  int my_id = -1, slot = lane;  // a choice, and which one it is
  float my_l = -INFINITY;
  if (BF16 && !scored) {
    choose_words<EPL>(key, lane, a.top_k, my_id, my_l);
  } else {
    // rounds of a warp-wide maximum; lane j keeps the j-th choice, and lane top_k
    // the runner-up where its distance matters
    float my_c = -INFINITY;
    // each lane's keys in descending order (equal ones by id), so that a round
    // only looks at their heads; up to eight: a longer list is scanned again
    constexpr bool kSorted = EPL <= 8;
    int at[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) at[i] = i;
    auto swap_if = [&](int x, int y) {
      const bool s = key[y] > key[x] || (key[y] == key[x] && at[y] < at[x]);
      const float kx = key[x], lx = l[x];
      const int ax = at[x];
      key[x] = s ? key[y] : kx, key[y] = s ? kx : key[y];
      l[x] = s ? l[y] : lx, l[y] = s ? lx : l[y];
      at[x] = s ? at[y] : ax, at[y] = s ? ax : at[y];
    };
    if (kSorted) merge_sort<EPL>(swap_if);
    auto to_front = [&] {  // the best of the list to its head
      if (kSorted) return;
#pragma unroll
      for (int i = 1; i < EPL; ++i) swap_if(0, i);
    };
    to_front();
    auto choose = [&](int from, int to) {  // the rounds from .. to - 1; how many choices there are
      for (int j = from; j < to; ++j) {
        const float c = redux_max(key[0]);
        if (c == -INFINITY) return j;  // nothing is left
        const int w = __ffs(__ballot_sync(0xffffffffu, key[0] == c)) - 1;  // the lowest lane: the lowest id
        const int id = __shfl_sync(0xffffffffu, lane * EPL + at[0], w);
        const float wl = __shfl_sync(0xffffffffu, l[0], w);
        if (lane == j) {
          my_id = id;
          my_l = wl;
          my_c = c;
        }
        if (lane == w) {
#pragma unroll
          for (int i = 0; i < EPL; ++i) {
            if (!kSorted && i > 0) break;
            key[i] = kSorted && i + 1 < EPL ? key[i + 1] : -INFINITY;
            if (kSorted && i + 1 < EPL) l[i] = l[i + 1], at[i] = at[i + 1];
          }
          to_front();
        }
      }
      return to;
    };
    int found = choose(0, min(32, a.top_k + scored));
    if (scored) {
      // Is a choice nearer to the next one than the largest errors of the row?  With all
      // 32 lanes taken by choices there is no room for the runner-up: such rows
      // are always computed in 64 bits.
      const float next = __shfl_down_sync(0xffffffffu, my_c, 1);
      const bool near = lane + 1 < found && !(my_c - next > 2.0f * key_error(most, most));
      bool whole = __any_sync(0xffffffffu, close) || a.top_k == 32 || bad || !(most < INFINITY);
      const uint32_t nears = __ballot_sync(0xffffffffu, near);
      if (!whole && nears) {
        // Each key's own error, |c - b| in place of its score.
        auto bias_of = [&](int id) { return a.bias ? a.bias[id] : 0.0f; };
        auto top_of = [&](float c, float b) { return c + key_error(fabsf(c - b), c); };
        // How high a key that was not chosen may be, but for those of bias tb and a
        // logit of at most tl: of equal biases the logits decide, then the ids.
        auto left_over = [&](float tl, float tb) {
          float high = -INFINITY;
#pragma unroll
          for (int i = 0; i < EPL; ++i)
            if (key[i] > -INFINITY) {
              const float b = bias_of(lane * EPL + at[i]);
              if (l[i] > tl || b != tb) high = fmaxf(high, top_of(key[i], b));
            }
          return redux_max(high);
        };
        int cut = min(a.top_k, found) - 1;  // the last choice
        float my_b = my_id >= 0 ? bias_of(my_id) : 0.0f;
        const float high = lane < found ? top_of(my_c, my_b) : -INFINITY;
        const float low = my_c - key_error(fabsf(my_c - my_b), my_c);
        // Of neighbours of equal biases and falling logits the last one stands for
        // all, and if the runner-up is such a neighbour of the last choice, it does.
        const float nl = __shfl_down_sync(0xffffffffu, my_l, 1), nb = __shfl_down_sync(0xffffffffu, my_b, 1);
        const bool same = lane + 1 < found && nl <= my_l && nb == my_b;
        float behind = __shfl_down_sync(0xffffffffu, high, 1);
        bool unsure = lane + 1 < found && !same && !(low > behind);
        if (!__any_sync(0xffffffffu, unsure)) {  // no two neighbours are near by their own errors: is any other key?
          const bool cut_same = __shfl_sync(0xffffffffu, same, cut);
          const float rest = left_over(__shfl_sync(0xffffffffu, my_l, cut), __shfl_sync(0xffffffffu, my_b, cut));
          behind = high;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) behind = fmaxf(behind, __shfl_down_sync(0xffffffffu, behind, o));
          behind = fmaxf(__shfl_down_sync(0xffffffffu, behind, 1), rest);
          unsure = lane <= cut + cut_same && !same && !(low > (lane + 1 < found ? behind : rest));
        }
        if (__any_sync(0xffffffffu, unsure)) {
          // Keys in 64 bits settle the order of the choices, and of three more
          // candidates where the runner-up is near the last choice; where another one
          // may stand before the last choice among them, the row is computed.
          if ((nears >> cut) & 1) found = choose(found, min(32, a.top_k + 4));
          my_b = my_id >= 0 ? bias_of(my_id) : 0.0f;
          const float end = __shfl_sync(0xffffffffu, my_c, found - 1);
          double k64 = -INFINITY;
          if (softmax) {
            float r[EPL];
            load_logits<EPL, BF16, WIDE>(a, row, lane, r);
            double total = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
              if (r[i] > -INFINITY) total += exp((double)r[i] - (double)top);
            total = warp_sum64(total);
            k64 = exp((double)my_l - (double)top) / total;
          } else {
            k64 = 1.0 / (1.0 + exp(-(double)my_l));
          }
          k64 += (double)my_b;
          int rank = 0;  // (candidates of equal scores and keys stand in the order of their ids)
          for (int i = 0; i < found; ++i) {
            const double o = __shfl_sync(0xffffffffu, k64, i);
            const float ol = __shfl_sync(0xffffffffu, my_l, i);
            rank += (o > k64) | ((o == k64) & ((ol > my_l) | ((ol == my_l) & (i < lane))));
          }
          if (lane < found) slot = rank;
          cut = __ffs(__ballot_sync(0xffffffffu, slot == min(a.top_k, found) - 1)) - 1;
          const double last = __shfl_sync(0xffffffffu, k64, cut);
          // (nothing is left above the last candidate; the same in all lanes)
          whole = !((double)(end + key_error(most, most)) < last) &&
                  !((double)left_over(__shfl_sync(0xffffffffu, my_l, cut), __shfl_sync(0xffffffffu, my_b, cut)) < last);
        }
      }
      if (whole) {
        slot = lane;
        float r[EPL];  // (the rounds have moved l, and a call's argument stands in memory)
        load_logits<EPL, BF16, WIDE>(a, row, lane, r);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (isnan(r[i])) r[i] = -INFINITY;
        my_id = choose_64<EPL>(a, r, lane, route_smem + (size_t)warp * a.experts);
        // the chosen logits, from the lanes that hold them
        my_l = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const float v = __shfl_sync(0xffffffffu, r[i], my_id >= 0 ? my_id / EPL : 0);
          if (my_id >= 0 && my_id % EPL == i) my_l = v;
        }
      }
    }
  }
  if (slot >= a.top_k) {  // candidates that were not chosen
    my_id = -1;
    my_l = -INFINITY;
  }

  float w = 0.0f;
  if (a.renormalize) {
    // Scores by the best one's exponential (of a logit of at most zero, under
    // sigmoid: e^l / (1 + e^l)), so that scores that underflow keep their ratio.
    const float high = redux_max(my_l);
    if (my_id >= 0) {
      w = softmax || high < 0.0f ? exp_diff(my_l, high) : sigmoid_f32(my_l);
      if (!softmax && high < 0.0f) w /= 1.0f + expf(my_l);
    }
    const float total = warp_sum(w);
    if (my_id >= 0) w /= total;
  } else if (my_id >= 0) {
    w = softmax ? exp_diff(my_l, top) / sum : sigmoid_f32(my_l);
  }
  if (slot < a.top_k) {
    a.ids[row * a.top_k + slot] = my_id;
    a.weights[row * a.top_k + slot] = bad ? NAN : w * a.scale;
  }
}

template <int EPL, bool BF16>
cudaError_t launch_epl(const RouteArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.m + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
  const int size = a.experts / a.groups, span = size / EPL;
  const bool whole = size % EPL == 0 && (span & (span - 1)) == 0;
  const size_t smem = a.groups > 1 && !whole ? sizeof(double) * kRouteWarps * a.experts : 0;
  // one load of up to 16 bytes a time, where every lane's logits start on its boundary
  constexpr int kElem = BF16 ? 2 : 4, kLoad = EPL * kElem < 16 ? EPL * kElem : 16;
  const bool wide = a.experts % EPL == 0 && reinterpret_cast<uintptr_t>(a.logits) % kLoad == 0 &&
                    (a.m == 1 || a.ld * kElem % kLoad == 0);
  return wide ? launch_pdl(moe_route_kernel<EPL, BF16, true>, grid, block, smem, s, a)
              : launch_pdl(moe_route_kernel<EPL, BF16, false>, grid, block, smem, s, a);
}

template <bool BF16>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  ProfScope prof(s, "moe_route");
  if (a.experts <= 32) return launch_epl<1, BF16>(a, s);
  if (a.experts <= 64) return launch_epl<2, BF16>(a, s);
  if (a.experts <= 128) return launch_epl<4, BF16>(a, s);
  if (a.experts <= 256) return launch_epl<8, BF16>(a, s);
  if (a.experts <= 512) return launch_epl<16, BF16>(a, s);
  return launch_epl<32, BF16>(a, s);
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
