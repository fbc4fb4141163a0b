// A router's choice of experts and the gradient of its logits (the operations are
// described in gemm.h at gemm_route and gemm_route_backward).
//
// A token belongs to a row of 16 lanes, so a wave takes four at a time and every
// reduction is four cross-lane steps within a row. Lane l holds the experts
// 64 j + 4 l .. 64 j + 4 l + 3 for j = 0, 1, ..: 16 bytes of float logits a load, whole
// lines over the lanes. The top_k are found one by one: each lane keeps the best of its
// own, a maximum over the row finds the next, its lane looks for another.
//
// Values that the choice compares are exact or 64 bits wide. Both scores rise with the
// logit, so where neither a bias nor sums of a group's scores come in, logits are compared
// themselves (as whole numbers in their order); else the scores are computed in FP64, so that
// experts whose scores lie next to each other are not taken for equal or the other way
// round by roundings of FP32.
#pragma once

#include <hip/hip_runtime.h>

#include "elem.hpp"
#include "lanes.hpp"

namespace gemm {
namespace mx {

constexpr int kRouteMaxExperts = 512, kRouteMaxTopK = 16, kRouteMaxGroups = 64;   // GEMM_ROUTE_MAX_*
constexpr int kSoftmax = 0, kSigmoid = 1;                                          // GEMM_ROUTE_*

struct RouteArgs {
  int tokens, experts, top_k, score, groups, top_groups, group_top, renormalize;
  float scale;
  const void *logits;
  long long ld;
  const float *bias;
  int *chosen;
  float *weights;
  int *counts;             // zeroed, or written whole by the only workgroup
  unsigned group_mul;      // e * group_mul >> 20 = e / (experts / groups) for e < 512
  int group_size;
};

struct RouteGradArgs {
  int tokens, experts, top_k, score, renormalize;
  float scale;
  const void *logits;
  long long ld;
  const int *chosen;
  const float *dweights;
  void *dlogits;
  long long ldd;
};

// ---------------------------------------------------------------------------
// Rows of 16 lanes.
template <int CTRL>
__device__ inline double dpp_double(double v) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
  const unsigned lo = static_cast<unsigned>(dpp<CTRL, 0xf>(0, static_cast<int>(b)));
  const unsigned hi = static_cast<unsigned>(dpp<CTRL, 0xf>(0, static_cast<int>(b >> 32)));
  return __builtin_bit_cast(double, static_cast<unsigned long long>(hi) << 32 | lo);
}
__device__ inline double row_max(double v) {
  v = fmax(v, dpp_double<0x121>(v));
  v = fmax(v, dpp_double<0x122>(v));
  v = fmax(v, dpp_double<0x124>(v));
  return fmax(v, dpp_double<0x128>(v));
}
__device__ inline double row_sum(double v) {
  v += dpp_double<0x121>(v);
  v += dpp_double<0x122>(v);
  v += dpp_double<0x124>(v);
  return v + dpp_double<0x128>(v);
}
__device__ inline float row_max(float v) {
  return __builtin_bit_cast(float, row_all(__builtin_bit_cast(int, v), [](int a, int b) {
    return __builtin_bit_cast(int, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
  }));
}
// v of the row's lane n.
template <class T>
__device__ inline T row_lane(T v, int n) {
  return __shfl(v, n, 16);
}
// A sum over the row, the same bits in every lane (each lane adds in another order, so
// one's sum is taken): equal scores stay equal whichever lanes hold them.
template <class T>
__device__ inline T row_total(T v) {
  return row_lane(row_sum(v), 0);
}

// What the choice compares: whole numbers in the order of logits, 0 for one that is not
// to be chosen; or values of 64 bits, -inf for those.
template <class KEY>
struct KeyOf;
template <>
struct KeyOf<unsigned> {
  static constexpr unsigned none = 0;
  static __device__ inline bool some(unsigned k) { return k != 0; }
};
template <>
struct KeyOf<double> {
  static constexpr double none = -__builtin_huge_val();
  static __device__ inline bool some(double k) { return k > -__builtin_huge_val(); }
};
__device__ inline unsigned logit_key(float v) {   // v finite or +inf
  const unsigned b = __builtin_bit_cast(unsigned, v + 0.0f);   // -0 equals +0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// 4 consecutive logits of a row from expert e on; -inf past the last.
template <int TYPE>
__device__ inline void load_logits(const typename Elem<TYPE>::store *row, int e, int experts, float *v) {
  typedef typename Elem<TYPE>::store store;
  typedef store store4 __attribute__((ext_vector_type(4), aligned(sizeof(store))));
  if (e + 4 <= experts) {
    const store4 x = *reinterpret_cast<const store4 *>(row + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = Elem<TYPE>::get(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = e + i < experts ? Elem<TYPE>::get(row[e + i]) : -__builtin_inff();
  }
}
__device__ inline int expert_of(int j, int l16) { return (j >> 2) * 64 + l16 * 4 + (j & 3); }

// The best of a lane's keys and the expert it belongs to (the lowest of equal ones: a
// lane's experts ascend).
template <int PER, class KEY>
__device__ inline void best_of(const KEY (&key)[PER], int l16, KEY &best, int &at) {
  best = KeyOf<KEY>::none;
  at = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (key[j] > best) {
      best = key[j];
      at = j;
    }
  }
  at = expert_of(at, l16);
}

// The best groups, as bits: a group's value is the largest key of its experts or the sum
// of the two largest. The row's keys pass through LDS, where a lane looks a whole group over,
// starting at another place than its neighbours (their groups lie a multiple of some
// power of two apart).
template <int PER, class KEY>
__device__ inline unsigned long long best_groups(const RouteArgs &a, const KEY (&key)[PER], int l16, KEY *keys) {
  wave_order();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = expert_of(j, l16);
    if (e < a.experts) keys[e] = key[j];
  }
  wave_order();
  constexpr int kMine = kRouteMaxGroups / 16;
  KEY value[kMine];
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int g = m * 16 + l16;
    KEY first = KeyOf<KEY>::none, second = KeyOf<KEY>::none;
    if (g < a.groups) {
      int at = l16 % a.group_size;
      for (int i = 0; i < a.group_size; ++i) {
        const KEY k = keys[g * a.group_size + at];
        if (++at == a.group_size) at = 0;
        second = k > first ? first : k > second ? k : second;
        first = k > first ? k : first;
      }
    }
    // (whole numbers are compared where the largest alone counts)
    if constexpr (sizeof(KEY) == 8)
      value[m] = a.group_top == 2 && KeyOf<KEY>::some(second) ? first + second : first;
    else
      value[m] = first;
  }
  unsigned long long stay = 0;
  for (int n = 0; n < a.top_groups; ++n) {
    KEY best = KeyOf<KEY>::none;
    int at = kRouteMaxGroups;
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      if (value[m] > best) {
        best = value[m];
        at = m * 16 + l16;
      }
    }
    const KEY most = row_max(best);
    if (!KeyOf<KEY>::some(most)) break;   // (rows differ: the lanes of one leave together)
    const int g = row_min(best == most ? at : kRouteMaxGroups);
    stay |= 1ull << g;
#pragma unroll
    for (int m = 0; m < kMine; ++m)
      if (m * 16 + l16 == g) value[m] = KeyOf<KEY>::none;
  }
  return stay;
}

// Routes the token t of this lane's row.
template <int TYPE, int PER, class KEY>
__device__ inline void route_token(const RouteArgs &a, long long t, int *counts, KEY *keys) {
  typedef typename Elem<TYPE>::store store;
  const int l16 = threadIdx.x & 15;
  const store *row = static_cast<const store *>(a.logits) + t * a.ld;
  float l[PER];
#pragma unroll
  for (int j = 0; j < PER; j += 4) load_logits<TYPE>(row, expert_of(j, l16), a.experts, &l[j]);
  // A NaN, for softmax also +inf, leaves the token without experts.
  unsigned largest = 0;
  float top = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const unsigned b = __builtin_bit_cast(unsigned, l[j]);
    largest = max(largest, b == 0xff800000u ? 0u : b & 0x7fffffffu);
    top = fmaxf(top, l[j]);
  }
  top = row_max(top);
  bool bad = row_max(largest) >= (a.score == kSoftmax ? 0x7f800000u : 0x7f800001u);
  KEY key[PER];
  if constexpr (sizeof(KEY) == 4) {
#pragma unroll
    for (int j = 0; j < PER; ++j) key[j] = l[j] == -__builtin_inff() ? 0u : logit_key(l[j]);
  } else {
    double s[PER], sum = 0.0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (a.score == kSoftmax) {
        s[j] = exp(static_cast<double>(l[j]) - static_cast<double>(top));
        sum += s[j];
      } else {
        s[j] = 1.0 / (1.0 + exp(-static_cast<double>(l[j])));
      }
    }
    const double scale = a.score == kSoftmax ? row_total(sum) : 1.0;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = expert_of(j, l16);
      double v = a.score == kSoftmax ? s[j] / scale : s[j];
      if (a.bias && e < a.experts) {
        const float b = a.bias[e];
        nan |= b != b;
        v += static_cast<double>(b);
      }
      key[j] = l[j] == -__builtin_inff() ? KeyOf<KEY>::none : v;
    }
    bad |= row_max(nan ? 1u : 0u) != 0;
  }
  if (a.groups > a.top_groups) {
    const unsigned long long stay = best_groups<PER, KEY>(a, key, l16, keys);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const unsigned g = (static_cast<unsigned>(expert_of(j, l16)) * a.group_mul) >> 20;
      if (!(stay >> (g & 63) & 1)) key[j] = KeyOf<KEY>::none;
    }
  }
  KEY best;
  int at;
  best_of<PER, KEY>(key, l16, best, at);
  int mine = -1;
  for (int n = 0; n < a.top_k; ++n) {
    const KEY most = row_max(best);
    const int expert = row_min(best == most ? at : kRouteMaxExperts);
    if (l16 == n && KeyOf<KEY>::some(most) && !bad) mine = expert;
    if (expert == at && KeyOf<KEY>::some(best)) {   // its lane looks for its next
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (expert_of(j, l16) == expert) key[j] = KeyOf<KEY>::none;
      best_of<PER, KEY>(key, l16, best, at);
    }
  }
  // Weights: lane n has the n-th choice. Renormalised ones are ratios to the largest
  // chosen score, which neither underflow together nor divide zero by zero:
  // sigmoid(l) = e^min(l, 0) / (1 + e^-|l|).
  const bool live = mine >= 0;
  const float logit = live ? Elem<TYPE>::get(row[mine]) : -__builtin_inff();
  float w = 0.0f;
  if (a.renormalize) {
    const float most = row_max(logit);
    if (a.score == kSoftmax)
      w = expf(logit - most);
    else
      w = expf(fminf(logit, 0.0f) - fminf(most, 0.0f)) / (1.0f + expf(-fabsf(logit)));
    w = live ? w : 0.0f;
    w /= row_total(w);
  } else if (a.score == kSoftmax) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += expf(l[j] - top);
    w = expf(logit - top) / row_total(sum);
  } else {
    w = logit >= 0.0f ? 1.0f / (1.0f + expf(-logit)) : expf(logit) / (1.0f + expf(logit));
  }
  if (l16 < a.top_k) {
    const long long out = t * a.top_k + l16;
    a.chosen[out] = mine;
    a.weights[out] = bad ? __builtin_nanf("") : live ? a.scale * w : 0.0f;
    if (counts && live) atomicAdd(&counts[mine], 1);
  }
}

// Tokens over the rows of the grid's workgroups, each row taking every so many. Counts
// are summed in LDS; a workgroup that is the only one writes them whole, several add theirs
// (whole numbers: the order of the additions does not show).
template <int TYPE, int PER, class KEY, int THREADS>
__global__ __launch_bounds__(THREADS) void route_kernel(RouteArgs a) {
  __shared__ int counts[kRouteMaxExperts];
  extern __shared__ __attribute__((aligned(16))) unsigned char dynamic[];   // a key for each row's experts, with groups
  if (a.counts) {
    for (int e = threadIdx.x; e < a.experts; e += THREADS) counts[e] = 0;
    __syncthreads();
  }
  const int row = threadIdx.x >> 4;
  KEY *keys = reinterpret_cast<KEY *>(dynamic) + row * a.experts;
  const long long rows = static_cast<long long>(gridDim.x) * (THREADS / 16);
  for (long long t = static_cast<long long>(blockIdx.x) * (THREADS / 16) + row; t < a.tokens; t += rows)
    route_token<TYPE, PER, KEY>(a, t, a.counts ? counts : nullptr, keys);
  if (a.counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += THREADS) {
      if (gridDim.x == 1) a.counts[e] = counts[e];
      else if (counts[e]) atomicAdd(&a.counts[e], counts[e]);
    }
  }
}

__global__ __launch_bounds__(512) void zero_counts_kernel(int *counts, int n) {
  if (static_cast<int>(threadIdx.x) < n) counts[threadIdx.x] = 0;
}

// The gradient of the logits. Lane n of a row has the token's n-th choice, and but for
// softmax without renormalising everything that is not zero comes from there:
//   softmax:              d_j = scale p_j ([j chosen] dw_j - sum dw_e p_e)
//   softmax renormalised: d_j = scale q_j (dw_j - sum q_e dw_e), j chosen
//   sigmoid:              d_j = scale s_j (1 - s_j) dw_j, j chosen
//   sigmoid renormalised: d_j = scale q_j (1 - s_j) (dw_j - sum q_e dw_e), j chosen
// with q the renormalised weights (without scale). Choices past the experts (-1) count
// nothing; a token without a choice gets zeros.
template <int TYPE, int PER>
__device__ inline void route_grad_token(const RouteGradArgs &a, long long t) {
  typedef typename Elem<TYPE>::store store;
  const int l16 = threadIdx.x & 15;
  const store *row = static_cast<const store *>(a.logits) + t * a.ld;
  const bool whole = a.score == kSoftmax && !a.renormalize;
  int e = -1;
  float dw = 0.0f, logit = -__builtin_inff();
  if (l16 < a.top_k) {
    e = a.chosen[t * a.top_k + l16];
    if (e < 0 || e >= a.experts) e = -1;
  }
  if (e >= 0) {
    dw = a.scale * a.dweights[t * a.top_k + l16];
    logit = Elem<TYPE>::get(row[e]);
  }
  const bool live = e >= 0;
  float d[PER], mine;
  float l[PER], top = 0.0f, inverse = 0.0f;
  if (whole) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; j += 4) load_logits<TYPE>(row, expert_of(j, l16), a.experts, &l[j]);
    top = l[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) top = fmaxf(top, l[j]);
    top = row_max(top);
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += l[j] = expf(l[j] - top);
    inverse = 1.0f / row_total(sum);
    const float p = live ? expf(logit - top) * inverse : 0.0f;
    mine = live ? p * dw : 0.0f;
    const float all = row_total(mine);
    const bool any = row_max(live ? 1u : 0u) != 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) d[j] = any ? -(l[j] * inverse) * all : 0.0f;
  } else {
    float s = 0.0f, rest = 0.0f;   // sigmoid(logit) and 1 - sigmoid(logit), each to its own precision
    if (a.score == kSigmoid) {
      const float small = expf(-fabsf(logit));
      const float big = 1.0f / (1.0f + small);
      s = logit >= 0.0f ? big : small * big;
      rest = logit >= 0.0f ? small * big : big;
    }
    if (a.renormalize) {
      const float most = row_max(logit);
      float q = a.score == kSoftmax ? expf(logit - most)
                                    : expf(fminf(logit, 0.0f) - fminf(most, 0.0f)) / (1.0f + expf(-fabsf(logit)));
      q = live ? q : 0.0f;
      q /= row_total(q);
      const float all = row_total(live ? q * dw : 0.0f);
      mine = q * (dw - all);
      if (a.score == kSigmoid) mine *= rest;
    } else {
      mine = s * rest * dw;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) d[j] = 0.0f;
  }
  mine = live ? mine : 0.0f;
  // Each choice to the lane that holds its expert, in order: one named twice counts twice.
  for (int n = 0; n < a.top_k; ++n) {
    const int expert = row_lane(e, n);
    const float v = row_lane(mine, n);
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (expert_of(j, l16) == expert) d[j] += v;
  }
  store *out = static_cast<store *>(a.dlogits) + t * a.ldd;
  typedef store store4 __attribute__((ext_vector_type(4), aligned(sizeof(store))));
#pragma unroll
  for (int j = 0; j < PER; j += 4) {
    const int first = expert_of(j, l16);
    if (first + 4 <= a.experts) {
      store4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = Elem<TYPE>::put(d[j + i]);
      *reinterpret_cast<store4 *>(out + first) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (first + i < a.experts) out[first + i] = Elem<TYPE>::put(d[j + i]);
    }
  }
}

template <int TYPE, int PER>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradArgs a) {
  const long long rows = static_cast<long long>(gridDim.x) * 16;
  for (long long t = static_cast<long long>(blockIdx.x) * 16 + (threadIdx.x >> 4); t < a.tokens; t += rows)
    route_grad_token<TYPE, PER>(a, t);
}

}  // namespace mx
}  // namespace gemm
