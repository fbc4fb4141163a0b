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
// themselves (as whole numbers in their order). Else scores are computed in FP32 first; where
// two values that the choice sets apart lie nearer to each other than their errors (one token in
// some hundred), FP64 values settle it: of a few candidates, a lane each, or of all.
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
  int row_bytes;           // of the LDS that a row's keys pass through
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
// to be chosen; or values, -inf for those: estimates in FP32, or as they are in FP64.
template <class KEY>
struct KeyOf;
template <>
struct KeyOf<unsigned> {
  static constexpr bool sums = false, estimate = false;
  static constexpr unsigned none = 0;
  static __device__ inline bool some(unsigned k) { return k != 0; }
};
template <>
struct KeyOf<float> {
  static constexpr bool sums = true, estimate = true;
  static constexpr float none = -__builtin_inff();
  static __device__ inline bool some(float k) { return k > -__builtin_inff(); }
};
template <>
struct KeyOf<double> {
  static constexpr bool sums = true, estimate = false;
  static constexpr double none = -__builtin_huge_val();
  static __device__ inline bool some(double k) { return k > -__builtin_huge_val(); }
};
// How far two estimates of up to `v` have to lie apart to be in order: a score is off by up to
// `error`, and the bias's addition rounds once. (By the values that are compared, not by the largest of all:
// an expert masked by a bias of -1e9 would leave nothing settled. 4096 tokens on 8 of 256 in groups
// with such a one 41 us and 13.)
__device__ inline float margin(float error, float v) { return fmaf(0x1p-23f, fabsf(v), 2.0f * error); }
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

// The two largest keys of group g, in a row's LDS: looked over by one lane, starting at another
// place than its neighbours (their groups lie a multiple of some power of two apart).
template <class KEY>
__device__ inline void group_top(const RouteArgs &a, int g, int l16, const KEY *keys, KEY &first, KEY &second) {
  first = second = KeyOf<KEY>::none;
  int at = l16 % a.group_size;
  for (int i = 0; i < a.group_size; ++i) {
    const KEY k = keys[g * a.group_size + at];
    if (++at == a.group_size) at = 0;
    second = k > first ? first : k > second ? k : second;
    first = k > first ? k : first;
  }
}
// What a group is worth: a sum of two keys, of estimates half of it: two finite keys near the
// type's lowest value (a bias that masks) would add to -inf in FP32, a group without experts.
template <class KEY>
__device__ inline KEY group_value(const RouteArgs &a, KEY first, KEY second) {
  // (whole numbers are compared where the largest alone counts)
  if constexpr (!KeyOf<KEY>::sums) return first;
  const KEY half = KeyOf<KEY>::estimate ? KEY(0.5) : KEY(1);
  return a.group_top != 2 ? first : KeyOf<KEY>::some(second) ? half * first + half * second : half * first;
}

// The best groups, as bits, from the values of groups l16, l16 + 16, ...; those that stay lose theirs.
constexpr int kRowGroups = kRouteMaxGroups / 16;
template <class KEY>
__device__ inline unsigned long long choose_groups(const RouteArgs &a, KEY (&value)[kRowGroups], int l16) {
  unsigned long long stay = 0;
  for (int n = 0; n < a.top_groups; ++n) {
    KEY best = KeyOf<KEY>::none;
    int at = kRouteMaxGroups;
#pragma unroll
    for (int m = 0; m < kRowGroups; ++m) {
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
    for (int m = 0; m < kRowGroups; ++m)
      if (m * 16 + l16 == g) value[m] = KeyOf<KEY>::none;
  }
  return stay;
}
// The same from a row's keys. With estimates `sure` says whether every group that stays is worth more than
// every other, whatever the errors: half a sum of two is off by the mean of theirs and a rounding of
// its own, error + 2^-24 (|first| + |second|) together; twice the second term, for the bounds' roundings.
template <class KEY>
__device__ inline unsigned long long best_groups(const RouteArgs &a, int l16, const KEY *keys, float error, bool &sure) {
  KEY value[kRowGroups];
  float least[kRowGroups], off[kRowGroups];
#pragma unroll
  for (int m = 0; m < kRowGroups; ++m) {
    value[m] = KeyOf<KEY>::none;
    least[m] = __builtin_inff();
    off[m] = 0.0f;
    if (m * 16 + l16 < a.groups) {
      KEY first, second;
      group_top(a, m * 16 + l16, l16, keys, first, second);
      value[m] = group_value(a, first, second);
      if constexpr (KeyOf<KEY>::estimate) {
        const float both = fabsf(first) + (a.group_top == 2 && KeyOf<KEY>::some(second) ? fabsf(second) : 0.0f);
        off[m] = fmaf(0x1p-23f, fminf(both, 0x1.fffffep127f), error);   // (finite: an infinite bias is exact)
        if (KeyOf<KEY>::some(first)) least[m] = value[m] - off[m];
      }
    }
  }
  const unsigned long long stay = choose_groups(a, value, l16);
  sure = true;
  if constexpr (KeyOf<KEY>::estimate) {
    float most = KeyOf<float>::none;
#pragma unroll
    for (int m = 0; m < kRowGroups; ++m) most = fmaxf(most, value[m] + off[m]);
    most = row_max(most);
    bool open = false;
#pragma unroll
    for (int m = 0; m < kRowGroups; ++m) open |= !KeyOf<float>::some(value[m]) && !(least[m] > most);   // (one that stays)
    sure = row_max(open && KeyOf<float>::some(most) ? 1u : 0u) == 0;
  }
  return stay;
}

// A sigmoid score with its bias in FP64.
template <int TYPE>
__device__ inline double sigmoid_value(const RouteArgs &a, const typename Elem<TYPE>::store *row, int e) {
  const double v = 1.0 / (1.0 + exp(-static_cast<double>(Elem<TYPE>::get(row[e]))));
  return a.bias ? v + static_cast<double>(a.bias[e]) : v;
}

// Where the estimates (in LDS) leave the groups open: the same from the FP64 values of the few
// experts of each group that may be among its two largest.
template <int TYPE>
__device__ unsigned long long settle_groups(const RouteArgs &a, const typename Elem<TYPE>::store *row, int l16,
                                            const float *keys, float error) {
  double value[kRowGroups];
#pragma unroll
  for (int m = 0; m < kRowGroups; ++m) value[m] = KeyOf<double>::none;
  const int size = a.group_size;
#pragma unroll 1
  for (int g = l16; g < a.groups; g += 16) {
    float first, second;
    group_top(a, g, l16, keys, first, second);
    const float last = a.group_top == 2 ? second : first, from = last - margin(error, last);
    double top[2] = {KeyOf<double>::none, KeyOf<double>::none};
#pragma unroll 1
    for (int e = g * size; e < g * size + size; ++e) {
      if (!KeyOf<float>::some(keys[e]) || keys[e] < from) continue;
      const double v = sigmoid_value<TYPE>(a, row, e);
      top[1] = v > top[0] ? top[0] : v > top[1] ? v : top[1];
      top[0] = v > top[0] ? v : top[0];
    }
#pragma unroll
    for (int m = 0; m < kRowGroups; ++m)
      if (m * 16 + l16 == g) value[m] = group_value(a, top[0], top[1]);
  }
  return choose_groups(a, value, l16);
}

// A row's keys to LDS.
template <int PER, class KEY>
__device__ inline const KEY *put_keys(const RouteArgs &a, const KEY (&key)[PER], int l16, void *lds) {
  KEY *keys = static_cast<KEY *>(lds);
  wave_order();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = expert_of(j, l16);
    if (e < a.experts) keys[e] = key[j];
  }
  wave_order();
  return keys;
}

// The choice: lane n's into `mine`, in descending order. Of float keys, where two that
// have to be told apart lie within their margin, `sure` is false, and the row's lanes
// have two more (up to 16) instead, `rest` being the best of the others.
template <int PER, class KEY>
__device__ inline int choose_experts(const RouteArgs &a, KEY (&key)[PER], int l16, float error, bool &sure, KEY &rest) {
  KEY best;
  int at;
  best_of<PER, KEY>(key, l16, best, at);
  int mine = -1;
  KEY last = KeyOf<KEY>::none;
  sure = true;
  for (int n = 0;; ++n) {
    const KEY most = row_max(best);
    if constexpr (KeyOf<KEY>::estimate) {
      // (not greater: also where both are infinite)
      if (n > 0 && n <= a.top_k && KeyOf<KEY>::some(most) && !(last - most > margin(error, fmaxf(fabsf(last), fabsf(most)))))
        sure = false;
      last = rest = most;
    }
    if (n >= a.top_k && (sure || n == min(a.top_k + 2, 16))) break;   // (rows differ: the lanes of one leave together)
    const int expert = row_min(best == most ? at : kRouteMaxExperts);
    if (l16 == n && KeyOf<KEY>::some(most)) mine = expert;
    if (expert == at && KeyOf<KEY>::some(best)) {   // its lane looks for its next
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (expert_of(j, l16) == expert) key[j] = KeyOf<KEY>::none;
      best_of<PER, KEY>(key, l16, best, at);
    }
  }
  return mine;
}

// The choice among candidates, one in each lane (-1: none), on their FP64 values. `sure` is
// false where an expert that is none of them may be among the best after all.
template <int TYPE>
__device__ int settle_experts(const RouteArgs &a, const typename Elem<TYPE>::store *row, int l16, int candidate,
                              float rest, float error, bool &sure) {
  const double v = candidate >= 0 ? sigmoid_value<TYPE>(a, row, candidate) : KeyOf<double>::none;
  const int number = candidate >= 0 ? candidate : kRouteMaxExperts + l16;
  int ahead = 0;
  for (int n = 0; n < 16; ++n) {
    const double w = row_lane(v, n);
    const int other = row_lane(number, n);
    ahead += w > v || (w == v && other < number) ? 1 : 0;
  }
  // to lane `ahead` of the row (all different)
  const int mine = __builtin_amdgcn_ds_permute(((threadIdx.x & 48) + ahead) * 4, candidate);
  const unsigned worst = row_max(ahead == a.top_k - 1 && !(v - static_cast<double>(rest) > margin(error, rest)) ? 1u : 0u);
  sure = !KeyOf<float>::some(rest) || worst == 0;
  return l16 < a.top_k ? mine : -1;
}

// Keys of experts whose group does not stay go.
template <int PER, class KEY>
__device__ inline void leave_groups(const RouteArgs &a, KEY (&key)[PER], int l16, unsigned long long stay) {
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const unsigned g = (static_cast<unsigned>(expert_of(j, l16)) * a.group_mul) >> 20;
    if (!(stay >> (g & 63) & 1)) key[j] = KeyOf<KEY>::none;
  }
}

// The FP64 values of all experts into LDS, and the groups that stay by them (all, without
// groups): where a few candidates do not settle the choice, and for softmax, whose values need
// the sum of all. Loops that are not unrolled: a launch waits for its slowest wave, and their
// instructions are quickly there.
template <int TYPE>
__device__ unsigned long long all_doubles(const RouteArgs &a, const typename Elem<TYPE>::store *row, float top, int l16,
                                          double *keys) {
  const double none = KeyOf<double>::none;
  double sum = 0.0;
  wave_order();
#pragma unroll 1
  for (int e = l16; e < a.experts; e += 16) {
    const float l = Elem<TYPE>::get(row[e]);
    double v = exp(a.score == kSoftmax ? static_cast<double>(l) - static_cast<double>(top) : -static_cast<double>(l));
    if (a.score == kSoftmax) sum += l == -__builtin_inff() ? 0.0 : v;
    else v = 1.0 / (1.0 + v);
    keys[e] = l == -__builtin_inff() ? none : v;
  }
  const double scale = a.score == kSoftmax ? row_total(sum) : 1.0;
#pragma unroll 1
  for (int e = l16; e < a.experts; e += 16) {
    double v = keys[e];
    if (v > none) {
      if (a.score == kSoftmax) v /= scale;
      if (a.bias) v += static_cast<double>(a.bias[e]);
      keys[e] = v;
    }
  }
  wave_order();
  if (a.groups == a.top_groups) return ~0ull;
  bool sure;
  return best_groups<double>(a, l16, keys, 0.0f, sure);
}

// The choice by them.
__device__ inline int choose_by_doubles(const RouteArgs &a, unsigned long long stay, int l16, double *keys) {
  const double none = KeyOf<double>::none;
#pragma unroll 1
  for (int e = l16; e < a.experts; e += 16)
    if (!(stay >> ((static_cast<unsigned>(e) * a.group_mul >> 20) & 63) & 1)) keys[e] = none;
  wave_order();
  int mine = -1;
#pragma unroll 1
  for (int n = 0; n < a.top_k; ++n) {
    double best = none;
    int at = kRouteMaxExperts;
#pragma unroll 4
    for (int e = l16; e < a.experts; e += 16) {
      const double v = keys[e];
      at = v > best ? e : at;
      best = v > best ? v : best;
    }
    const double most = row_max(best);
    const int expert = row_min(best == most ? at : kRouteMaxExperts);
    if (!(most > none)) break;   // (the row's lanes leave together)
    if (l16 == n) mine = expert;
    if ((expert & 15) == l16) keys[expert] = none;
    wave_order();
  }
  return mine;
}

// VALUES: the order of the logits does not settle the choice.
template <int TYPE, int PER, bool VALUES>
__device__ inline void route_token(const RouteArgs &a, long long t, int *counts, double *keys) {
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
  int mine = -1;
  if constexpr (!VALUES) {
    unsigned key[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) key[j] = l[j] == -__builtin_inff() ? 0u : logit_key(l[j]);
    bool sure;
    if (a.groups > a.top_groups)
      leave_groups<PER, unsigned>(a, key, l16, best_groups<unsigned>(a, l16, put_keys<PER>(a, key, l16, keys), 0.0f, sure));
    unsigned rest;
    mine = choose_experts<PER, unsigned>(a, key, l16, 0.0f, sure, rest);
  } else {
    // Estimates. e^-l by v_exp_f32 is off by (|l| + 1) 2^-23 of itself (the argument's rounding, its
    // own), a sigmoid by s (1 - s) of that, which is below 2^-24 for both terms together with
    // |l| s (1 - s) < 0.23; 1 + e^-l and the reciprocal add 2^-24 + 2^-23: within 2^-22, taken
    // twice. A softmax: |x| e^x < 0.37, a product, a sum of up to 36 terms: within 2^-18 of the
    // largest, taken twice. (Adding the bias: margin.)
    float key[PER], bias[PER], sum = 0.0f;
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < PER; j += 4) load_logits<kF32>(a.bias, expert_of(j, l16), a.experts, &bias[j]);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) bias[j] = 0.0f;
    }
    bool nan = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (a.score == kSoftmax) {
        key[j] = __expf(l[j] - top);
        sum += key[j];
      } else {
        key[j] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[j]));
      }
    }
    float error = 0x1p-21f;
    if (a.score == kSoftmax) {
      const float inverse = 1.0f / row_total(sum);
      error = 0x1p-17f * inverse;
#pragma unroll
      for (int j = 0; j < PER; ++j) key[j] *= inverse;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      nan |= bias[j] != bias[j];
      key[j] = l[j] == -__builtin_inff() ? KeyOf<float>::none : key[j] + bias[j];
    }
    bad |= row_max(nan ? 1u : 0u) != 0;
    if (a.groups > a.top_groups) {
      bool apart;
      const float *in_lds = put_keys<PER>(a, key, l16, keys);
      unsigned long long stay = best_groups<float>(a, l16, in_lds, error, apart);
      if (!apart && !bad)   // (a row's lanes go together)
        stay = a.score == kSigmoid ? settle_groups<TYPE>(a, row, l16, in_lds, error) : all_doubles<TYPE>(a, row, top, l16, keys);
      leave_groups<PER, float>(a, key, l16, stay);
    }
    if (!a.bias) {   // the groups are settled: the logits say the rest
      unsigned order[PER], rest;
#pragma unroll
      for (int j = 0; j < PER; ++j) order[j] = KeyOf<float>::some(key[j]) ? logit_key(l[j]) : 0u;
      bool exact;
      mine = choose_experts<PER, unsigned>(a, order, l16, 0.0f, exact, rest);
    } else {
      float rest;
      bool sure;
      mine = choose_experts<PER, float>(a, key, l16, error, sure, rest);
      if (!sure && !bad && a.score == kSigmoid) mine = settle_experts<TYPE>(a, row, l16, mine, rest, error, sure);
      if (!sure && !bad) mine = choose_by_doubles(a, all_doubles<TYPE>(a, row, top, l16, keys), l16, keys);
    }
  }
  if (bad) mine = -1;
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
// Bound by a wave's chain of maxima, or with many tokens by its instructions: 65536 tokens on 4 of 64
// experts 11 us by logits, 19 by values with a bias (16.8 MB read); 4096 on 8 of 256 7 and 10,
// in groups 13, and 19 where some token needs FP64 values; one token 4.4. Counts add 2 to 7.
template <int TYPE, int PER, bool VALUES, int THREADS>
__global__ __launch_bounds__(THREADS) void route_kernel(RouteArgs a) {
  __shared__ int counts[kRouteMaxExperts];
  extern __shared__ __attribute__((aligned(16))) unsigned char dynamic[];   // a key for each row's experts, with groups
  if (a.counts) {
    for (int e = threadIdx.x; e < a.experts; e += THREADS) counts[e] = 0;
    __syncthreads();
  }
  const int row = threadIdx.x >> 4;
  double *keys = reinterpret_cast<double *>(dynamic + row * a.row_bytes);
  const long long rows = static_cast<long long>(gridDim.x) * (THREADS / 16);
  for (long long t = static_cast<long long>(blockIdx.x) * (THREADS / 16) + row; t < a.tokens; t += rows)
    route_token<TYPE, PER, VALUES>(a, t, a.counts ? counts : nullptr, keys);
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
// 65536 tokens on 4 of 64 experts (16.8 MB written) 9 us, 4096 on 8 of 256 in bfloat16 4.6.
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
