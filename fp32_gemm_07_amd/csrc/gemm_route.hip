// The gemm_route* entry points (declared and documented in gemm.h): argument checks,
// choice of kernel, launches.
#include "gemm.h"

#include "host_checks.hpp"
#include "host_shared.hpp"
#include "route_kernels.hpp"

namespace {

using namespace gemm::mx;
using namespace gemm::host;

static_assert(kRouteMaxExperts == GEMM_ROUTE_MAX_EXPERTS && kRouteMaxTopK == GEMM_ROUTE_MAX_TOP_K &&
                  kRouteMaxGroups == GEMM_ROUTE_MAX_GROUPS && kSoftmax == GEMM_ROUTE_SOFTMAX &&
                  kSigmoid == GEMM_ROUTE_SIGMOID,
              "router limits");

int check_router(int tokens, const gemm_route_t *r, int type, int ld) {
  if (!r) return GEMM_ERR_NULL_PTR;
  if (tokens < 0 || r->experts < 1 || r->experts > kRouteMaxExperts || r->top_k < 1 || r->top_k > kRouteMaxTopK ||
      r->groups < 1 || r->groups > kRouteMaxGroups || r->experts % r->groups != 0 || r->top_groups < 1 ||
      r->top_groups > r->groups || r->group_top < 1 || r->group_top > 2 ||
      r->top_k > r->experts / r->groups * r->top_groups || ld < r->experts ||
      static_cast<long long>(tokens) * ld > kMaxElements)
    return GEMM_ERR_INVALID_DIM;
  if (!valid_type(type) || (r->score != kSoftmax && r->score != kSigmoid)) return GEMM_ERR_INVALID_TYPE;
  return GEMM_OK;
}

// Calls f with the experts that a lane of a row of 16 holds.
template <class F>
void with_experts(int experts, F &&f) {
  if (experts <= 64) f(std::integral_constant<int, 4>());
  else if (experts <= 128) f(std::integral_constant<int, 8>());
  else if (experts <= 256) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 32>());
}

template <int TYPE, int PER, bool VALUES>
int launch_route(RouteArgs a, int cus, hipStream_t stream) {
  // LDS for a row's keys: doubles, or whole numbers where groups are chosen.
  const size_t row_keys = VALUES ? 8 * static_cast<size_t>(a.experts) : a.groups > a.top_groups ? 4 * static_cast<size_t>(a.experts + a.experts % 2) : 0;
  a.row_bytes = static_cast<int>(row_keys);
  // Few tokens: one workgroup, which needs no counts zeroed by a launch before it.
  // (Of fewer waves where a lane holds more experts: their values take its registers.)
  constexpr int kOne = PER <= (VALUES ? 4 : 8) ? 1024 : PER <= 16 ? 512 : 256;
  if (a.counts && a.tokens <= 64) {
    hipLaunchKernelGGL((route_kernel<TYPE, PER, VALUES, kOne>), dim3(1), dim3(kOne), row_keys * (kOne / 16), stream, a);
    return launched();
  }
  if (a.counts) {
    hipLaunchKernelGGL(zero_counts_kernel, dim3(1), dim3(512), 0, stream, a.counts, a.experts);
    const int st = launched();
    if (st != GEMM_OK) return st;
  }
  // Each workgroup adds its counts to the same few words, which takes some 15 ns each: no more
  // than one a CU (65536 tokens on 64 experts: 256 of 1024 threads 24 us, 2048 of 256 48).
  const long long blocks = ceil_div(a.tokens, 16);
  if (a.counts && blocks > cus) {
    hipLaunchKernelGGL((route_kernel<TYPE, PER, VALUES, kOne>),
                       dim3(static_cast<unsigned>(std::min<long long>(ceil_div(a.tokens, kOne / 16), cus))), dim3(kOne),
                       row_keys * (kOne / 16), stream, a);
  } else {
    hipLaunchKernelGGL((route_kernel<TYPE, PER, VALUES, 256>), dim3(static_cast<unsigned>(std::min(blocks, 8LL * cus))),
                       dim3(256), row_keys * 16, stream, a);
  }
  return launched();
}

}  // namespace

extern "C" {

int gemm_route(int tokens, const gemm_route_t *router, const void *logits, int logits_type,
               int ld_logits, const float *bias, int *chosen, float *weights, int *counts,
               hipStream_t stream) {
  int st = check_router(tokens, router, logits_type, ld_logits);
  if (st != GEMM_OK) return st;
  const gemm_route_t &r = *router;
  const size_t choices = 4 * static_cast<size_t>(tokens) * r.top_k;
  const Range in[] = {{logits, extent(tokens, r.experts, ld_logits, logits_type)},
                      {bias, bias ? 4 * static_cast<size_t>(r.experts) : 0}};
  const Range out[] = {{chosen, choices}, {weights, choices}, {counts, counts ? 4 * static_cast<size_t>(r.experts) : 0}};
  if (tokens > 0 && (!logits || !chosen || !weights)) return GEMM_ERR_NULL_PTR;
  if (!aligned(logits, elem_size(logits_type)) || !aligned(bias, 4) || !aligned(chosen, 4) || !aligned(weights, 4) ||
      !aligned(counts, 4))
    return GEMM_ERR_ALIGNMENT;
  st = check_outputs(out, in);
  if (st != GEMM_OK || (tokens == 0 && !counts)) return st;
  int dev = 0, cus = 0;
  st = gemm::host_check_device(&dev, &cus);
  if (st != GEMM_OK) return st;
  const int size = r.experts / r.groups;
  const RouteArgs a{tokens, r.experts, r.top_k, r.score, r.groups, r.top_groups, r.group_top, r.renormalize != 0,
                    r.scale, logits, ld_logits, bias, chosen, weights, counts,
                    static_cast<unsigned>(ceil_div(1 << 20, size)), size, 0};
  // Scores are computed where the order of the logits does not settle the choice.
  const bool values = bias || (r.top_groups < r.groups && r.group_top == 2 && size > 1);
  with_type(logits_type, [&](auto t) {
    with_experts(r.experts, [&](auto per) {
      constexpr int T = decltype(t)::value, PER = decltype(per)::value;
      st = values ? launch_route<T, PER, true>(a, cus, stream) : launch_route<T, PER, false>(a, cus, stream);
    });
  });
  return st;
}

int gemm_route_backward(int tokens, const gemm_route_t *router, const void *logits,
                        int logits_type, int ld_logits, const int *chosen, const float *dweights,
                        void *dlogits, int ld_dlogits, hipStream_t stream) {
  int st = check_router(tokens, router, logits_type, ld_logits);
  if (st != GEMM_OK) return st;
  const gemm_route_t &r = *router;
  if (ld_dlogits < r.experts || static_cast<long long>(tokens) * ld_dlogits > kMaxElements) return GEMM_ERR_INVALID_DIM;
  if (tokens == 0) return GEMM_OK;
  if (!logits || !chosen || !dweights || !dlogits) return GEMM_ERR_NULL_PTR;
  if (!aligned(logits, elem_size(logits_type)) || !aligned(dlogits, elem_size(logits_type)) || !aligned(chosen, 4) ||
      !aligned(dweights, 4))
    return GEMM_ERR_ALIGNMENT;
  const size_t choices = 4 * static_cast<size_t>(tokens) * r.top_k;
  const Range in[] = {{logits, extent(tokens, r.experts, ld_logits, logits_type)}, {chosen, choices}, {dweights, choices}};
  const Range out[] = {{dlogits, extent(tokens, r.experts, ld_dlogits, logits_type)}};
  st = check_outputs(out, in);
  if (st != GEMM_OK) return st;
  int dev = 0, cus = 0;
  st = gemm::host_check_device(&dev, &cus);
  if (st != GEMM_OK) return st;
  const RouteGradArgs a{tokens, r.experts, r.top_k, r.score, r.renormalize != 0, r.scale, logits, ld_logits,
                        chosen, dweights, dlogits, ld_dlogits};
  with_type(logits_type, [&](auto t) {
    with_experts(r.experts, [&](auto per) {
      hipLaunchKernelGGL((route_grad_kernel<decltype(t)::value, decltype(per)::value>),
                         dim3(static_cast<unsigned>(std::min<long long>(ceil_div(tokens, 16), 16LL * cus))), dim3(256), 0,
                         stream, a);
    });
  });
  return launched();
}

}  // extern "C"
