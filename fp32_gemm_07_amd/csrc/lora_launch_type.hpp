// The launches of one element type; included by that type's translation unit alone.
#pragma once

#include "lora_launch.hpp"

namespace gemm {
namespace mx {

template <class F>
void with_rank(int rank, F &&f) {
  switch (rank_tiles(rank)) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    default: f(std::integral_constant<int, 8>()); break;
  }
}

template <int TYPE>
int launch_shrink(ShrinkArgs a, int problems, const ShrinkPlan &plan, hipStream_t stream) {
  a.units_by = plan.units_by;
  const long long units = host::ceil_div(a.r.rows, 64) * a.units_by;
  a.blocks0 = static_cast<int>(units * a.p[0].splits);
  const dim3 blocks(static_cast<unsigned>(a.blocks0 + (problems > 1 ? units * a.p[1].splits : 0)));
  with_rank(a.r.rank, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    if constexpr (RT < 8) {
      if (plan.waves == 8) {
        hipLaunchKernelGGL((shrink_kernel<TYPE, RT, 1, 8>), blocks, dim3(512), 0, stream, a);
        return;
      }
    }
    if (plan.tiles == 2) hipLaunchKernelGGL((shrink_kernel<TYPE, RT, 2, 4>), blocks, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((shrink_kernel<TYPE, RT, 1, 4>), blocks, dim3(256), 0, stream, a);
  });
  return host::launched();
}

template <int TYPE, int RT, int J, bool SUM>
void launch_expand_columns(ExpandArgs a, int cus, hipStream_t stream) {
  const long long columns = host::ceil_div(a.N, 64 * J), windows = host::ceil_div(a.r.rows, 64);
  // Two workgroups a CU, then more windows for each: an adapter's columns stay in registers, and
  // loads ahead. (8192 x 4096 bfloat16, rank 16: 4 windows 31 us, 2 33, 1 36, 8 37.)
  // With fewer, the units of a window are dealt out among several.
  a.windows = static_cast<int>(std::max<long long>(1, columns * windows / (2LL * cus)));
  const long long blocks = columns * host::ceil_div(windows, a.windows);
  a.units_by = static_cast<int>(std::max<long long>(1, std::min<long long>({2LL * cus / blocks, a.r.rows, SUM ? 64 : 8})));
  hipLaunchKernelGGL((expand_kernel<TYPE, RT, J, SUM>), dim3(static_cast<unsigned>(blocks * a.units_by)), dim3(256), 0,
                     stream, a);
}
template <int TYPE>
int launch_expand(const ExpandArgs &a, bool few, int cus, hipStream_t stream) {
  with_rank(a.r.rank, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    if (!few) launch_expand_columns<TYPE, RT, 4, false>(a, cus, stream);
    else if (host::ceil_div(a.N, 256) * a.r.rows < cus) launch_expand_columns<TYPE, RT, 1, true>(a, cus, stream);
    else launch_expand_columns<TYPE, RT, 4, true>(a, cus, stream);
  });
  return host::launched();
}

template <int TYPE>
int launch_small(const SmallArgs &a, hipStream_t stream) {
  const dim3 blocks(static_cast<unsigned>(host::ceil_div(a.N, kSmallCols) * a.units_by));
  if (a.r.rank <= 16) hipLaunchKernelGGL((small_kernel<TYPE, 1>), blocks, dim3(64 * kSmallWaves), 0, stream, a);
  else hipLaunchKernelGGL((small_kernel<TYPE, 2>), blocks, dim3(64 * kSmallWaves), 0, stream, a);
  return host::launched();
}

template <int TYPE>
int launch_prepare(const PrepareArgs &a, int blocks, hipStream_t stream) {
  hipLaunchKernelGGL(prepare_kernel<TYPE>, dim3(static_cast<unsigned>(blocks)), dim3(1024), 0, stream, a);
  return host::launched();
}

template <int TYPE>
int launch_grads(GradArgs a, int most_slots, hipStream_t stream) {
  const long long slot_blocks = static_cast<long long>(a.blocks) * a.rank_blocks;
  return host::in_ranges(most_slots, host::max_blocks(256) / slot_blocks, [&](long long slot0, int count) {
    a.slot0 = static_cast<int>(slot0);
    with_rank(std::min(a.r.rank, 64), [&](auto rt) {
      if constexpr (decltype(rt)::value <= 4)
        hipLaunchKernelGGL((grad_kernel<TYPE, decltype(rt)::value>), dim3(static_cast<unsigned>(count * slot_blocks)),
                           dim3(256), 0, stream, a);
    });
    return host::launched();
  });
}

template <int TYPE>
int launch_sum(const GradSumArgs &a, int blocks, hipStream_t stream) {
  hipLaunchKernelGGL(grad_sum_kernel<TYPE>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, a);
  return host::launched();
}

template <int TYPE>
const LoraLaunches &launches_of() {
  static const LoraLaunches l{launch_shrink<TYPE>, launch_expand<TYPE>, launch_small<TYPE>, launch_prepare<TYPE>, launch_grads<TYPE>,
                              launch_sum<TYPE>};
  return l;
}

}  // namespace mx
}  // namespace gemm
