// Launches of the low-rank adapters' kernels. Each element type's are compiled in a translation
// unit of their own (lora_f32.hip, lora_bf16.hip, lora_f16.hip): there are many, and so they
// compile side by side.
#pragma once

#include "host_checks.hpp"
#include "lora_kernels.hpp"

namespace gemm {
namespace mx {

// How shrink is launched (shrink_plan in gemm_lora.hip says which, when and why).
struct ShrinkPlan {
  int tiles, waves, units_by, splits;
  bool few;
};

struct LoraLaunches {
  // The first one or two of a.p; fills in units_by and blocks0.
  int (*shrink)(ShrinkArgs a, int problems, const ShrinkPlan &plan, hipStream_t stream);
  // Fills in windows and units_by.
  int (*expand)(const ExpandArgs &a, bool few, int cus, hipStream_t stream);
  int (*small)(const SmallArgs &a, hipStream_t stream);
  int (*prepare)(const PrepareArgs &a, int blocks, hipStream_t stream);
  int (*grads)(GradArgs a, int most_slots, hipStream_t stream);
  int (*sum)(const GradSumArgs &a, int blocks, hipStream_t stream);
};
const LoraLaunches &lora_launches_f32();
const LoraLaunches &lora_launches_bf16();
const LoraLaunches &lora_launches_f16();

// 16-column tiles of H for a rank: 1, 2, 4 or 8.
inline int rank_tiles(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

}  // namespace mx
}  // namespace gemm
