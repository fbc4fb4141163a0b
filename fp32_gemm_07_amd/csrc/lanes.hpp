// Sums and maxima across the lanes of a row of 16 and of a wave (DPP).
#pragma once

#include <hip/hip_runtime.h>

namespace gemm {
namespace mx {

template <int CTRL, int ROWS>
__device__ inline int dpp(int identity, int v) {
  return __builtin_amdgcn_update_dpp(identity, v, CTRL, ROWS, 0xf, false);
}
// v of the lane N further on in its row of 16 (0 past the row).
template <int N>
__device__ inline float from_lane(float v) {
  return __builtin_bit_cast(float, dpp<0x100 + N, 0xf>(0, __builtin_bit_cast(int, v)));
}
// op over the 16 lanes of a row (rotations by 1, 2, 4, 8), in every lane.
template <class OP>
__device__ inline int row_all(int v, OP &&op) {
  v = op(v, dpp<0x121, 0xf>(0, v));
  v = op(v, dpp<0x122, 0xf>(0, v));
  v = op(v, dpp<0x124, 0xf>(0, v));
  return op(v, dpp<0x128, 0xf>(0, v));
}
__device__ inline unsigned row_max(unsigned v) {
  return static_cast<unsigned>(row_all(static_cast<int>(v), [](int a, int b) {
    return static_cast<int>(max(static_cast<unsigned>(a), static_cast<unsigned>(b)));
  }));
}
__device__ inline int row_min(int v) {
  return row_all(v, [](int a, int b) { return min(a, b); });
}
__device__ inline float row_sum(float v) {
  return __builtin_bit_cast(float, row_all(__builtin_bit_cast(int, v), [](int a, int b) {
    return __builtin_bit_cast(int, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }));
}
// Running sums over a wave: shifts within rows, then the last lane of each row
// and of the first half handed on (row_bcast 15, 31).
__device__ inline int wave_running_sum(int v) {
  v += dpp<0x111, 0xf>(0, v);
  v += dpp<0x112, 0xf>(0, v);
  v += dpp<0x114, 0xf>(0, v);
  v += dpp<0x118, 0xf>(0, v);
  v += dpp<0x142, 0xa>(0, v);
  return v + dpp<0x143, 0xc>(0, v);
}

}  // namespace mx
}  // namespace gemm
