// Checks of arguments and helpers for launches that the entry points on typed float
// matrices share.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "elem.hpp"
#include "gemm.h"
#include "host_shared.hpp"

namespace gemm {
namespace host {

using mx::kBf16;
using mx::kF16;
using mx::kF32;

constexpr long long kMaxElements = 1LL << 40;

inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
inline bool valid_type(int t) { return t == kF32 || t == kBf16 || t == kF16; }
inline size_t elem_size(int t) { return t == kF32 ? 4 : 2; }
inline bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Bytes from the first to the last element of a stored matrix.
inline size_t extent(long long rows, long long cols, long long ld, int type) {
  return rows > 0 && cols > 0 ? elem_size(type) * static_cast<size_t>((rows - 1) * ld + cols) : 0;
}

inline int launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? GEMM_OK : gemm::host_fail(e);
}

// A launch takes fewer than 2^32 threads, so at most this many workgroups.
constexpr long long max_blocks(long long threads) { return ((1LL << 32) - 1) / threads; }

// launch(at, count), which returns a status, for successive ranges of at most `most`
// of `total`.
template <class F>
int in_ranges(long long total, long long most, F &&launch) {
  int st = GEMM_OK;
  for (long long at = 0; at < total && st == GEMM_OK; at += most)
    st = launch(at, static_cast<int>(std::min(most, total - at)));
  return st;
}

// Calls f.template operator()<TYPE>() for a valid element type.
template <class F>
void with_type(int type, F &&f) {
  switch (type) {
    case kF32: f(std::integral_constant<int, kF32>()); break;
    case kBf16: f(std::integral_constant<int, kBf16>()); break;
    default: f(std::integral_constant<int, kF16>()); break;
  }
}

// A range that a call reads or writes.
struct Range {
  const void *p;
  size_t bytes;
};

// Outputs, each apart from the others and from every input.
template <size_t OUT, size_t IN>
int check_outputs(const Range (&out)[OUT], const Range (&in)[IN]) {
  for (size_t i = 0; i < OUT; ++i) {
    for (const Range &r : in)
      if (gemm::host_overlaps(out[i].p, out[i].bytes, r.p, r.bytes)) return GEMM_ERR_ALIAS;
    for (size_t j = 0; j < i; ++j)
      if (gemm::host_overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return GEMM_ERR_ALIAS;
  }
  return GEMM_OK;
}

// A caller's workspace (null: the library's) of `need` bytes: large enough,
// aligned, and apart from everything else that the call touches.
inline int check_workspace(const void *workspace, size_t bytes, size_t need, std::initializer_list<Range> others) {
  if (!workspace || need == 0) return GEMM_OK;
  if (bytes < need) return GEMM_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return GEMM_ERR_ALIGNMENT;
  for (const Range &r : others)
    if (gemm::host_overlaps(workspace, need, r.p, r.bytes)) return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

}  // namespace host
}  // namespace gemm
