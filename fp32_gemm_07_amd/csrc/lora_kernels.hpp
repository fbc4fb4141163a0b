// Low-rank adapters beside a shared projection: every row of X has an adapter of its own
// (the operations are described in gemm.h at gemm_lora and gemm_lora_backward).
//   shrink:  H = s X A^T          rows x rank, FP32
//   expand:  Y = C + H B^T
// and backward, with A and B transposed first (few bytes) so that both serve again:
//   shrink:  H = s X A^T,  G = s dY B
//   expand:  dX = C' + G A
//   grads:   dA = G^T X,  dB = dY^T H, sums over the rows of one adapter.
// A rank is far below the balance of the matrix units, so all of these are bound by the
// bytes of X, C and Y (dY, dX): each is read or written once a kernel, straight
// between memory and registers. What is small (adapters, H, G) comes from L2.
//
// Rows are looked at 64 at a time (a window: a lane each). Those of one adapter, up to 16
// or some times 16, make a unit, wherever they lie in the window: they are the columns of
// 16x16 matrix instructions, so an adapter is read once for all of its rows there, be they
// a prompt's or single tokens between those of other requests. An instruction's columns do
// not mix: what another row or adapter holds, NaN included, never reaches a row.
//
// Precision: products of 16-bit inputs are exact and summed in FP32. H and G stay FP32:
// they enter the second products as three bfloat16 parts whose sum is exact. FP32
// inputs go through FP32 matrix instructions throughout.
#pragma once

#include <type_traits>

#include "gemm_kernels.hpp"
#include "mx_moe.hpp"

namespace gemm {
namespace mx {

constexpr int kLoraMaxRank = 128, kLoraMaxAdapters = 1024;   // GEMM_LORA_MAX_*

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// What every kernel knows of the adapters: each row's, its rank and its scale.
struct LoraRows {
  int rows, rank, adapters;
  const int *ids;
  const int *ranks;      // null: all `rank`
  const float *scales;   // null: all 1
  // A row's adapter, -1: none. (For rows past the last: the last one's.)
  __device__ inline int load_id(int row) const { return ids[min(row, rows - 1)]; }
  __device__ inline int id_of(int loaded) const { return loaded >= 0 && loaded < adapters ? loaded : -1; }
  __device__ inline int rank_of(int a) const { return ranks ? max(0, min(rank, ranks[a])) : rank; }
};

// 16 bytes of a row as an operand of a matrix instruction: 8 values of 16 bits (k = 8g ..
// 8g + 7 of 32), or 4 floats, one for each of 4 instructions (k = 4g .. 4g + 3 of 16).
template <int TYPE>
constexpr int kLaneK = TYPE == kF32 ? 4 : 8;

template <int TYPE>
__device__ inline uintx4 load_k(const typename Elem<TYPE>::store *p) {
  return *reinterpret_cast<const uintx4_any *>(p);
}
// The same at a row's end: `left` values (may be negative), zeros behind them. (All loads at
// once, then the choice: one after the other each would be waited for.)
template <int TYPE>
__device__ inline uintx4 load_k(const typename Elem<TYPE>::store *p, int left) {
  if (left >= kLaneK<TYPE>) return load_k<TYPE>(p);
  uintx4 v = {};
  if (left > 0) {
    typename Elem<TYPE>::store x[kLaneK<TYPE>];
#pragma unroll
    for (int i = 0; i < kLaneK<TYPE>; ++i) x[i] = p[min(i, left - 1)];
#pragma unroll
    for (int i = 0; i < kLaneK<TYPE>; ++i) {
      if constexpr (TYPE == kF32) v[i] = i < left ? __builtin_bit_cast(unsigned, x[i]) : 0u;
      else v[i / 2] |= i < left ? static_cast<unsigned>(x[i]) << (16 * (i % 2)) : 0u;
    }
  }
  return v;
}
template <int TYPE>
__device__ inline f32x4 multiply(const uintx4 &a, const uintx4 &b, f32x4 acc) {
  if constexpr (TYPE == kBf16) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else if constexpr (TYPE == kF16) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned x = a[i], y = b[i];
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y), acc, 0, 0, 0);
    }
  }
  return acc;
}

// 8 floats, 4 to a register quad, as operands of a kind that multiplies them with TYPE.
__device__ inline void floats8(const f32x4 &a, const f32x4 &b, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
// 8 halfs as two bfloat16 parts (exact: 11 bits in 8 and 8).
__device__ inline void split_halfs(const uintx4 &h, bf16x8 (&out)[2]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned w = h[i];
    v[2 * i] = Elem<kF16>::get(static_cast<u16>(w));
    v[2 * i + 1] = Elem<kF16>::get(static_cast<u16>(w >> 16));
  }
  split8<2>(v, out);
}

// n > 0 batches through two sets of registers: fetch(set) loads the next batch, use(set) works
// on one that is there.
template <class S, class F, class G>
__device__ inline void two_deep(int n, S &even, S &odd, F &&fetch, G &&use) {
  fetch(even);
  for (; n > 2; n -= 2) {
    fetch(odd);
    __builtin_amdgcn_sched_barrier(0);
    use(even);
    fetch(even);
    __builtin_amdgcn_sched_barrier(0);
    use(odd);
  }
  if (n == 2) {
    fetch(odd);
    __builtin_amdgcn_sched_barrier(0);
    use(even);
    use(odd);
  } else {
    use(even);
  }
}

// The units of a range of windows in order: rows of one adapter (of none for id -1, where those
// count too), up to 16 MT of them. Everything but `row` is uniform over the wave.
template <int MT>
struct Units {
  const LoraRows &r;
  const bool with_none;      // rows without an adapter make units too
  int window, end;
  int my_id;                 // of this lane's row in the window (-2: past the last row)
  int next_id;               // of its row in the next one, as loaded: on its way meanwhile
  unsigned long long todo = 0, same = 0, mask;
  int base = 0, first;
  // The current unit.
  int id;
  int row[MT];               // of column i16; rows - 1 past the unit's last
  bool real[MT];

  __device__ inline Units(const LoraRows &rows, bool none, int first, int last)
      : r(rows), with_none(none), window(first - 1), end(last) {
    next_id = r.load_id(first * 64 + (threadIdx.x & 63));
  }
  // The next unit, without its rows: a window of many units is stepped through by workgroups that
  // want few of them (64 rows on 64 adapters of 1024 x 1024, rank 8: 29 us with the rows of each).
  __device__ inline bool step() {
    if (!same) {
      while (!todo) {
        if (++window >= end) return false;
        const int at = window * 64 + (threadIdx.x & 63);
        my_id = at < r.rows ? r.id_of(next_id) : -2;
        next_id = r.load_id(at + 64);
        todo = __ballot(with_none ? my_id >= -1 : my_id >= 0);
      }
      id = __builtin_amdgcn_readlane(my_id, __builtin_ctzll(todo));
      same = __ballot(my_id == id);
      todo &= ~same;
      base = 0;
    }
    mask = same;
    first = base;
    base += 16 * MT;
    if (base >= __popcll(same)) same = 0;
    return true;
  }
  // Its rows.
  __device__ inline void rows() {
    const int lane = threadIdx.x & 63, i16 = lane & 15;
    if (mask == ~0ull) {   // the whole window: row by row
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        real[m] = true;
        row[m] = window * 64 + first + m * 16 + i16;
      }
      return;
    }
    // Lane l's row of the window goes to the lane of its number among the unit's.
    const int count = __popcll(mask);
    const int number = __popcll(mask & ((1ull << lane) - 1)) - first;
    const bool mine = (mask >> lane & 1) && number >= 0 && number < 64;
    const int from = __builtin_amdgcn_ds_permute((mine ? number : 63) * 4, mine ? lane : 0);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      real[m] = m * 16 + i16 < count - first;
      const int at = window * 64 + __shfl(from, m * 16 + i16);
      row[m] = real[m] ? at : r.rows - 1;
    }
  }
};

// ---------------------------------------------------------------------------
// shrink.
struct Shrink {
  const void *z;       // rows x K
  long long ldz;
  const void *w;       // adapter a's rank x K at w + a * w_adapter, row stride ldw
  long long w_adapter, ldw;
  int K, k_split;      // columns of a workgroup's range, a multiple of 64
  int splits;
  void *h;             // for expand, or null: [rows][3][RP] bfloat16 parts; for FP32 or where
  bool floats;         // expand is to sum over ranges [split][rows][RP] floats
  void *parts;         // for the gradients, or null: [3][RP][positions] bfloat16 parts, for FP32 [RP][positions] floats
};
struct ShrinkArgs {
  LoraRows r;
  Shrink p[2];         // blocks of p[0] first
  int blocks0, units_by;
  const int *position; // of each row among the rows sorted by adapter (with parts)
  int positions;
};

// One workgroup: every units_by-th unit of a window, over a range of K that its W waves share;
// their sums are added in order through LDS. A wave's operands of the next U chunks are
// on their way while those of the last are multiplied.
// Bound by memory: 8192 x 4096 bfloat16 (67 MB), rank 16, 18 us by itself (3.8 TB/s), 29 behind an
// expand whose 67 MB are still on their way out; rank 32, two of them (backward) 53.
template <int TYPE, int RT, int MT, int W>
__global__ __launch_bounds__(64 * W) void shrink_kernel(ShrinkArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int RP = 16 * RT, kLane = kLaneK<TYPE>, kChunk = 4 * kLane;
  constexpr int U = RT + MT > 8 ? 1 : RT + MT > 3 ? 2 : 4;   // chunks at a time
  __shared__ __attribute__((aligned(16))) f32x4 sums[2][W * MT * RT * 64];
  const bool second = static_cast<int>(blockIdx.x) >= a.blocks0;
  const Shrink p = second ? a.p[1] : a.p[0];
  int block = second ? blockIdx.x - a.blocks0 : blockIdx.x;
  const int split = block % p.splits;
  block /= p.splits;
  // (Workgroups that a window has no unit for come last: dealt out between the others they
  // would leave whole XCDs idle.)
  const int windows = (a.r.rows + 63) / 64, group = block / windows, window = block - group * windows;
  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k_wave = (p.k_split / W + 63) / 64 * 64;
  const int k1 = min(p.K, (split + 1) * p.k_split);
  const int ka = min(k1, split * p.k_split + wave * k_wave), kb = wave == W - 1 ? k1 : min(k1, ka + k_wave);

  Units<MT> unit(a.r, false, window, window + 1);
  int turn = 0;
  int skip = group;   // units of other workgroups before the next of this one's
  while (unit.step()) {
    if (skip-- > 0) continue;
    skip = a.units_by - 1;
    unit.rows();
    // (The adapter's own rank comes in at the end alone, so that no load waits for it.)
    const int id = unit.id, rank = a.r.rank_of(id);
    const float scale = a.r.scales ? a.r.scales[id] : 1.0f;
    f32x4 acc[MT][RT] = {};
    {
      const store *w = static_cast<const store *>(p.w) + id * p.w_adapter + g * kLane;
      const store *wr[RT], *zr[MT];
#pragma unroll
      for (int t = 0; t < RT; ++t) wr[t] = w + min(t * 16 + i16, a.r.rank - 1) * p.ldw;   // (past the rank: not kept)
#pragma unroll
      for (int m = 0; m < MT; ++m) zr[m] = static_cast<const store *>(p.z) + unit.row[m] * p.ldz + g * kLane;
      struct Fetched {
        uintx4 w[U][RT], z[U][MT];
      };
      int k = ka, next = ka;
      auto fetch = [&](Fetched &f) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int m = 0; m < MT; ++m) f.z[u][m] = load_k<TYPE>(zr[m] + next + u * kChunk);
#pragma unroll
          for (int t = 0; t < RT; ++t) f.w[u][t] = load_k<TYPE>(wr[t] + next + u * kChunk);
        }
        next += U * kChunk;
      };
      auto use = [&](const Fetched &f) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[m][t] = multiply<TYPE>(f.w[u][t], f.z[u][m], acc[m][t]);
      };
      const int batches = (kb - ka) / (U * kChunk);
      if (batches > 0) {
        Fetched even, odd;
        two_deep(batches, even, odd, fetch, use);
        k += batches * (U * kChunk);
      }
      for (; k < kb; k += kChunk) {
        const int rest = kb - k - g * kLane;
        uintx4 wv[RT], zv[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) zv[m] = load_k<TYPE>(zr[m] + k, rest);
#pragma unroll
        for (int t = 0; t < RT; ++t) wv[t] = load_k<TYPE>(wr[t] + k, rest);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[m][t] = multiply<TYPE>(wv[t], zv[m], acc[m][t]);
      }
    }
    // One barrier a unit: the next one's sums go to the other half.
    f32x4 *half = sums[turn & 1];
    ++turn;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < RT; ++t) half[((wave * MT + m) * RT + t) * 64 + lane] = acc[m][t];
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if ((m * RT + t) % W != wave) continue;
        f32x4 v = half[(m * RT + t) * 64 + lane];
#pragma unroll
        for (int s = 1; s < W; ++s) v += half[((s * MT + m) * RT + t) * 64 + lane];
        // 4 neighbouring columns of H for one row, scaled, zeros past the rank
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = t * 16 + 4 * g + i < rank ? v[i] * scale : 0.0f;
        const int row = unit.row[m];
        if (!unit.real[m]) continue;
        if (p.h && (TYPE == kF32 || p.floats))
          *reinterpret_cast<f32x4 *>(static_cast<float *>(p.h) + (static_cast<long long>(split) * a.r.rows + row) * RP +
                                     t * 16 + 4 * g) = v;
        const int at = p.parts ? a.position[row] : 0;
        if constexpr (TYPE == kF32) {
          if (p.parts) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              static_cast<float *>(p.parts)[static_cast<long long>(t * 16 + 4 * g + i) * a.positions + at] = v[i];
          }
        } else {
          typedef u16 u16x4 __attribute__((ext_vector_type(4)));
          u16x4 part[3];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float rest = v[i];
#pragma unroll
            for (int q = 0; q < 3; ++q) {
              part[q][i] = static_cast<u16>(__builtin_bit_cast(unsigned, rest) >> 16);
              rest = __builtin_isinf(rest) ? 0.0f : rest - Elem<kBf16>::get(part[q][i]);
            }
          }
          if (p.h && !p.floats) {
            u16 *to = static_cast<u16 *>(p.h) + static_cast<long long>(row) * (3 * RP) + t * 16 + 4 * g;
#pragma unroll
            for (int q = 0; q < 3; ++q) *reinterpret_cast<u16x4 *>(to + q * RP) = part[q];
          }
          if (p.parts) {
            const long long plane = static_cast<long long>(RP) * a.positions;
#pragma unroll
            for (int q = 0; q < 3; ++q)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                static_cast<u16 *>(p.parts)[q * plane + static_cast<long long>(t * 16 + 4 * g + i) * a.positions + at] = part[q][i];
          }
        }
      }
  }
}

// 16 J rows of an adapter's N x rank matrix from row n0 on, as operands: row m of operand j is row
// n0 + 16 j + m.
template <int TYPE, int J, int KS, int PB>
__device__ __attribute__((always_inline)) inline void load_b(const typename Elem<TYPE>::store *w, long long ldw, int n0, int N, int stored,
                                                                 uintx4 (&b)[J][KS][PB]) {
  constexpr int kLane = kLaneK<TYPE>;
  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int n = min(n0 + 16 * j + i16, N - 1);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int r = s * 4 * kLane + g * kLane;
      b[j][s][0] = load_k<TYPE>(w + n * ldw + r, stored - r);
    }
  }
}

// What is stored behind the adapter's own rank goes (apart from the loads: none waits for the
// rank); halfs in two parts (PB).
template <int TYPE, int J, int KS, int PB>
__device__ __attribute__((always_inline)) inline void finish_b(int stored, int rank, uintx4 (&b)[J][KS][PB]) {
  constexpr int kLane = kLaneK<TYPE>;
  const int g = (threadIdx.x & 63) >> 4;
  if (rank < stored) {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int real = rank - (s * 4 * kLane + g * kLane);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (TYPE == kF32) b[j][s][0][i] = i < real ? b[j][s][0][i] : 0;
          else b[j][s][0][i] = 2 * i + 1 < real ? b[j][s][0][i] : 2 * i < real ? b[j][s][0][i] & 0xffff : 0;
        }
    }
  }
  if constexpr (PB == 2) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        bf16x8 parts[2];
        split_halfs(b[j][s][0], parts);
        b[j][s][0] = __builtin_bit_cast(uintx4, parts[0]);
        b[j][s][1] = __builtin_bit_cast(uintx4, parts[1]);
      }
  }
}

// The lane's columns of H of one row as operands, from floats: bfloat16 parts, or as they are.
template <int TYPE, int PH>
__device__ __attribute__((always_inline)) inline void hidden_operand(const f32x4 (&v)[kLaneK<TYPE> / 4], uintx4 (&h)[PH]) {
  if constexpr (TYPE == kF32) {
    h[0] = __builtin_bit_cast(uintx4, v[0]);
  } else {
    float y[8];
    floats8(v[0], v[1], y);
    bf16x8 parts[3];
    split8<3>(y, parts);
#pragma unroll
    for (int q = 0; q < PH; ++q) h[q] = __builtin_bit_cast(uintx4, parts[q]);
  }
}

// sum = B H^T of such operands. Small products come first (the third part of H times the second
// of B is below 2^-24). The other parts of an infinity, or products of zeros with one, are NaN:
// where neither the sum nor that of the first parts is finite, the latter stands alone.
template <int TYPE, int J, int KS, int PB, int PH>
__device__ __attribute__((always_inline)) inline void multiply_parts(const uintx4 (&b)[J][KS][PB], const uintx4 (&h)[KS][PH], f32x4 (&sum)[J]) {
  if constexpr (TYPE == kF32) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      sum[j] = f32x4{};
#pragma unroll
      for (int s = 0; s < KS; ++s) sum[j] = multiply<kF32>(b[j][s][0], h[s][0], sum[j]);
    }
  } else {
    auto first = [&](int j, f32x4 acc) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < KS; ++s) acc = multiply<kBf16>(b[j][s][0], h[s][0], acc);
      return acc;
    };
    float check = 0.0f;   // NaN with anything that is not finite
#pragma unroll
    for (int j = 0; j < J; ++j) {
      sum[j] = f32x4{};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int q = PH - 1; q > 0; --q) sum[j] = multiply<kBf16>(b[j][s][0], h[s][q], sum[j]);
        if constexpr (PB == 2) {
          sum[j] = multiply<kBf16>(b[j][s][1], h[s][1], sum[j]);
          sum[j] = multiply<kBf16>(b[j][s][1], h[s][0], sum[j]);
        }
      }
      sum[j] = first(j, sum[j]);
#pragma unroll
      for (int v = 0; v < 4; ++v) check = fmaf(sum[j][v], 0.0f, check);
    }
    if (__any(check != check)) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const f32x4 alone = first(j, f32x4{});
#pragma unroll
        for (int v = 0; v < 4; ++v)   // (a sum that is finite stays, whatever brought the wave here)
          sum[j][v] = __builtin_isfinite(sum[j][v]) || __builtin_isfinite(alone[v]) ? sum[j][v] : alone[v];
      }
    }
  }
}

// 4 neighbouring values of a row, the first `left` of them.
template <int TYPE>
__device__ inline void store4(typename Elem<TYPE>::store *p, int left, const float *v) {
  typedef typename Elem<TYPE>::store store;
  typedef store vec4 __attribute__((ext_vector_type(4), aligned(sizeof(store))));
  if (left >= 4) {
    *reinterpret_cast<vec4 *>(p) = vec4{Elem<TYPE>::put(v[0]), Elem<TYPE>::put(v[1]), Elem<TYPE>::put(v[2]), Elem<TYPE>::put(v[3])};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = Elem<TYPE>::put(v[i]);
  }
}

// ---------------------------------------------------------------------------
// expand.
struct ExpandArgs {
  LoraRows r;
  const void *h;           // as shrink left it: parts, or sums of `splits` ranges
  int splits;
  const void *w;           // adapter a's N x rank at w + a * w_adapter, row stride ldw
  long long w_adapter, ldw;
  const void *c;           // null: zeros
  long long ldc;
  void *y;
  long long ldy;
  int N, windows;          // of a workgroup
  int units_by;            // workgroups that the units are dealt out among
  bool in_place;           // c is y
};

// A wave keeps 16 J rows of an adapter's B in registers and takes unit after unit, every
// units_by-th of its windows'; they are loaded again where the adapter changes. C and H of
// the next units are on their way meanwhile. The products leave through LDS, so that C and Y
// move as whole lines of a row (128 bytes with J = 4), which the layout of the
// instructions' results, 16 rows beside each other, would cut into halves.
// Bound by memory: 8192 x 4096 bfloat16, rank 16, 31 us for 134 MB (4.3 TB/s; a copy of as many bytes
// takes 26), rank 32 34; with stores of 64 bytes a row and a load inside a branch it took 42.
// SUM: H are floats of several ranges of K (few rows), which are summed here. What is loaded
// for a unit depends on nothing else, so that the compiler can count how many loads may be
// on their way: without a C, Y is read in its place and the values are not used.
template <int TYPE, int RT, int J, bool SUM>
__global__ __launch_bounds__(256) void expand_kernel(ExpandArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int RP = 16 * RT, kLane = kLaneK<TYPE>, COLS = 16 * J;
  constexpr int KS = TYPE == kF32 ? RT : (RT + 1) / 2;   // operands along the rank: of 16 or 32
  constexpr int PB = TYPE == kF16 ? 2 : 1;               // parts of B
  constexpr int PH = TYPE == kF32 ? 1 : 3;               // parts of H
  constexpr int VEC = J == 1 ? 4 : kLane;                // values of C and Y that a lane moves at a time
  constexpr int kRowLanes = COLS / VEC, kRowsAt = 64 / kRowLanes, CW = 16 / kRowsAt;
  constexpr int kDepth = KS * PH + CW <= 8 ? 4 : 2;      // units on their way (SUM: one)
  constexpr int kStride = COLS + 4;                      // floats of a row in LDS
  __shared__ __attribute__((aligned(16))) float stages[4][16 * kStride];
  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float *stage = stages[wave];
  const int col_blocks = (a.N + 4 * COLS - 1) / (4 * COLS);
  const int nb = (blockIdx.x % col_blocks * 4 + wave) * COLS;
  if (nb >= a.N) return;
  const int windows = (a.r.rows + 63) / 64, ranges = (windows + a.windows - 1) / a.windows;
  const int range = blockIdx.x / col_blocks, group = range / ranges;   // (group slowest, as in shrink)
  const int window0 = (range - group * ranges) * a.windows, window1 = min(window0 + a.windows, windows);
  const int n_lane = nb + lane % kRowLanes * VEC, left = a.N - n_lane;

  uintx4 b[J][KS][PB];
  int have = -1;
  const store *c_or_y = static_cast<const store *>(a.c ? a.c : a.y);
  const long long ld_c_or_y = a.c ? a.ldc : a.ldy;
  auto load_adapter = [&](int id) __attribute__((always_inline)) {
    const int rank = a.r.rank_of(id);
    load_b<TYPE>(static_cast<const store *>(a.w) + id * a.w_adapter, a.ldw, nb, a.N, a.r.rank, b);
    finish_b<TYPE>(a.r.rank, rank, b);
    // (here, or every use of them would wait for all loads)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int s = 0; s < KS; ++s) arrived(b[j][s][0]);
  };

  struct Fetched {
    int id;
    int row[CW];   // of the lane's values; ~row past the unit's last
    uintx4 c[CW], h[KS][PH];
  };
  Units<1> unit(a.r, !a.in_place, window0, window1);
  int skip = group;   // units of other workgroups before the next of this one's
  auto advance = [&]() __attribute__((always_inline)) {
    bool more = unit.step();
    for (; more && skip > 0; --skip) more = unit.step();
    skip = a.units_by - 1;
    if (more) unit.rows();
    return more;
  };
  // WHOLE: all of the wave's columns exist.
  auto run = [&](auto whole) __attribute__((always_inline)) {
    constexpr bool WHOLE = decltype(whole)::value;
    auto fetch = [&](Fetched &f) __attribute__((always_inline)) {
      f.id = unit.id;
      const int mine = unit.row[0], marked = unit.real[0] ? mine : ~mine;
#pragma unroll
      for (int q = 0; q < CW; ++q) {
        f.row[q] = __shfl(marked, q * kRowsAt + lane / kRowLanes);
        const store *c = c_or_y + max(f.row[q], ~f.row[q]) * ld_c_or_y + n_lane;
        if constexpr (VEC < kLane) {
          typedef store store4 __attribute__((ext_vector_type(4), aligned(sizeof(store))));
          store4 v = {};
          if (WHOLE || left >= 4) {
            v = *reinterpret_cast<const store4 *>(c);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < left) v[i] = c[i];
          }
          f.c[q] = uintx4{static_cast<unsigned>(v[0]) | static_cast<unsigned>(v[1]) << 16,
                          static_cast<unsigned>(v[2]) | static_cast<unsigned>(v[3]) << 16, 0, 0};
        } else if constexpr (WHOLE) {
          f.c[q] = load_k<TYPE>(c);
        } else {
          f.c[q] = load_k<TYPE>(c, left);
        }
      }
      // (Of the 32 ranks of an operand the upper 16 do not exist where RP is 16: the lower again.)
      if constexpr (TYPE != kF32 && !SUM) {
        const u16 *h = static_cast<const u16 *>(a.h) + static_cast<long long>(mine) * (3 * RP);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int q = 0; q < PH; ++q)
            f.h[s][q] = *reinterpret_cast<const uintx4 *>(h + q * RP + (s * 32 + g * 8) % RP);
      } else {
        const float *h = static_cast<const float *>(a.h) + static_cast<long long>(mine) * RP;
        const long long range = static_cast<long long>(a.r.rows) * RP;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const float *from = h + (s * 4 * kLane + g * kLane) % RP;
          f32x4 v[kLane / 4];
#pragma unroll
          for (int i = 0; i < kLane / 4; ++i) v[i] = reinterpret_cast<const f32x4 *>(from)[i];
          if constexpr (SUM) {   // four more ranges at a time
            for (int q = 1; q < a.splits; q += 4) {
              f32x4 x[4][kLane / 4];
#pragma unroll
              for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < kLane / 4; ++i)
                  x[m][i] = reinterpret_cast<const f32x4 *>(from + min(q + m, a.splits - 1) * range)[i];
#pragma unroll
              for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < kLane / 4; ++i) v[i] += q + m < a.splits ? x[m][i] : f32x4{};
            }
          }
          hidden_operand<TYPE>(v, f.h[s]);
        }
      }
    };
    // H B^T of a unit to LDS: lane (g, i16) has columns 16 j + 4 g .. + 3 of row i16.
    auto product = [&](const Fetched &f) __attribute__((always_inline)) {
      const bool upper = RP % 32 != 0 && g >= 2;   // ranks that do not exist
      uintx4 h[KS][PH];
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int q = 0; q < PH; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) h[s][q][i] = TYPE != kF32 && upper ? 0u : f.h[s][q][i];
      f32x4 sum[J];
      multiply_parts<TYPE>(b, h, sum);
      wave_order();
#pragma unroll
      for (int j = 0; j < J; ++j) *reinterpret_cast<f32x4 *>(stage + i16 * kStride + 16 * j + 4 * g) = sum[j];
      wave_order();
    };
    auto finish = [&](const Fetched &f) __attribute__((always_inline)) {
      if (f.id >= 0) {
        if (f.id != have) {
          load_adapter(f.id);
          have = f.id;
        }
        product(f);
      }
#pragma unroll
      for (int q = 0; q < CW; ++q) {
        float out[8];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const unsigned w = TYPE == kF32 ? f.c[q][i % 4] : f.c[q][i / 2];
          if (!a.c) out[i] = 0.0f;
          else if constexpr (TYPE == kF32) out[i] = __builtin_bit_cast(float, w);
          else out[i] = Elem<TYPE>::get(static_cast<u16>(i % 2 ? w >> 16 : w));
        }
        if (f.id >= 0) {
          const float *from = stage + (q * kRowsAt + lane / kRowLanes) * kStride + lane % kRowLanes * VEC;
#pragma unroll
          for (int i = 0; i < VEC; i += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(from + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) out[i + k] += v[k];
          }
        }
        if (f.row[q] < 0) continue;
        store *y = static_cast<store *>(a.y) + f.row[q] * a.ldy + n_lane;
        if constexpr (VEC == 8) {
          store8<TYPE>(y, WHOLE ? 8 : left, out);
        } else {
          store4<TYPE>(y, WHOLE ? 4 : left, out);
        }
      }
    };
    if (!advance()) return;
    if (unit.id >= 0) {   // (before what H may have to be summed from)
      load_adapter(unit.id);
      have = unit.id;
    }
    if constexpr (SUM) {
      Fetched f;
      do {
        fetch(f);
        finish(f);
      } while (advance());
      return;
    }
    // (After the last unit the same again: a branch around loads would wait for them.)
    Fetched f[kDepth];
    bool more[kDepth];
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      more[d] = d == 0 || (more[d - 1] && advance());
      fetch(f[d]);
    }
    while (true) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (!more[d]) return;
        finish(f[d]);
        more[d] = more[(d + kDepth - 1) % kDepth] && advance();
        fetch(f[d]);
      }
    }
  };
  if (nb + COLS <= a.N) run(std::true_type());
  else run(std::false_type());
}

// ---------------------------------------------------------------------------
// Both products in one kernel, for a few rows on adapters of a rank up to 32.
struct SmallArgs {
  LoraRows r;          // up to 64 rows
  const void *x;
  long long ldx;
  const void *a, *b;   // as in gemm.h
  const void *c;       // null: zeros
  long long ldc;
  void *y;
  long long ldy;
  int N, K, units_by;
  bool in_place;
};
constexpr int kSmallWaves = 8, kSmallCols = 16 * kSmallWaves;

// One workgroup: 128 columns of Y, every units_by-th unit. Its waves share K for H, each workgroup
// for itself: A is read once for each 128 columns, from L2. Then each wave makes 16 columns. What
// bounds it is the chain of waits, so whatever a unit needs is loaded at once: B, C, the first
// operands of H.
template <int TYPE, int RT>
__global__ __launch_bounds__(64 * kSmallWaves) void small_kernel(SmallArgs a) {
  typedef typename Elem<TYPE>::store store;
  typedef store vec4 __attribute__((ext_vector_type(4), aligned(sizeof(store))));
  constexpr int W = kSmallWaves, kLane = kLaneK<TYPE>, kChunk = 4 * kLane, U = RT == 1 ? 8 : 4;
  constexpr int KS = TYPE == kF32 ? RT : (RT + 1) / 2, PB = TYPE == kF16 ? 2 : 1, PH = TYPE == kF32 ? 1 : 3;
  constexpr int kStride = 20;   // floats of a row in LDS
  __shared__ __attribute__((aligned(16))) f32x4 sums[W * RT * 64];
  __shared__ __attribute__((aligned(16))) float stages[W][16 * kStride];
  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col_blocks = (a.N + kSmallCols - 1) / kSmallCols;
  const int group = blockIdx.x / col_blocks;
  const int col0 = (blockIdx.x - group * col_blocks) * kSmallCols;
  const int nb = col0 + wave * 16;   // (may lie past the last column)
  const int k_wave = ((a.K + W - 1) / W + 63) / 64 * 64;
  const int ka = min(a.K, wave * k_wave), kb = min(a.K, ka + k_wave);
  float *stage = stages[wave];
  // A lane moves 4 columns of one row of C and Y. (Without a C, Y is read and not used.)
  const int col = nb + lane % 4 * 4, left = a.N - col;
  const store *c_or_y = static_cast<const store *>(a.c ? a.c : a.y) + min(col, a.N - 1);
  const long long ld_c_or_y = a.c ? a.ldc : a.ldy;

  Units<1> unit(a.r, !a.in_place, 0, 1);
  auto run = [&](auto whole) __attribute__((always_inline)) {
    constexpr bool WHOLE = decltype(whole)::value;
    int skip = group;
    while (unit.step()) {
      if (skip-- > 0) continue;
      skip = a.units_by - 1;
      unit.rows();
      const int id = max(unit.id, 0);   // (without an adapter: one's loads, not used)
      const int marked = __shfl(unit.real[0] ? unit.row[0] : ~unit.row[0], lane / 4), row = max(marked, ~marked);
      const long long adapter = static_cast<long long>(id) * a.r.rank;
      uintx4 b[1][KS][PB];
      load_b<TYPE>(static_cast<const store *>(a.b) + adapter * a.N, a.r.rank, min(nb, a.N - 1), a.N, a.r.rank, b);
      const store *from_c = c_or_y + row * ld_c_or_y;
      vec4 c = {};
      if constexpr (WHOLE) {
        c = *reinterpret_cast<const vec4 *>(from_c);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = from_c[max(0, min(i, left - 1))];
      }
      const int rank = a.r.rank_of(id);
      const float scale = a.r.scales ? a.r.scales[id] : 1.0f;
      const store *w = static_cast<const store *>(a.a) + adapter * a.K + g * kLane;
      const store *z = static_cast<const store *>(a.x) + unit.row[0] * a.ldx + g * kLane;
      const store *wr[RT];
#pragma unroll
      for (int t = 0; t < RT; ++t) wr[t] = w + static_cast<long long>(min(t * 16 + i16, a.r.rank - 1)) * a.K;
      f32x4 acc[RT] = {};
      struct Fetched {
        uintx4 w[U][RT], z[U];
      };
      int k = ka;
      const int batches = (kb - ka) / (U * kChunk);
      if (batches > 0) {
        Fetched even, odd;
        two_deep(
            batches, even, odd,
            [&](Fetched &f) __attribute__((always_inline)) {
#pragma unroll
              for (int u = 0; u < U; ++u) {
                f.z[u] = load_k<TYPE>(z + k + u * kChunk);
#pragma unroll
                for (int t = 0; t < RT; ++t) f.w[u][t] = load_k<TYPE>(wr[t] + k + u * kChunk);
              }
              k += U * kChunk;
            },
            [&](const Fetched &f) __attribute__((always_inline)) {
#pragma unroll
              for (int u = 0; u < U; ++u)
#pragma unroll
                for (int t = 0; t < RT; ++t) acc[t] = multiply<TYPE>(f.w[u][t], f.z[u], acc[t]);
            });
      }
      // (the rest two chunks at a time)
      for (; k < kb; k += 2 * kChunk) {
        const int rest = kb - k - g * kLane;
        uintx4 zv[2], wv[2][RT];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          zv[u] = load_k<TYPE>(z + k + u * kChunk, rest - u * kChunk);
#pragma unroll
          for (int t = 0; t < RT; ++t) wv[u][t] = load_k<TYPE>(wr[t] + k + u * kChunk, rest - u * kChunk);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[t] = multiply<TYPE>(wv[u][t], zv[u], acc[t]);
      }
      __syncthreads();   // (the unit before has been read)
#pragma unroll
      for (int t = 0; t < RT; ++t) sums[(wave * RT + t) * 64 + lane] = acc[t];
      __syncthreads();
      // The lane's columns of H of row i16, scaled, zeros past the rank: value v of lane (g, i16) of tile t
      // is column 16 t + 4 g + v.
      finish_b<TYPE>(a.r.rank, rank, b);
      uintx4 h[KS][PH];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        f32x4 v[kLane / 4];
#pragma unroll
        for (int i = 0; i < kLane / 4; ++i) {
          const int r = s * 4 * kLane + g * kLane + 4 * i;
          const f32x4 *from = sums + r % (16 * RT) / 16 * 64 + r % 16 / 4 * 16 + i16;
          v[i] = from[0];
#pragma unroll
          for (int q = 1; q < W; ++q) v[i] += from[q * RT * 64];
#pragma unroll
          for (int m = 0; m < 4; ++m) v[i][m] = r + m < rank ? v[i][m] * scale : 0.0f;
        }
        hidden_operand<TYPE>(v, h[s]);
      }
      f32x4 sum[1];
      multiply_parts<TYPE>(b, h, sum);
      wave_order();
      *reinterpret_cast<f32x4 *>(stage + i16 * kStride + 4 * g) = sum[0];
      wave_order();
      const f32x4 v = *reinterpret_cast<const f32x4 *>(stage + lane / 4 * kStride + lane % 4 * 4);
      float out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        out[i] = a.c ? Elem<TYPE>::get(c[i]) : 0.0f;
        out[i] = unit.id >= 0 ? out[i] + v[i] : out[i];
      }
      if (marked >= 0) store4<TYPE>(static_cast<store *>(a.y) + row * a.ldy + col, left, out);
    }
  };
  // WHOLE: all of the workgroup's columns exist. (Of the workgroup's, not of the wave's: its waves
  // have to meet at the same barriers.)
  if (col0 + kSmallCols <= a.N) run(std::true_type());
  else run(std::false_type());
}

// ---------------------------------------------------------------------------
// Backward: the rows sorted by adapter, A and B transposed.

// A stretch of up to `slot_rows` rows of one adapter, in the sorted order.
struct Slot {
  int adapter, first, count;   // positions
  int partial;                 // where its sums go: -1 straight to the gradient, else a partial sum
};
struct LoraPlan {
  int slots, pad[3];
};
struct PrepareArgs {
  LoraRows r;
  int slot_rows, N;
  LoraPlan *plan;
  Slot *slots;
  int2 *sums;           // adapter: its first partial sum, how many (-1: written straight)
  int *order;           // position -> row
  int *position;        // row -> position
  const void *a, *b;    // rank x K and N x rank for each adapter
  void *at, *bt;        // K x rank and rank x N for each
  int K;
  int a_tiles, b_tiles; // of each adapter's: kTransRows columns of A, rows of B
};
constexpr int kTransRows = 64;   // columns of A, rows of B of a tile

// Lanes of the wave that have the same id (valid ones).
__device__ inline unsigned long long same_id(int id, bool valid, int bits) {
  unsigned long long m = __ballot(valid);
  for (int b = 0; b < bits; ++b) {
    const bool one = (id >> b) & 1;
    const unsigned long long ones = __ballot(one);
    m &= one ? ones : ~ones;
  }
  return m;
}

// Workgroup 0 sorts the rows by adapter, keeping their order (so that sums over them do not
// depend on timing): every wave counts a stretch of rows, running sums over adapters and
// waves say where each wave's rows of an adapter go, and each wave puts its
// rows there. An adapter's positions begin at a multiple of 32. The other workgroups share the
// tiles of A and B, which they transpose, of those adapters that rows have. (64 rows on 32 of
// 1024 adapters, 4096 x 4096, rank 16: 156 us backward, and 640 with workgroups for every adapter; 8192 rows on 64: 161 and 185.)
// 10 us for 8192 rows and 4 adapters of rank 32 and 4096 x 4096: the waits of a few dependent steps.
template <int TYPE>
__global__ __launch_bounds__(1024) void prepare_kernel(PrepareArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int W = 16;
  __shared__ int lds[W * kLoraMaxAdapters + 3 * 16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (blockIdx.x > 0) {
    // The adapters that rows have, in order: first a flag for each, then their list in its place.
    int *used = lds + kLoraMaxRank * (kTransRows + 1), *sums = lds + W * kLoraMaxAdapters;
    used[threadIdx.x] = 0;
    __syncthreads();
    for (int row0 = 0; row0 < a.r.rows; row0 += 8 * 1024) {   // 8192 ids on their way at a time
      int loaded[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) loaded[i] = a.r.load_id(row0 + i * 1024 + threadIdx.x);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (a.r.id_of(loaded[i]) >= 0) used[loaded[i]] = 1;
    }
    __syncthreads();
    const bool mine = used[threadIdx.x] != 0;
    const unsigned long long wave_has = __ballot(mine);
    if (lane == 0) sums[wave] = __popcll(wave_has);
    __syncthreads();
    int many_used = 0, before = 0;
    for (int w = 0; w < W; ++w) {
      before += w < wave ? sums[w] : 0;
      many_used += sums[w];
    }
    if (mine) used[before + __popcll(wave_has & ((1ull << lane) - 1))] = threadIdx.x;
    __syncthreads();

    store *tile = reinterpret_cast<store *>(lds);   // [rank][64], a row of 65
    const int tiles = a.a_tiles + a.b_tiles, rank = a.r.rank;
    for (int unit = blockIdx.x - 1; unit < many_used * tiles; unit += gridDim.x - 1) {
      const int id = used[unit / tiles], at = unit % tiles;
      const bool second = at >= a.a_tiles;
      const int size = second ? a.N : a.K;            // across the ranks
      const int n0 = (second ? at - a.a_tiles : at) * kTransRows, many = min(kTransRows, size - n0);
      const long long adapter = static_cast<long long>(id) * rank * size;
      const store *from = static_cast<const store *>(second ? a.b : a.a) + adapter;
      store *to = static_cast<store *>(second ? a.bt : a.at) + adapter;
      // the ranks along a row (B, A transposed), or 64 neighbours of one rank (A, B transposed)
      auto along = [&](bool load) {
        for (int i = threadIdx.x; i < many * rank; i += 1024) {
          store &v = tile[i % rank * (kTransRows + 1) + i / rank];
          if (load) v = from[static_cast<long long>(n0) * rank + i];
          else to[static_cast<long long>(n0) * rank + i] = v;
        }
      };
      auto across = [&](bool load) {
        for (int i = threadIdx.x; i < kTransRows * rank; i += 1024) {
          const int n = i % kTransRows, r = i / kTransRows;
          if (n >= many) continue;
          store &v = tile[r * (kTransRows + 1) + n];
          if (load) v = from[static_cast<long long>(r) * size + n0 + n];
          else to[static_cast<long long>(r) * size + n0 + n] = v;
        }
      };
      if (second) along(true); else across(true);
      __syncthreads();
      if (second) across(false); else along(false);
      __syncthreads();
    }
    return;
  }
  int *count = lds, *across = lds + W * kLoraMaxAdapters;   // [wave][adapter]; sums over the waves' adapters
  const int bits = 32 - __builtin_clz(max(a.r.adapters - 1, 1));
  for (int i = threadIdx.x; i < W * kLoraMaxAdapters; i += 1024) count[i] = 0;
  __syncthreads();
  const int per = ((a.r.rows + W - 1) / W + 63) / 64 * 64;
  const int from = min(a.r.rows, wave * per), to = min(a.r.rows, from + per);
  // step(row, id) for 64 of the wave's rows after the other, the ids of 8 such on their way at a time.
  auto over_rows = [&](auto &&step) __attribute__((always_inline)) {
    constexpr int kAt = 8;
    for (int row0 = from; row0 < to; row0 += 64 * kAt) {
      int loaded[kAt];
#pragma unroll
      for (int i = 0; i < kAt; ++i) loaded[i] = a.r.load_id(row0 + i * 64 + lane);
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        const int row = row0 + i * 64 + lane;
        if (row - lane < to) step(row, row < to ? a.r.id_of(loaded[i]) : -1);
      }
    }
  };
  over_rows([&](int, int id) {
    const unsigned long long same = same_id(id, id >= 0, bits);
    if (id >= 0 && (same & ((1ull << lane) - 1)) == 0) count[wave * kLoraMaxAdapters + id] += __popcll(same);
    wave_order();
  });
  __syncthreads();
  // Thread t has adapter t: its rows, positions (rounded up to 32), slots and partial sums,
  // and running sums of the last three over all adapters.
  const int id = threadIdx.x;
  int rows = 0;
  if (id < a.r.adapters) {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int n = count[w * kLoraMaxAdapters + id];
      count[w * kLoraMaxAdapters + id] = rows;
      rows += n;
    }
  }
  const int slots = (rows + a.slot_rows - 1) / a.slot_rows;
  int v[3] = {(rows + 31) / 32 * 32, slots, slots > 1 ? slots : 0}, before[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int upto = wave_running_sum(v[i]);
    before[i] = upto - v[i];
    if (lane == 63) across[i * W + wave] = upto;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i)
    for (int w = 0; w < wave; ++w) before[i] += across[i * W + w];
  if (threadIdx.x == 1023) a.plan->slots = before[1] + v[1];
  if (id < a.r.adapters) {
    for (int s = 0; s < slots; ++s)
      a.slots[before[1] + s] = Slot{id, before[0] + s * a.slot_rows, min(a.slot_rows, rows - s * a.slot_rows),
                                    slots > 1 ? before[2] + s : -1};
    a.sums[id] = make_int2(before[2], slots == 1 ? -1 : slots);
#pragma unroll
    for (int w = 0; w < W; ++w) count[w * kLoraMaxAdapters + id] += before[0];
  }
  __syncthreads();
  over_rows([&](int row, int mine) {
    const unsigned long long same = same_id(mine, mine >= 0, bits);
    const int number = __popcll(same & ((1ull << lane) - 1));
    if (mine >= 0) {
      const int at = count[wave * kLoraMaxAdapters + mine] + number;
      a.order[at] = row;
      a.position[row] = at;
    }
    wave_order();
    if (mine >= 0 && number == 0) count[wave * kLoraMaxAdapters + mine] += __popcll(same);
    wave_order();
  });
}

// ---------------------------------------------------------------------------
// grads.
struct Grad {
  const void *z;         // rows x cols: X, or dY
  long long ldz;
  int cols;
  const void *parts;     // of G, or H
  float *partial;        // [partial sum][cols x rank or rank x cols]
  float *out;            // the same for each adapter
};
struct GradArgs {
  LoraRows r;
  const LoraPlan *plan;
  const Slot *slots;
  const int *order;
  int positions;
  Grad p[2];             // dA: rank x cols; dB: cols x rank
  int blocks0, blocks;   // column blocks of the first, of both
  int slot0;             // of the launch
  int rp, rank_blocks;   // ranks of `parts`, and the stretches of 16 RT that they are taken in
};

// One workgroup: a slot's rows, 16 CL columns (CL of a lane) and 16 RT ranks (128 ranks
// would not fit the registers: two workgroups share them). Its waves take 32 rows (16 of
// FP32) in turn, and their sums are added in order at the end. A lane loads CL neighbouring columns of 8 rows
// (4 of FP32): turned in its registers, these are the operands of CL instructions, whose
// column i16 is column CL i16 + j.
// Bound by memory: 8192 rows of 4096 + 4096 bfloat16 (134 MB), rank 32, 40 us (3.4 TB/s).
template <int TYPE, int RT>
__global__ __launch_bounds__(256) void grad_kernel(GradArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int CL = kLaneK<TYPE>, kRows = kLaneK<TYPE>, kStep = 4 * kRows;
  constexpr int PZ = TYPE == kF16 ? 2 : 1, PP = TYPE == kF32 ? 1 : 3;
  __shared__ __attribute__((aligned(16))) f32x4 sums[CL * RT * 64];
  const int lane = threadIdx.x & 63, i16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot_at = a.slot0 + blockIdx.x / (a.blocks * a.rank_blocks);
  const int rank0 = blockIdx.x % a.rank_blocks * (16 * RT);
  int block = blockIdx.x / a.rank_blocks % a.blocks;
  if (slot_at >= a.plan->slots) return;
  const bool second = block >= a.blocks0;
  const Grad p = second ? a.p[1] : a.p[0];
  if (second) block -= a.blocks0;
  const Slot slot = a.slots[slot_at];
  const int n = (block * 16 + i16) * CL, left = p.cols - n;
  const long long plane = static_cast<long long>(a.rp) * a.positions;
  f32x4 acc[CL][RT] = {};
  struct Fetched {
    uintx4 x[kRows], p[RT][PP];
  };
  // The lane's rows of a step; past the slot's last the last again.
  auto rows_of = [&](int at, int (&rows)[kRows]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) rows[i] = a.order[slot.first + min(at + g * kRows + i, slot.count - 1)];
  };
  // WHOLE: all of the workgroup's columns exist.
  auto fetch = [&](auto whole, Fetched &f, int at, const int (&rows)[kRows]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const store *z = static_cast<const store *>(p.z) + rows[i] * p.ldz + n;
      if constexpr (decltype(whole)::value) f.x[i] = load_k<TYPE>(z);
      else f.x[i] = load_k<TYPE>(z, left);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int q = 0; q < PP; ++q) {
        const long long from = (rank0 + t * 16 + i16) * static_cast<long long>(a.positions) + slot.first + at + g * kRows;
        if constexpr (TYPE == kF32) f.p[t][q] = *reinterpret_cast<const uintx4 *>(static_cast<const float *>(p.parts) + from);
        else f.p[t][q] = *reinterpret_cast<const uintx4 *>(static_cast<const u16 *>(p.parts) + q * plane + from);
      }
  };
  // Rows past the slot's last: zeros on both sides.
  auto cut = [&](Fetched &f, int at) __attribute__((always_inline)) {
    const int real = slot.count - at - g * kRows;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) f.x[i][c] = i < real ? f.x[i][c] : 0;
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int q = 0; q < PP; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (TYPE == kF32) f.p[t][q][i] = i < real ? f.p[t][q][i] : 0;
          else f.p[t][q][i] = 2 * i + 1 < real ? f.p[t][q][i] : 2 * i < real ? f.p[t][q][i] & 0xffff : 0;
        }
  };
  auto add = [&](const Fetched &f) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < CL; ++j) {
      uintx4 z[PZ];
      if constexpr (TYPE == kF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[0][i] = f.x[i][j];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          z[0][i] = __builtin_amdgcn_perm(f.x[2 * i + 1][j / 2], f.x[2 * i][j / 2], j % 2 ? 0x07060302 : 0x05040100);
        if constexpr (PZ == 2) {
          bf16x8 parts[2];
          split_halfs(z[0], parts);
          z[0] = __builtin_bit_cast(uintx4, parts[0]);
          z[1] = __builtin_bit_cast(uintx4, parts[1]);
        }
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        if constexpr (TYPE == kF32) {
          acc[j][t] = multiply<kF32>(f.p[t][0], z[0], acc[j][t]);
        } else {
#pragma unroll
          for (int q = 0; q < PP; ++q) acc[j][t] = multiply<kBf16>(f.p[t][q], z[0], acc[j][t]);
          if constexpr (PZ == 2) {   // (the third part times the second is below 2^-24)
            acc[j][t] = multiply<kBf16>(f.p[t][0], z[1], acc[j][t]);
            acc[j][t] = multiply<kBf16>(f.p[t][1], z[1], acc[j][t]);
          }
        }
      }
    }
  };
  // The rows of the step after the next and the operands of the next are on their way while
  // one is multiplied.
  int at = wave * kStep;
  const int steps = (slot.count - at + 4 * kStep - 1) / (4 * kStep);
  auto run = [&](auto whole) __attribute__((always_inline)) {
    int rows[kRows];
    auto step = [&](Fetched &cur, Fetched &next) __attribute__((always_inline)) {
      // (past the last step: its rows, and positions that exist, once more; without, as
      // shrink does it, 8192 rows of rank 32 took 47 us where this takes 40)
      const int then = min(at + 4 * kStep, wave * kStep + (steps - 1) * 4 * kStep);
      fetch(whole, next, then, rows);
      rows_of(then + 4 * kStep, rows);
      __builtin_amdgcn_sched_barrier(0);
      if (at + kStep > slot.count) cut(cur, at);
      add(cur);
      at += 4 * kStep;
    };
    Fetched even, odd;
    rows_of(at, rows);
    fetch(whole, even, at, rows);
    rows_of(min(at + 4 * kStep, wave * kStep + (steps - 1) * 4 * kStep), rows);
    in_turn(steps, even, odd, step);
  };
  if (steps > 0) {
    if ((block * 16 + 16) * CL <= p.cols) run(std::true_type());
    else run(std::false_type());
  }
  // The waves' sums in order.
  for (int w = 3; w > 0; --w) {
    __syncthreads();
    if (wave == w) {
#pragma unroll
      for (int j = 0; j < CL; ++j)
#pragma unroll
        for (int t = 0; t < RT; ++t) sums[(j * RT + t) * 64 + lane] = acc[j][t];
    }
    __syncthreads();
    if (wave == w - 1) {
#pragma unroll
      for (int j = 0; j < CL; ++j)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[j][t] += sums[(j * RT + t) * 64 + lane];
    }
  }
  if (wave != 0) return;
  const int own = a.r.rank_of(slot.adapter);   // (behind it zeros, whatever Z holds)
  const long long size = static_cast<long long>(a.r.rank) * p.cols;
  float *out = slot.partial < 0 ? p.out + slot.adapter * size : p.partial + slot.partial * size;
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = rank0 + t * 16 + 4 * g + v;
      if (r >= a.r.rank) continue;
#pragma unroll
      for (int j = 0; j < CL; ++j)
        if (j < left) out[second ? static_cast<long long>(n + j) * a.r.rank + r : static_cast<long long>(r) * p.cols + n + j] = r < own ? acc[j][t][v] : 0.0f;
    }
}

// Gradients of the adapters with several slots, whose partial sums are added in order, and
// zeros for those that no row has (4 adapters of rank 32, 4096 + 4096, two or three slots each: 5 us).
struct GradSumArgs {
  const int2 *sums;
  const float *partial[2];
  float *out[2];
  long long size[2];     // of one adapter's
  int blocks;            // workgroups for each adapter's, of each of the two
};
template <int>
__global__ __launch_bounds__(256) void grad_sum_kernel(GradSumArgs a) {
  const int id = blockIdx.x / (2 * a.blocks), block = blockIdx.x % (2 * a.blocks);
  const int2 s = a.sums[id];
  if (s.y < 0) return;
  const bool second = block >= a.blocks;
  const long long size = second ? a.size[1] : a.size[0];
  const float *partial = (second ? a.partial[1] : a.partial[0]) + s.x * size;
  float *out = (second ? a.out[1] : a.out[0]) + id * size;
  const long long first = (static_cast<long long>(second ? block - a.blocks : block) * 256 + threadIdx.x) * 4;
  for (long long at = first; at < size; at += a.blocks * 1024LL) {
    if (at + 4 <= size) {
      typedef f32x4 f32x4_any __attribute__((aligned(4)));
      f32x4 v = {};
      for (int i = 0; i < s.y; ++i) v += *reinterpret_cast<const f32x4_any *>(partial + i * size + at);
      *reinterpret_cast<f32x4_any *>(out + at) = v;
    } else {
      for (long long k = at; k < size; ++k) {
        float v = 0.0f;
        for (int i = 0; i < s.y; ++i) v += partial[i * size + k];
        out[k] = v;
      }
    }
  }
}

}  // namespace mx
}  // namespace gemm
