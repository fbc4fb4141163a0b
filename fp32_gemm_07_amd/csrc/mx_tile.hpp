// The tiled product of two microscaled operands.
#pragma once

#include "gemm_kernels.hpp"
#include "mx_kernels.hpp"

namespace gemm {
namespace mx {

// A BM x BN tile per workgroup of 4 waves (2 x 2), v_mfma_scale_f32_32x32x64 on
// e2m1 operands.
//
// Both operands are K-contiguous rows of codes, so both are staged the same way:
// a stage is 128 values of K, 64 bytes a row, copied straight into LDS (16 bytes
// a lane) through a ring of 4 stages. Within a stage row x keeps its 16-byte
// chunk c (one block of 32 values) at c ^ ((x >> 2) & 3): 16 consecutive rows of
// one chunk, which 16 lanes read at a time, then meet every bank once. The
// scales of 512 values (16 bytes a row) go through a ring of 2 of their own.
//
// A stage is two steps of 64 values: lane (h, i) of an instruction holds block
// 2 * step + h of row i. The registers of one step are read from LDS while the
// instructions of the step before run. The wait for the next stage's copies and
// the workgroup's barrier stand in the middle of a stage's second step, when
// all of the stage has been read; the stage is then refilled, 4 stages
// ahead.
//
// Rows past M or N and stages past the K range are outside the copies' buffer
// ranges and read as zeros (a zero scale byte is 2^-127, not NaN).
//
// 8192^3 with 256 x 256 tiles takes 305 us, 3.6 PFLOP/s. The instructions alone (no
// reads, copies or stores) take 195 us on the same data: random operands draw so
// much power that the chip's matrix rate falls from 8.7 to 6.3 PFLOP/s. Copies add
// 70 us, LDS reads 33, the start and end of a tile about 10 of its 76.
// Smaller tiles are bound by the latency of a stage (LDS reads and a barrier around
// few instructions): 0.35 us a stage for 128 x 128, whether 4 or 8 stages are kept.
// 16 bytes of C: alpha * sums + beta * C, or with RAW the sums.
template <int TYPE, bool RAW>
__device__ inline void store_vec(typename Elem<TYPE>::store *c, const float *s, float alpha, float beta) {
  constexpr int kVec = TYPE == kF32 ? 4 : 8;
  typedef typename Elem<TYPE>::store store;
  struct __attribute__((aligned(16))) Vec {
    store e[kVec];
  } v;
  if (!RAW && beta != 0.0f) v = *reinterpret_cast<const Vec *>(c);
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float r = RAW ? s[e] : beta == 0.0f ? alpha * s[e] : fmaf(alpha, s[e], beta * Elem<TYPE>::get(v.e[e]));
    v.e[e] = Elem<TYPE>::put(r);
  }
  *reinterpret_cast<Vec *>(c) = v;
}

struct TileArgs {
  const unsigned char *ac, *as, *bc, *bs;
  void *C;       // of the launch's type, or with a split float partial sums
  int M, N, KP;
  int ldc;
  float alpha, beta;
  int k_chunk;   // values of K of a split, a multiple of 128
  int tiles_m, tiles_n, splits;
};

template <int BM, int BN>
struct TileShape {
  static constexpr int FM = BM / 64, FN = BN / 64;        // 32 x 32 blocks of a wave (2 x 2 waves)
  static constexpr int kStage = (BM + BN) * 64;           // bytes of codes of a stage
  static constexpr int kScales = (BM + BN) * 16;          // bytes of scales of 4 stages
  static constexpr int kStages = 4;
  static constexpr int kLds = kStages * kStage + 2 * kScales;
  static constexpr int kCopies = kStage / 4096;           // a wave's copies of a stage
  static constexpr int kScaleCopies = (kScales + 4095) / 4096;
};

template <int BM, int BN, int TYPE, bool SPLIT, int WPE>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(WPE, WPE)))
void tile_kernel(TileArgs a) {
  using S = TileShape<BM, BN>;
  constexpr int FM = S::FM, FN = S::FN, NS = S::kStages;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[S::kLds];

  const TileCoord tc = map_tile(blockIdx.x, a.tiles_m, a.tiles_n, a.splits, kGroupM);
  const int m0 = __builtin_amdgcn_readfirstlane(tc.tm) * BM;
  const int n0 = __builtin_amdgcn_readfirstlane(tc.tn) * BN;
  const int split = __builtin_amdgcn_readfirstlane(tc.split);
  const int k0 = split * a.k_chunk;
  const int stages = (min(a.KP, k0 + a.k_chunk) - k0) / 128;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 31, h = lane >> 5;
  const int wm = wave >> 1, wn = wave & 1;

  // Copies. Instruction q of a stage fills rows 16q .. 16q + 15 (A's rows, then B's),
  // 4 lanes a row; wave w takes q = w, w + 4, ..
  const long long code_row = a.KP / 2, scale_row = a.KP / 32;
  const u32x4 ra = make_buffer_rsrc(a.ac + m0 * code_row + k0 / 2, (a.M - m0) * code_row - k0 / 2);
  const u32x4 rb = make_buffer_rsrc(a.bc + n0 * code_row + k0 / 2, (a.N - n0) * code_row - k0 / 2);
  const u32x4 rsa = make_buffer_rsrc(a.as + m0 * scale_row + k0 / 32, (a.M - m0) * scale_row - k0 / 32);
  const u32x4 rsb = make_buffer_rsrc(a.bs + n0 * scale_row + k0 / 32, (a.N - n0) * scale_row - k0 / 32);
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(lds));
  const unsigned lane_off = static_cast<unsigned>((lane >> 2) * code_row) +
                            static_cast<unsigned>(((lane & 3) ^ ((lane >> 4) & 3)) * 16);
  auto copy_codes = [&](int q4, int stage, int base) {
    const int q = wave + 4 * q4;   // q4 is a constant, so is the operand (BM, BN multiples of 64)
    const bool of_a = q4 * 64 < BM;
    const unsigned row = static_cast<unsigned>(of_a ? q * 16 : q * 16 - BM);
    const unsigned so = stage < stages ? static_cast<unsigned>(stage) * 64u : kOutOfRange;
    dma_copy<4>(of_a ? ra : rb, lane_off + row * static_cast<unsigned>(code_row) + so,
                lds0 + base + q * 1024);
  };
  // Instruction q of 4 stages' scales fills rows 64q .. 64q + 63, a lane a row.
  auto copy_scales = [&](int q4, int super) {
    const int q = wave + 4 * q4;
    if (S::kScales % 4096 == 0 || q * 1024 < S::kScales) {
      const bool of_a = q * 64 < BM;
      const unsigned row = static_cast<unsigned>(of_a ? q * 64 : q * 64 - BM) + lane;
      const unsigned so = super * 4 < stages ? static_cast<unsigned>(super) * 16u : kOutOfRange;
      dma_copy<4>(of_a ? rsa : rsb, row * static_cast<unsigned>(scale_row) + so,
                  lds0 + NS * S::kStage + (super & 1) * S::kScales + q * 1024);
    }
  };

  // Operand registers of a step; scales of a stage, as read and shifted so that
  // byte 2 * step is the lane's.
  intx4 fa[2][FM], fb[2][FN];
  int sa[FM], sb[FN], sa_raw[FM], sb_raw[FN];
  const int sw = (i >> 2) & 3;
  const int off0 = i * 64 + ((h ^ sw) * 16);
  const unsigned char *la = lds + wm * (BM / 2) * 64, *lb = lds + (BM + wn * (BN / 2)) * 64;
  const unsigned char *lsa = lds + NS * S::kStage + (wm * (BM / 2) + i) * 16;
  const unsigned char *lsb = lds + NS * S::kStage + (BM + wn * (BN / 2) + i) * 16;
  auto read_a = [&](int f, int base, int step) {
    fa[step][f] = *reinterpret_cast<const intx4 *>(la + base + f * 2048 + (off0 ^ (step * 32)));
  };
  auto read_b = [&](int f, int base, int step) {
    fb[step][f] = *reinterpret_cast<const intx4 *>(lb + base + f * 2048 + (off0 ^ (step * 32)));
  };
  auto read_scales = [&](int stage) {
    const int at = ((stage >> 2) & 1) * S::kScales + (stage & 3) * 4;
#pragma unroll
    for (int f = 0; f < FM; ++f) sa_raw[f] = *reinterpret_cast<const int *>(lsa + at + f * 512);
#pragma unroll
    for (int f = 0; f < FN; ++f) sb_raw[f] = *reinterpret_cast<const int *>(lsb + at + f * 512);
  };

  f32x16 acc[FM][FN] = {};

  // Prologue: the first 4 stages and their scales on their way.
#pragma unroll
  for (int q = 0; q < S::kScaleCopies; ++q) copy_scales(q, 0);
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int q = 0; q < S::kCopies; ++q) copy_codes(q, s, s * S::kStage);
  wait_vmcnt<3 * S::kCopies>();
  asm volatile("s_barrier" : : : "memory");
#pragma unroll
  for (int f = 0; f < FM; ++f) read_a(f, 0, 0);
#pragma unroll
  for (int f = 0; f < FN; ++f) read_b(f, 0, 0);
  read_scales(0);

  constexpr int kMfmas = FM * FN;
  for (int t = 0; t < stages; ++t) {
    const int base = (t & 3) * S::kStage, next = ((t + 1) & 3) * S::kStage;
    // The scales of the next 4 stages, into the half that the 4 before this one had
    // (all read before the last barrier). A branch after the instructions below
    // would let the compiler move all of them behind it.
    if ((t & 3) == 0) {
#pragma unroll
      for (int q = 0; q < S::kScaleCopies; ++q) copy_scales(q, (t >> 2) + 1);
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = static_cast<int>(static_cast<unsigned>(sa_raw[f]) >> (8 * h));
#pragma unroll
    for (int f = 0; f < FN; ++f) sb[f] = static_cast<int>(static_cast<unsigned>(sb_raw[f]) >> (8 * h));
    // first step; the second step's registers are read meanwhile
    unroll_steps<0, kMfmas>([&](auto n_c) {
      constexpr int n = decltype(n_c)::value;
      constexpr int fm = n / FN, fn = n % FN;
      acc[fm][fn] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          widen(fb[0][fn]), widen(fa[0][fm]), acc[fm][fn], 4, 4, 0, sb[fn], 0, sa[fm]);
      if constexpr (n < FM) read_a(n, base, 1);
      else if constexpr (n < FM + FN) read_b(n - FM, base, 1);
      if constexpr (n == kMfmas - 1 && FM + FN > kMfmas) {
#pragma unroll
        for (int f = kMfmas; f < FM + FN; ++f) read_b(f - FM, base, 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    // second step
    constexpr int kBefore = kMfmas / 4;
    unroll_steps<0, kMfmas>([&](auto n_c) {
      constexpr int n = decltype(n_c)::value;
      constexpr int fm = n / FN, fn = n % FN;
      if constexpr (n == kBefore) {
        // all of this stage is read, the next one's copies have landed
        wait_vmcnt<2 * S::kCopies>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
      acc[fm][fn] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          widen(fb[1][fn]), widen(fa[1][fm]), acc[fm][fn], 4, 4, 2, sb[fn], 2, sa[fm]);
      if constexpr (n == kBefore) {
        read_scales(t + 1);
#pragma unroll
        for (int f = 0; f < FM; ++f) read_a(f, next, 0);
#pragma unroll
        for (int f = 0; f < FN; ++f) read_b(f, next, 0);
      }
      if constexpr (n >= kBefore) {
        constexpr int span = kMfmas - kBefore;
        constexpr int q0 = (n - kBefore) * S::kCopies / span, q1 = (n - kBefore + 1) * S::kCopies / span;
#pragma unroll
        for (int q = q0; q < q1; ++q) copy_codes(q, t + NS, base);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  wait_vmcnt<0>();   // no copy may land after the workgroup's LDS is another's

  // B's rows are the instructions' rows: accumulator v of lane (h, i) is row i of C
  // and column 8 (v / 4) + 4 h + v % 4 of a block, four neighbouring columns at a
  // time. 32 rows of the wave's tile pass through its own piece of LDS and leave
  // as whole rows, 16 bytes a lane (each lane storing what it holds, a few bytes
  // to each of 32 rows, took 14 us for a 256 x 256 tile, this 2 us).
  asm volatile("s_barrier" : : : "memory");   // everybody has read the last stage
  constexpr int kCols = BN / 2, kStride = kCols + 4;
  static_assert(4 * 32 * kStride * 4 <= S::kLds, "fits the ring");
  float *out = reinterpret_cast<float *>(lds) + wave * (32 * kStride);
  constexpr int OUT = SPLIT ? kF32 : TYPE;
  typedef typename Elem<OUT>::store store;
  constexpr int kVec = OUT == kF32 ? 4 : 8;             // elements of 16 bytes
  constexpr int kLanes = kCols / kVec, kRows = 64 / kLanes;   // lanes of a row, rows at a time
  store *c = static_cast<store *>(a.C) + (SPLIT ? static_cast<long long>(split) * a.M * a.N : 0);
  const long long ldc = SPLIT ? a.N : a.ldc;
  const int col = n0 + wn * kCols + (lane % kLanes) * kVec;
  const bool vec = col + kVec <= a.N && ldc % kVec == 0 && reinterpret_cast<uintptr_t>(c) % 16 == 0;
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
    for (int fn = 0; fn < FN; ++fn)
#pragma unroll
      for (int v = 0; v < 16; v += 4)
        *reinterpret_cast<f32x4 *>(out + i * kStride + fn * 32 + 2 * v + 4 * h) =
            f32x4{acc[fm][fn][v], acc[fm][fn][v + 1], acc[fm][fn][v + 2], acc[fm][fn][v + 3]};
    wave_order();
#pragma unroll 4
    for (int r = lane / kLanes; r < 32; r += kRows) {
      const int row = m0 + wm * (BM / 2) + fm * 32 + r;
      float s[kVec];
#pragma unroll
      for (int e = 0; e < kVec; e += 4) {
        const f32x4 q = *reinterpret_cast<const f32x4 *>(out + r * kStride + (lane % kLanes) * kVec + e);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[e + k] = q[k];
      }
      if (row >= a.M) continue;
      store *p = c + row * ldc + col;
      if (vec) {
        store_vec<OUT, SPLIT>(p, s, a.alpha, a.beta);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (col + e < a.N) {
            if constexpr (SPLIT) p[e] = s[e];
            else store_c<OUT>(p + e, s[e], a.alpha, a.beta);
          }
      }
    }
    wave_order();
  }
}

// C <- alpha * (sum of the splits' partial sums, in ascending order) + beta * C.
template <int TYPE>
__global__ __launch_bounds__(256) void split_reduce_kernel(const float *__restrict__ ws,
                                                           typename Elem<TYPE>::store *__restrict__ C,
                                                           long long count, int N, int ldc, int splits,
                                                           float alpha, float beta) {
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < count; i += gridDim.x * 256LL) {
    float s = ws[i];
    for (int p = 1; p < splits; ++p) s += ws[p * count + i];
    const long long r = i / N;
    store_c<TYPE>(C + r * ldc + (i - r * N), s, alpha, beta);
  }
}

}  // namespace mx
}  // namespace gemm
