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
// a stage is 256 values of K, 128 bytes a row (a whole line: with half lines the L2
// cache serves as many requests for half the bytes), copied straight into LDS (16
// bytes a lane) through a ring of NS = 2 or 4 stages. Within a stage row x keeps its
// 16-byte chunk c (one block of 32 values) at c ^ ((x >> 1) & 7): 16 consecutive
// rows of one chunk, which 16 lanes read at a time, then meet every bank once. The
// scales of 2 stages (16 bytes a row) go through a ring of their own.
//
// A stage is four steps of 64 values: lane (h, i) of an instruction holds block
// 2 * step + h of row i. The registers of one step are read from LDS while the
// instructions of the step before run. The wait for the next stage's copies and
// the workgroup's barrier stand in a stage's last step, when all of the stage has
// been read; the stage is then refilled, NS stages ahead. Where the K range is an
// odd number of 128s its last two steps stand alone behind the loop.
//
// Rows past M or N and stages past the K range are outside the copies' buffer
// ranges and read as zeros (a zero scale byte is 2^-127, not NaN).
//
// 8192^3 with 256 x 256 tiles takes 292 to 306 us from chip to chip (3.8 to 3.6 PFLOP/s):
// 571,000 cycles a CU, in 46% of which the matrix pipe is busy, at a mean 1.9 GHz of 2.4. Its
// instructions in a loop of their own take 173 us on random operands (6.36 PFLOP/s)
// and 122 on constant ones (9.0): the difference is power. The cycles beside them
// are what feeds them: with stages of 128 values of K, when it took 305 us, this
// kernel without its copies, reads and stores took 195, the copies added 70, the LDS
// reads 33, and of a tile's 76 us 10 were its start and end. 4096^3 (46 to 51 us, one tile a
// CU): 95,000 cycles, the pipe busy in 34%, at 1.9 to 2.1 GHz.
// Smaller tiles are bound by what a CU gets from the L2 cache, about 10 TB/s for the
// chip in half lines: 4096^3 with 128 x 128 tiles took 54 us, in whole lines 46.
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

template <int BM, int BN, int NS>
struct TileShape {
  static constexpr int FM = BM / 64, FN = BN / 64;        // 32 x 32 blocks of a wave (2 x 2 waves)
  static constexpr int kStage = (BM + BN) * 128;          // bytes of codes of a stage
  static constexpr int kScales = (BM + BN) * 16;          // bytes of scales of a pair of stages
  static constexpr int kAhead = NS / 2;                   // pairs of stages that the scales run ahead
  static constexpr int kPairs = NS;                       // and that are kept
  static constexpr int kLds = NS * kStage + kPairs * kScales;
  static constexpr int kCopies = kStage / 4096;           // a wave's copies of a stage
  static constexpr int kScaleCopies = (kScales + 4095) / 4096;
};

template <int BM, int BN, int NS, int TYPE, bool SPLIT, int WPE>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(WPE, WPE)))
void tile_kernel(TileArgs a) {
  using S = TileShape<BM, BN, NS>;
  constexpr int FM = S::FM, FN = S::FN;
  __shared__ __attribute__((aligned(1024))) unsigned char lds[S::kLds];

  const TileCoord tc = map_tile(blockIdx.x, a.tiles_m, a.tiles_n, a.splits, kGroupM);
  const int m0 = __builtin_amdgcn_readfirstlane(tc.tm) * BM;
  const int n0 = __builtin_amdgcn_readfirstlane(tc.tn) * BN;
  const int split = __builtin_amdgcn_readfirstlane(tc.split);
  const int k0 = split * a.k_chunk;
  const int halves = (min(a.KP, k0 + a.k_chunk) - k0) / 128;
  const int stages = (halves + 1) / 2, whole = halves / 2;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 31, h = lane >> 5;
  const int wm = wave >> 1, wn = wave & 1;

  // Copies. Instruction q of a stage fills rows 8q .. 8q + 7 (A's rows, then B's), 8
  // lanes a row; wave w takes q = w, w + 4, .. (so the row's bit 3 is the wave's bit 0).
  const long long code_row = a.KP / 2, scale_row = a.KP / 32;
  const u32x4 ra = make_buffer_rsrc(a.ac + m0 * code_row + k0 / 2, (a.M - m0) * code_row - k0 / 2);
  const u32x4 rb = make_buffer_rsrc(a.bc + n0 * code_row + k0 / 2, (a.N - n0) * code_row - k0 / 2);
  const u32x4 rsa = make_buffer_rsrc(a.as + m0 * scale_row + k0 / 32, (a.M - m0) * scale_row - k0 / 32);
  const u32x4 rsb = make_buffer_rsrc(a.bs + n0 * scale_row + k0 / 32, (a.N - n0) * scale_row - k0 / 32);
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(lds));
  const unsigned lane_off = static_cast<unsigned>((lane >> 3) * code_row) +
                            static_cast<unsigned>(((lane & 7) ^ ((wave & 1) * 4 + (lane >> 4))) * 16);
  auto copy_codes = [&](int q4, int stage, int base) {
    const int q = wave + 4 * q4;   // q4 is a constant, so is the operand (BM, BN multiples of 64)
    const bool of_a = q4 * 32 < BM;
    const unsigned row = static_cast<unsigned>(of_a ? q * 8 : q * 8 - BM);
    const unsigned so = stage < stages ? static_cast<unsigned>(stage) * 128u : kOutOfRange;
    dma_copy<4>(of_a ? ra : rb, lane_off + row * static_cast<unsigned>(code_row) + so,
                lds0 + base + q * 1024);
  };
  // Instruction q of a pair of stages' scales fills rows 64q .. 64q + 63, a lane a row.
  auto copy_scales = [&](int q4, int pair) {
    const int q = wave + 4 * q4;
    if (S::kScales % 4096 == 0 || q * 1024 < S::kScales) {
      const bool of_a = q * 64 < BM;
      const unsigned row = static_cast<unsigned>(of_a ? q * 64 : q * 64 - BM) + lane;
      const unsigned so = pair * 2 < stages ? static_cast<unsigned>(pair) * 16u : kOutOfRange;
      dma_copy<4>(of_a ? rsa : rsb, row * static_cast<unsigned>(scale_row) + so,
                  lds0 + NS * S::kStage + (pair & (S::kPairs - 1)) * S::kScales + q * 1024);
    }
  };

  // Operand registers of a step (two sets in turn); scales of a stage, as read and
  // shifted so that the lane's byte of step s is byte 2 (s % 2) of word s / 2.
  intx4 fa[2][FM], fb[2][FN];
  uintx2 sa[FM], sb[FN], sa_raw[FM], sb_raw[FN];
  const int off0 = i * 128 + ((h ^ ((i >> 1) & 7)) * 16);
  const unsigned char *la = lds + wm * (BM / 2) * 128, *lb = lds + (BM + wn * (BN / 2)) * 128;
  const unsigned char *lsa = lds + NS * S::kStage + (wm * (BM / 2) + i) * 16;
  const unsigned char *lsb = lds + NS * S::kStage + (BM + wn * (BN / 2) + i) * 16;
  auto read_a = [&](int f, int base, int step) {
    fa[step & 1][f] = *reinterpret_cast<const intx4 *>(la + base + f * 4096 + (off0 ^ (step * 32)));
  };
  auto read_b = [&](int f, int base, int step) {
    fb[step & 1][f] = *reinterpret_cast<const intx4 *>(lb + base + f * 4096 + (off0 ^ (step * 32)));
  };
  auto read_scales = [&](int stage) {
    const int at = ((stage >> 1) & (S::kPairs - 1)) * S::kScales + (stage & 1) * 8;
#pragma unroll
    for (int f = 0; f < FM; ++f) sa_raw[f] = *reinterpret_cast<const uintx2 *>(lsa + at + f * 512);
#pragma unroll
    for (int f = 0; f < FN; ++f) sb_raw[f] = *reinterpret_cast<const uintx2 *>(lsb + at + f * 512);
  };
  auto shift_scales = [&]() {
#pragma unroll
    for (int f = 0; f < FM; ++f) sa[f] = sa_raw[f] >> static_cast<unsigned>(8 * h);
#pragma unroll
    for (int f = 0; f < FN; ++f) sb[f] = sb_raw[f] >> static_cast<unsigned>(8 * h);
  };

  f32x16 acc[FM][FN] = {};

  // Prologue: the first NS stages and their scales on their way.
#pragma unroll
  for (int f = 0; f < S::kAhead; ++f)
#pragma unroll
    for (int q = 0; q < S::kScaleCopies; ++q) copy_scales(q, f);
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int q = 0; q < S::kCopies; ++q) copy_codes(q, s, s * S::kStage);
  wait_vmcnt<(NS - 1) * S::kCopies>();
  asm volatile("s_barrier" : : : "memory");
#pragma unroll
  for (int f = 0; f < FM; ++f) read_a(f, 0, 0);
#pragma unroll
  for (int f = 0; f < FN; ++f) read_b(f, 0, 0);
  read_scales(0);

  constexpr int kMfmas = FM * FN;
  // Instruction n of a step.
  auto mfma = [&](auto step_c, auto n_c) __attribute__((always_inline)) {
    constexpr int step = decltype(step_c)::value, n = decltype(n_c)::value;
    constexpr int fm = n / FN, fn = n % FN;
    const int wa = static_cast<int>(sa[fm][step / 2]), wb = static_cast<int>(sb[fn][step / 2]);
    acc[fm][fn] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        widen(fb[step & 1][fn]), widen(fa[step & 1][fm]), acc[fm][fn], 4, 4, 2 * (step & 1), wb,
        2 * (step & 1), wa);
  };
  // The instructions of a step, the next step's registers read meanwhile.
  auto step_and_read = [&](auto step_c, int base) __attribute__((always_inline)) {
    constexpr int step = decltype(step_c)::value;
    unroll_steps<0, kMfmas>([&](auto n_c) {
      constexpr int n = decltype(n_c)::value;
      mfma(step_c, n_c);
      if constexpr (n < FM) read_a(n, base, step + 1);
      else if constexpr (n < FM + FN) read_b(n - FM, base, step + 1);
      if constexpr (n == kMfmas - 1 && FM + FN > kMfmas) {
#pragma unroll
        for (int f = kMfmas; f < FM + FN; ++f) read_b(f - FM, base, step + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  for (int t = 0; t < whole; ++t) {
    const int base = (t & (NS - 1)) * S::kStage, next = ((t + 1) & (NS - 1)) * S::kStage;
    // The scales of a pair of stages that starts NS later, into room whose scales have
    // all been read before the last barrier. A branch after the instructions below
    // would let the compiler move all of them behind it.
    if ((t & 1) == 0) {
#pragma unroll
      for (int q = 0; q < S::kScaleCopies; ++q) copy_scales(q, (t >> 1) + S::kAhead);
    }
    shift_scales();
    step_and_read(std::integral_constant<int, 0>(), base);
    step_and_read(std::integral_constant<int, 1>(), base);
    step_and_read(std::integral_constant<int, 2>(), base);
    constexpr int kBefore = kMfmas / 4;
    unroll_steps<0, kMfmas>([&](auto n_c) {
      constexpr int n = decltype(n_c)::value;
      if constexpr (n == kBefore) {
        // all of this stage is read, the next one's copies have landed
        wait_vmcnt<(NS - 2) * S::kCopies>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
      mfma(std::integral_constant<int, 3>(), n_c);
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
  if (whole < stages) {   // half a stage: two steps
    shift_scales();
    step_and_read(std::integral_constant<int, 0>(), (whole & (NS - 1)) * S::kStage);
    unroll_steps<0, kMfmas>([&](auto n_c) { mfma(std::integral_constant<int, 1>(), n_c); });
  }
  wait_vmcnt<0>();   // no copy may land after the workgroup's LDS is another's

  // B's rows are the instructions' rows: accumulator v of lane (h, i) is row i of C
  // and column 8 (v / 4) + 4 h + v % 4 of a block, four neighbouring columns at a
  // time. 32 rows of the wave's tile pass through its own piece of LDS and leave
  // as whole rows, 16 bytes a lane (each lane storing what it holds, a few bytes
  // to each of 32 rows, took 14 us for a 256 x 256 tile, this 2 us).
  // Everybody has read the last stage.
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory");
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
