// Kernels on microscaled 4-bit operands (MXFP4: e2m1 numbers, an e8m0 scale for
// each 32 of them along K): conversion from and to float matrices, the product
// of two operands, and a mixture-of-experts layer for a few tokens. The formats
// and entry points are described in gemm.h.
#pragma once

#include <hip/hip_runtime.h>

namespace gemm {
namespace mx {

constexpr int kBlock = 32;    // values that share a scale
constexpr int kAlign = 128;   // a row's values are padded to a multiple of this

constexpr int kF32 = 0, kBf16 = 1, kF16 = 2;   // GEMM_TYPE_*

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef unsigned uintx2 __attribute__((ext_vector_type(2)));
typedef unsigned uintx4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned short u16;

// ---------------------------------------------------------------------------
// Element types.
template <int TYPE>
struct Elem;
template <>
struct Elem<kF32> {
  typedef float store;
  static __device__ inline float get(float v) { return v; }
  static __device__ inline float put(float v) { return v; }
};
template <>
struct Elem<kBf16> {
  typedef u16 store;
  static __device__ inline float get(u16 v) {
    return __builtin_bit_cast(float, static_cast<unsigned>(v) << 16);
  }
  static __device__ inline u16 put(float v) {
    return __builtin_bit_cast(u16, static_cast<__bf16>(v));   // nearest, ties to even
  }
};
template <>
struct Elem<kF16> {
  typedef u16 store;
  static __device__ inline float get(u16 v) {
    return static_cast<float>(__builtin_bit_cast(_Float16, v));
  }
  static __device__ inline u16 put(float v) {
    return __builtin_bit_cast(u16, static_cast<_Float16>(v));
  }
};

// 16 bytes at any element's address: the memory system takes loads and stores that
// are not aligned to their size.
typedef uintx4 uintx4_any __attribute__((aligned(2)));

// 8 consecutive values from p, the first `n` of them, zeros for the rest.
template <int TYPE>
__device__ inline void load8(const typename Elem<TYPE>::store *p, int n, float (&v)[8]) {
  if (n >= 8) {
    if constexpr (TYPE == kF32) {
      const uintx4 a = reinterpret_cast<const uintx4_any *>(p)[0];
      const uintx4 b = reinterpret_cast<const uintx4_any *>(p)[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned x = a[i], y = b[i];   // (the cast of a vector's element itself takes the first)
        v[i] = __builtin_bit_cast(float, x);
        v[4 + i] = __builtin_bit_cast(float, y);
      }
    } else {
      const uintx4 a = *reinterpret_cast<const uintx4_any *>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = Elem<TYPE>::get(static_cast<u16>(a[i]));
        v[2 * i + 1] = Elem<TYPE>::get(static_cast<u16>(a[i] >> 16));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? Elem<TYPE>::get(p[i]) : 0.0f;
  }
}

template <int TYPE>
__device__ inline void store8(typename Elem<TYPE>::store *p, int n, const float (&v)[8]) {
  if (n >= 8) {
    if constexpr (TYPE == kF32) {
      uintx4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __builtin_bit_cast(unsigned, v[i]);
        b[i] = __builtin_bit_cast(unsigned, v[4 + i]);
      }
      reinterpret_cast<uintx4_any *>(p)[0] = a;
      reinterpret_cast<uintx4_any *>(p)[1] = b;
    } else {
      uintx4 a;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[i] = Elem<TYPE>::put(v[2 * i]) | (static_cast<unsigned>(Elem<TYPE>::put(v[2 * i + 1])) << 16);
      *reinterpret_cast<uintx4_any *>(p) = a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = Elem<TYPE>::put(v[i]);
  }
}

// Order between the LDS accesses of a wave's lanes: LDS serves them in order, so only
// the compiler has to keep them.
__device__ inline void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------------------
// The e8m0 scale of a block and its values.

// Scale byte of a block whose largest magnitude has these FP32 bits: the
// exponent of 2^(floor(log2 max) - 2), so that the maximum falls into [4, 8)
// where e2m1 ends (6); 255 for an infinity or a NaN (as bits, both lie above
// every finite number).
__device__ inline unsigned scale_byte(unsigned max_bits) {
  const unsigned e = max_bits >> 23;
  return e == 255 ? 255u : (e < 2 ? 0u : e - 2);
}
// 1 / scale as a float; the byte is at most 252 here, so it is normal.
__device__ inline float inverse_scale(unsigned byte) {
  return __builtin_bit_cast(float, (254u - byte) << 23);
}
// The scale as a float: 2^-127 is subnormal, 255 is NaN.
__device__ inline float scale_value(unsigned byte) {
  const unsigned bits = byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23;
  return __builtin_bit_cast(float, bits);
}
__device__ inline unsigned magnitude_bits(float v) {
  return __builtin_bit_cast(unsigned, v) & 0x7fffffffu;
}

// 8 values times 1 / scale -> 8 codes, the first in the low bits. The
// instruction rounds to nearest, ties to even, and saturates at 6.
__device__ inline unsigned encode8(const float (&v)[8], float inv) {
  unsigned r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * inv, v[1] * inv, 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * inv, v[3] * inv, 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * inv, v[5] * inv, 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * inv, v[7] * inv, 1.0f, 3);
  return r;
}
__device__ inline void decode8(unsigned codes, float scale, float (&v)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
  v[0] = a[0] * scale; v[1] = a[1] * scale;
  v[2] = b[0] * scale; v[3] = b[1] * scale;
  v[4] = c[0] * scale; v[5] = c[1] * scale;
  v[6] = d[0] * scale; v[7] = d[1] * scale;
}

// ---------------------------------------------------------------------------
// Rows of 8-value chunks over workgroups of 256 threads: 2^tpr_log2 threads
// (16 to 256) side by side along a row, so 256 >> tpr_log2 rows a pass, and
// PASSES passes. Workgroups run over the column groups first.
struct RowMap {
  int tpr_log2;
  int col_groups;
};
constexpr int kRowPasses = 4;

// Quantisation along the stored rows. A block of 32 is 4 neighbouring lanes: the
// maximum crosses them in two cross-lane steps, each lane writes its 4 bytes of
// codes. Bound by memory: 8192 x 8192 bfloat16 (134 MB in, 36 MB out) takes 42 us,
// 4.1 TB/s where a large copy reaches 4.9.
template <int TYPE>
__global__ __launch_bounds__(256) void quantize_rows_kernel(
    const typename Elem<TYPE>::store *__restrict__ X, int ldx, unsigned *__restrict__ codes,
    unsigned char *__restrict__ scales, int rows, int K, int KP, RowMap map) {
  const int group = blockIdx.x / map.col_groups;
  const int tpr = 1 << map.tpr_log2;
  const int chunk = (blockIdx.x - group * map.col_groups) * tpr + (threadIdx.x & (tpr - 1));
  const int rows_pass = 256 >> map.tpr_log2;
  const int k = chunk * 8;
  if (k >= KP) return;   // whole blocks of lanes: KP is a multiple of 128
  const long long row0 =
      static_cast<long long>(group) * (rows_pass * kRowPasses) + (threadIdx.x >> map.tpr_log2);
  float v[kRowPasses][8];
#pragma unroll
  for (int p = 0; p < kRowPasses; ++p) {
    const long long row = row0 + p * rows_pass;
    load8<TYPE>(X + row * ldx + k, row < rows ? K - k : 0, v[p]);
  }
#pragma unroll
  for (int p = 0; p < kRowPasses; ++p) {
    const long long row = row0 + p * rows_pass;
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, magnitude_bits(v[p][i]));
    m = max(m, static_cast<unsigned>(__shfl_xor(static_cast<int>(m), 1)));
    m = max(m, static_cast<unsigned>(__shfl_xor(static_cast<int>(m), 2)));
    const unsigned s = scale_byte(m);
    const unsigned c = s == 255 ? 0u : encode8(v[p], inverse_scale(s));
    if (row < rows) {
      codes[row * (KP / 8) + chunk] = c;
      if ((chunk & 3) == 0) scales[row * (KP / 32) + (chunk >> 2)] = static_cast<unsigned char>(s);
    }
  }
}

template <int TYPE>
__global__ __launch_bounds__(256) void dequantize_rows_kernel(
    const unsigned *__restrict__ codes, const unsigned char *__restrict__ scales,
    typename Elem<TYPE>::store *__restrict__ Y, int ldy, int rows, int K, int KP, RowMap map) {
  const int group = blockIdx.x / map.col_groups;
  const int tpr = 1 << map.tpr_log2;
  const int chunk = (blockIdx.x - group * map.col_groups) * tpr + (threadIdx.x & (tpr - 1));
  const int rows_pass = 256 >> map.tpr_log2;
  const int k = chunk * 8;
  if (k >= K) return;
  const long long row0 =
      static_cast<long long>(group) * (rows_pass * kRowPasses) + (threadIdx.x >> map.tpr_log2);
  unsigned c[kRowPasses], s[kRowPasses];
#pragma unroll
  for (int p = 0; p < kRowPasses; ++p) {
    const long long row = row0 + p * rows_pass;
    c[p] = row < rows ? codes[row * (KP / 8) + chunk] : 0u;
    s[p] = row < rows ? scales[row * (KP / 32) + (chunk >> 2)] : 0u;
  }
#pragma unroll
  for (int p = 0; p < kRowPasses; ++p) {
    const long long row = row0 + p * rows_pass;
    if (row >= rows) continue;
    float v[8];
    decode8(c[p], scale_value(s[p]), v);
    store8<TYPE>(Y + row * ldy + k, K - k, v);
  }
}

// ---------------------------------------------------------------------------
// Quantisation across the stored rows (the operand's rows are X's columns): a
// workgroup of 8 waves takes 128 operand rows by 256 values of K, a wave one block
// of 32 of each row. Lanes run along the stored rows, two neighbouring values a
// lane (256 bytes and more a load), and a lane collects the 32 values of its two
// blocks itself; the codes pass through LDS so that each operand row is
// written in runs of 64 or 128 bytes. Bound by memory latency: all 32 loads of a
// lane are in flight at once. 4097 x 4095 FP32 (67 MB in, 9 MB out) takes 28 us.
// With one value a lane and 4 waves a tile, 4096 x 4096 bfloat16 took 36 us, so
// 15.
constexpr int kColWaves = 8;
constexpr int kColThreads = 64 * kColWaves;
constexpr int kColK = kColWaves * kBlock;   // values of K of a tile
constexpr int kColStride = 36;              // LDS words of a row's 128 code bytes, padded

constexpr int kColRows = 128;               // operand rows of a tile

// Two neighbouring elements as loaded or to be stored, at any element's address.
template <int TYPE>
struct Neighbours {
  typename Elem<TYPE>::store e[2];
};

template <int TYPE>
__global__ __launch_bounds__(kColThreads) void quantize_columns_kernel(
    const typename Elem<TYPE>::store *__restrict__ X, int ldx, unsigned *__restrict__ codes,
    unsigned *__restrict__ scales, int rows, int K, int KP, int k_tiles) {
  constexpr int VEC = 2, kRows = kColRows;
  __shared__ __attribute__((aligned(16))) unsigned tile[kRows * kColStride];
  __shared__ __attribute__((aligned(4))) unsigned char tile_scales[kRows * 8];
  const int rt = blockIdx.x / k_tiles;
  const int k0 = (blockIdx.x - rt * k_tiles) * kColK;
  const long long r0 = static_cast<long long>(rt) * kRows;
  const int lane = threadIdx.x & 63, b = threadIdx.x >> 6;
  const int kb = k0 + b * kBlock;
  const bool both = r0 + lane * VEC + 1 < rows, one = r0 + lane * VEC < rows;
  if (kb < KP) {
    typedef Neighbours<TYPE> Pair;
    const typename Elem<TYPE>::store *p = X + static_cast<long long>(kb) * ldx + r0 + lane * VEC;
    Pair raw[kBlock] = {};
    if (both && kb + kBlock <= K) {
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        raw[i] = *reinterpret_cast<const Pair *>(p + static_cast<long long>(i) * ldx);
    } else if (one) {
#pragma unroll
      for (int i = 0; i < kBlock; ++i)
        if (kb + i < K) {
          raw[i].e[0] = p[static_cast<long long>(i) * ldx];
          if (both) raw[i].e[1] = p[static_cast<long long>(i) * ldx + 1];
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      unsigned m = 0;
      float v[4][8];
#pragma unroll
      for (int i = 0; i < kBlock; ++i) {
        v[i / 8][i % 8] = Elem<TYPE>::get(raw[i].e[e]);
        m = max(m, magnitude_bits(v[i / 8][i % 8]));
      }
      const unsigned s = scale_byte(m);
      uintx4 c;
#pragma unroll
      for (int q = 0; q < 4; ++q) c[q] = s == 255 ? 0u : encode8(v[q], inverse_scale(s));
      const int row = lane * VEC + e;
      *reinterpret_cast<uintx4 *>(&tile[row * kColStride + b * 4]) = c;
      tile_scales[row * 8 + b] = static_cast<unsigned char>(s);
    }
  }
  __syncthreads();
  const int words = min(kColK, KP - k0) / 8;   // code words of a row here: 16 or 32
#pragma unroll
  for (int i = 0; i < kRows * 8 / kColThreads; ++i) {
    const int e = threadIdx.x + kColThreads * i;
    const int r = e >> 3, w = (e & 7) * 4;
    if (r0 + r < rows && w < words)
      *reinterpret_cast<uintx4 *>(codes + (r0 + r) * (KP / 8) + k0 / 8 + w) =
          *reinterpret_cast<const uintx4 *>(&tile[r * kColStride + w]);
  }
  if (threadIdx.x < kRows * 2) {
    const int r = threadIdx.x >> 1, w = threadIdx.x & 1;
    if (r0 + r < rows && w * 16 < words)
      scales[(r0 + r) * (KP / 128) + k0 / 128 + w] =
          reinterpret_cast<const unsigned *>(tile_scales)[r * 2 + w];
  }
}

// The way back, the same tiles.
template <int TYPE>
__global__ __launch_bounds__(kColThreads) void dequantize_columns_kernel(
    const unsigned *__restrict__ codes, const unsigned char *__restrict__ scales,
    typename Elem<TYPE>::store *__restrict__ Y, int ldy, int rows, int K, int KP, int k_tiles) {
  constexpr int VEC = 2, kRows = kColRows;
  __shared__ __attribute__((aligned(16))) unsigned tile[kRows * kColStride];
  const int rt = blockIdx.x / k_tiles;
  const int k0 = (blockIdx.x - rt * k_tiles) * kColK;
  const long long r0 = static_cast<long long>(rt) * kRows;
  const int words = min(kColK, KP - k0) / 8;
#pragma unroll
  for (int i = 0; i < kRows * 8 / kColThreads; ++i) {
    const int e = threadIdx.x + kColThreads * i;
    const int r = e >> 3, w = (e & 7) * 4;
    if (r0 + r < rows && w < words)
      *reinterpret_cast<uintx4 *>(&tile[r * kColStride + w]) =
          *reinterpret_cast<const uintx4 *>(codes + (r0 + r) * (KP / 8) + k0 / 8 + w);
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, b = threadIdx.x >> 6;
  const int kb = k0 + b * kBlock;
  const long long row = r0 + lane * VEC;
  if (row >= rows || kb >= K) return;
  const bool both = row + 1 < rows;
  uintx4 c[VEC];
  float s[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    c[e] = *reinterpret_cast<const uintx4 *>(&tile[(lane * VEC + e) * kColStride + b * 4]);
    s[e] = scale_value(scales[min(row + e, rows - 1LL) * (KP / 32) + kb / 32]);
  }
  typedef Neighbours<TYPE> Pair;
  typename Elem<TYPE>::store *p = Y + static_cast<long long>(kb) * ldy + row;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[VEC][8];
#pragma unroll
    for (int e = 0; e < VEC; ++e) decode8(c[e][q], s[e], v[e]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      Pair out;
#pragma unroll
      for (int e = 0; e < VEC; ++e) out.e[e] = Elem<TYPE>::put(v[e][i]);
      if (kb + 8 * q + i < K) {
        if (both)
          *reinterpret_cast<Pair *>(p + static_cast<long long>(8 * q + i) * ldy) = out;
        else
          p[static_cast<long long>(8 * q + i) * ldy] = out.e[0];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Product.

// C <- alpha * sum + beta * C for one element; beta * c is rounded on its own
// and c not read when beta == 0, as in the FP32 general form.
template <int TYPE>
__device__ inline void store_c(typename Elem<TYPE>::store *c, float sum, float alpha, float beta) {
  const float r = beta == 0.0f ? alpha * sum : fmaf(alpha, sum, beta * Elem<TYPE>::get(*c));
  *c = Elem<TYPE>::put(r);
}

__device__ inline intx8 widen(const intx4 v) { return intx8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// A few rows of A (up to 16 * MT: a decoding step) by all rows of B. Bound by B's
// bytes, which are read once, straight from memory into registers: a workgroup
// takes 16 rows of B (its instructions' rows; A's rows are the columns), its 8
// waves share K, a wave taking kSkinnyAt neighbouring chunks of 128 at a time.
// The waves' sums are added in order. 1 x 4096 x 4096 (8.9 MB, other weights every
// call) takes 4.8 us, half of it the launch; the tiled kernel with 4 splits and
// their sum takes 2.2 us more.
constexpr int kSkinnyWaves = 8, kSkinnyAt = 4;

template <int TYPE, int MT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(
    const unsigned char *__restrict__ ac, const unsigned char *__restrict__ as,
    const unsigned char *__restrict__ bc, const unsigned char *__restrict__ bs,
    typename Elem<TYPE>::store *__restrict__ C, int M, int N, int KP, int ldc, float alpha,
    float beta) {
  __shared__ __attribute__((aligned(16))) f32x4 red[kSkinnyWaves * MT * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const long long code_row = KP / 2, scale_row = KP / 32;
  // Rows past the last: the last one again, not stored.
  const long long rb = min(n0 + i, N - 1);
  const unsigned char *pb = bc + rb * code_row + g * 16, *sb = bs + rb * scale_row + g;
  const unsigned char *pa[MT], *sa[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const long long ra = min(t * 16 + i, M - 1);
    pa[t] = ac + ra * code_row + g * 16;
    sa[t] = as + ra * scale_row + g;
  }
  f32x4 acc[MT] = {};
  const int steps = KP / 128;
  for (int s0 = wave * kSkinnyAt; s0 < steps; s0 += kSkinnyWaves * kSkinnyAt) {
    intx4 b[kSkinnyAt], a[MT][kSkinnyAt];
    int fb[kSkinnyAt], fa[MT][kSkinnyAt];
#pragma unroll
    for (int u = 0; u < kSkinnyAt; ++u) {
      const int s = min(s0 + u, steps - 1);   // past the end: the last one again, not used
      b[u] = *reinterpret_cast<const intx4 *>(pb + s * 64);
      fb[u] = sb[s * 4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        a[t][u] = *reinterpret_cast<const intx4 *>(pa[t] + s * 64);
        fa[t][u] = sa[t][s * 4];
      }
    }
#pragma unroll
    for (int u = 0; u < kSkinnyAt; ++u) {
      if (s0 + u < steps) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
          acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(widen(b[u]), widen(a[t][u]), acc[t],
                                                                    4, 4, 0, fb[u], 0, fa[t][u]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) red[(wave * MT + t) * 64 + lane] = acc[t];
  __syncthreads();
  if (wave < MT) {
    f32x4 s = red[wave * 64 + lane];
#pragma unroll
    for (int w = 1; w < kSkinnyWaves; ++w) s += red[(w * MT + wave) * 64 + lane];
    const int m = wave * 16 + i;
    if (m < M) {
      typename Elem<TYPE>::store *c = C + static_cast<long long>(m) * ldc + n0 + 4 * g;
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (n0 + 4 * g + v < N) store_c<TYPE>(c + v, s[v], alpha, beta);
    }
  }
}

// C <- beta * C.
template <int TYPE>
__global__ __launch_bounds__(256) void scale_kernel(typename Elem<TYPE>::store *__restrict__ C,
                                                    long long count, int N, int ldc, float beta) {
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < count; i += gridDim.x * 256LL) {
    const long long r = i / N;
    typename Elem<TYPE>::store *c = C + r * ldc + (i - r * N);
    *c = Elem<TYPE>::put(beta == 0.0f ? 0.0f : beta * Elem<TYPE>::get(*c));
  }
}

}  // namespace mx
}  // namespace gemm
