// A mixture-of-experts layer for a few tokens on microscaled weights, in two
// kernels (the operation is described in gemm.h at gemm_mx_moe):
//   up:    route, then for each reached expert G x and U x, a = w silu(Gx) Ux
//          into the workspace;
//   down:  route again, Y = sum over the reached experts of D a.
// Every workgroup works the routing out for itself from the logits (a few
// microseconds at most, and no third launch or hand-over between workgroups).
//
// Both products stream their weights from memory once, straight into
// registers: 16 weight rows are the rows of v_mfma_f32_16x16x32_bf16, 16 tokens
// its columns. A lane loads the 16 bytes of one row's block of 32 codes and
// that block's scale, and turns 8 codes at a time into bfloat16 (exact: e2m1
// has 2 bits of mantissa) for one instruction; which k an instruction's lane
// group carries is free as long as both operands agree, so lane group g takes
// block g of a row's 128 values.
// Activations keep their precision by being split into bfloat16 parts
// whose sum is exact: a bfloat16 is one part, a half two, a float three; the
// hidden activations (FP32 sums) are kept in two parts (16 bits) where the
// outputs are rounded to 16 bits or fewer, in three for FP32 outputs. The
// matrix instructions are far from the bound (the weights' bytes), so the
// parts cost nothing that shows.
#pragma once

#include "mx_kernels.hpp"

namespace gemm {
namespace mx {

constexpr int kMoeWaves = 8;
constexpr int kMoeThreads = 64 * kMoeWaves;
constexpr int kMaxTokens = 64, kMaxExperts = 512, kMaxTopK = 16;   // GEMM_MX_MOE_MAX_*
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kTokenTiles = kMaxTokens / 16;

template <int TYPE>
struct Parts {
  static constexpr int x = TYPE == kF32 ? 3 : TYPE == kF16 ? 2 : 1;   // of the inputs
  static constexpr int h = TYPE == kF32 ? 3 : 2;                      // of the hidden activations
};

struct MoeArgs {
  int tokens, hidden, inter, experts, top_k, renormalize;
  const float *logits;
  int ld_logits;
  const void *x;
  int ldx;
  const unsigned char *w1c, *w1s, *w2c, *w2s;
  void *y;
  int ldy;
  u16 *h;   // workspace: Parts<TYPE>::h planes of (tokens * top_k) x IP bfloat16
};

// What a workgroup knows after routing. Pairs (token, expert) are numbered by
// expert, then token; pair numbers index the rows of the hidden activations.
struct Routing {
  unsigned lo[kMaxExperts], hi[kMaxExperts];   // tokens that chose the expert, one bit each
  u16 base[kMaxExperts];                       // the expert's first pair
  u16 active[kMaxExperts];                     // reached experts, ascending
  unsigned char token[kMaxPairs];              // the pair's token
  float weight[kMaxPairs];                     // the pair's weight
  u16 chosen[kMaxTokens * kMaxTopK];           // token t's experts at t * kMaxTopK
  float chosen_weight[kMaxTokens * kMaxTopK];
  unsigned char count[kMaxTokens];             // how many it has
  unsigned nan_lo, nan_hi;                     // tokens whose logits hold a NaN or +inf
  int num_active;
};

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}
__device__ inline unsigned wave_max(unsigned v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2)
    v = max(v, static_cast<unsigned>(__shfl_xor(static_cast<int>(v), d)));
  return v;
}

// Routes all tokens; ends with a barrier. A wave takes a token at a time, its
// lanes the experts lane, lane + 64, ..: top_k rounds of a maximum over the
// wave. Logits are compared as whole numbers in their order (0: not to be
// chosen).
__device__ inline void route(const MoeArgs &a, Routing &r) {
  constexpr int kPer = kMaxExperts / 64;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = threadIdx.x; e < a.experts; e += kMoeThreads) r.lo[e] = r.hi[e] = 0;
  if (threadIdx.x == 0) r.nan_lo = r.nan_hi = 0;
  __syncthreads();
  for (int t = wave; t < a.tokens; t += kMoeWaves) {
    const float *l = a.logits + static_cast<long long>(t) * a.ld_logits;
    unsigned key[kPer];
    float val[kPer];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = j * 64 + lane;
      key[j] = 0;
      val[j] = -__builtin_inff();
      if (j * 64 < a.experts && e < a.experts) {
        val[j] = l[e] + 0.0f;   // -0 compares equal to +0
        const unsigned b = __builtin_bit_cast(unsigned, val[j]);
        if (magnitude_bits(val[j]) > 0x7f800000u || b == 0x7f800000u)
          bad = true;
        else if (b != 0xff800000u)
          key[j] = b & 0x80000000u ? ~b : b | 0x80000000u;
      }
    }
    if (__ballot(bad)) {
      if (lane == 0) {
        atomicOr(t < 32 ? &r.nan_lo : &r.nan_hi, 1u << (t & 31));
        r.count[t] = 0;
      }
      continue;
    }
    float top = 0.0f, all = 0.0f, some = 0.0f, mine = 0.0f;
    int n = 0, my_expert = 0;
    for (; n < a.top_k; ++n) {
      unsigned best = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j * 64 < a.experts) best = max(best, key[j]);
      best = wave_max(best);
      if (best == 0) break;
      const float logit =
          __builtin_bit_cast(float, best & 0x80000000u ? best & 0x7fffffffu : ~best);
      if (n == 0) {
        top = logit;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (j * 64 < a.experts) all += expf(val[j] - top);
        all = wave_sum(all);
      }
      int expert = -1;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (j * 64 < a.experts && expert < 0) {
          const unsigned long long who = __ballot(key[j] == best);
          if (who) {
            const int first = __builtin_ctzll(who);
            expert = j * 64 + first;
            if (lane == first) key[j] = 0;
          }
        }
      }
      const float p = expf(logit - top);
      some += p;
      if (lane == n) {
        mine = p;
        my_expert = expert;
      }
    }
    if (lane == 0) r.count[t] = static_cast<unsigned char>(n);
    if (lane < n) {
      r.chosen[t * kMaxTopK + lane] = static_cast<u16>(my_expert);
      r.chosen_weight[t * kMaxTopK + lane] = mine / (a.renormalize ? some : all);
      atomicOr(t < 32 ? &r.lo[my_expert] : &r.hi[my_expert], 1u << (t & 31));
    }
  }
  __syncthreads();
  if (wave == 0) {
    int pairs = 0, active = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < a.experts ? __popc(r.lo[e]) + __popc(r.hi[e]) : 0;
      int before = c;   // inclusive prefix sum over the lanes
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(before, d);
        if (lane >= d) before += o;
      }
      const unsigned long long who = __ballot(c > 0);
      if (e < a.experts) r.base[e] = static_cast<u16>(pairs + before - c);
      if (c > 0)
        r.active[active + __popcll(who & ((1ull << lane) - 1))] = static_cast<u16>(e);
      pairs += __shfl(before, 63);
      active += __popcll(who);
    }
    if (lane == 0) r.num_active = active;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * kMaxTopK; i += kMoeThreads) {
    const int t = i / kMaxTopK, n = i % kMaxTopK;
    if (n < r.count[t]) {
      const int e = r.chosen[i];
      const unsigned long long m = r.lo[e] | (static_cast<unsigned long long>(r.hi[e]) << 32);
      const int p = r.base[e] + __popcll(m & ((1ull << t) - 1));
      r.token[p] = static_cast<unsigned char>(t);
      r.weight[p] = r.chosen_weight[i];
    }
  }
  __syncthreads();
}

// 8 floats into PARTS bfloat16 vectors whose sum is exact for PARTS = 3 (and for
// fewer bits accordingly): each part is what is left, cut off after its 8 bits.
// Past an infinity nothing is left.
template <int PARTS>
__device__ inline void split8(const float (&v)[8], bf16x8 (&out)[PARTS]) {
  float rest[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rest[i] = v[i];
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    uintx4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned a = __builtin_bit_cast(unsigned, rest[2 * i]);
      const unsigned b = __builtin_bit_cast(unsigned, rest[2 * i + 1]);
      w[i] = (a >> 16) | (b & 0xffff0000u);
    }
    out[p] = __builtin_bit_cast(bf16x8, w);
    if (p + 1 < PARTS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float part =
            __builtin_bit_cast(float, __builtin_bit_cast(unsigned, rest[i]) & 0xffff0000u);
        rest[i] = __builtin_isinf(rest[i]) ? 0.0f : rest[i] - part;
      }
    }
  }
}

// 8 values of x at p (n of them in range) as bfloat16 parts.
template <int TYPE, bool VEC>
__device__ inline void load_x8(const typename Elem<TYPE>::store *p, int n,
                               bf16x8 (&out)[Parts<TYPE>::x]) {
  if constexpr (TYPE == kBf16) {
    if (VEC && n >= 8) {
      out[0] = *reinterpret_cast<const bf16x8 *>(p);
    } else {
      uintx4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (2 * i < n ? p[2 * i] : 0u) |
               (2 * i + 1 < n ? static_cast<unsigned>(p[2 * i + 1]) << 16 : 0u);
      out[0] = __builtin_bit_cast(bf16x8, w);
    }
  } else {
    float v[8];
    load8<TYPE, VEC>(p, n, v);
    split8<Parts<TYPE>::x>(v, out);
  }
}

// 8 codes under a scale as bfloat16.
__device__ inline bf16x8 weights8(unsigned codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Sums acc over the workgroup's waves into wave order through LDS: afterwards
// thread i < 64 * TILES holds the sum of lane i % 64's accumulators of tile i / 64.
template <int TILES>
__device__ inline f32x4 reduce_waves(const f32x4 (&acc)[TILES], int used, f32x4 *red) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int t = 0; t < TILES; ++t)
    if (t < used) red[(wave * TILES + t) * 64 + lane] = acc[t];
  __syncthreads();
  f32x4 s = {};
  if (wave < used) {
    s = red[wave * 64 + lane];
#pragma unroll
    for (int w = 1; w < kMoeWaves; ++w) s += red[(w * TILES + wave) * 64 + lane];
  }
  __syncthreads();
  return s;
}

template <int TYPE, bool VEC>
__global__ __launch_bounds__(kMoeThreads) void moe_up_kernel(MoeArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int PX = Parts<TYPE>::x, PH = Parts<TYPE>::h;
  __shared__ Routing r;
  __shared__ __attribute__((aligned(16))) f32x4 red[kMoeWaves * 2 * kTokenTiles * 64];
  route(a, r);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int HP = (a.hidden + kAlign - 1) / kAlign * kAlign;
  const int IP = (a.inter + kAlign - 1) / kAlign * kAlign;
  const int tiles = IP / 16;
  const long long plane = static_cast<long long>(a.tokens) * a.top_k * IP;
  const store *x = static_cast<const store *>(a.x);
  for (int item = blockIdx.x; item < r.num_active * tiles; item += gridDim.x) {
    const int ai = item / tiles;
    const int row0 = (item - ai * tiles) * 16;
    const int e = r.active[ai];
    const int base = r.base[e];
    const int count = __popc(r.lo[e]) + __popc(r.hi[e]);
    const int used = (count + 15) / 16;
    f32x4 acc[2 * kTokenTiles] = {};   // gate and up of each tile of 16 tokens
    if (row0 < a.inter) {
      const long long row = min(row0 + i16, a.inter - 1);
      const long long gate = static_cast<long long>(e) * 2 * a.inter + row, up = gate + a.inter;
      const unsigned char *gc = a.w1c + gate * (HP / 2) + g * 16, *gs = a.w1s + gate * (HP / 32) + g;
      const unsigned char *uc = a.w1c + up * (HP / 2) + g * 16, *us = a.w1s + up * (HP / 32) + g;
      for (int c = wave; c < HP / 128; c += kMoeWaves) {
        const uintx4 wg = *reinterpret_cast<const uintx4 *>(gc + c * 64);
        const uintx4 wu = *reinterpret_cast<const uintx4 *>(uc + c * 64);
        const float fg = scale_value(gs[c * 4]), fu = scale_value(us[c * 4]);
        const int k = c * 128 + g * 32;
#pragma unroll
        for (int t = 0; t < kTokenTiles; ++t) {
          if (t < used) {
            const int n = t * 16 + i16;
            const store *px = x + static_cast<long long>(n < count ? r.token[base + n] : 0) * a.ldx + k;
            const int left = n < count ? a.hidden - k : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              bf16x8 xv[PX];
              load_x8<TYPE, VEC>(px + j * 8, left - j * 8, xv);
              const bf16x8 vg = weights8(wg[j], fg), vu = weights8(wu[j], fu);
#pragma unroll
              for (int p = 0; p < PX; ++p) {
                acc[2 * t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vg, xv[p], acc[2 * t], 0, 0, 0);
                acc[2 * t + 1] =
                    __builtin_amdgcn_mfma_f32_16x16x32_bf16(vu, xv[p], acc[2 * t + 1], 0, 0, 0);
              }
            }
          }
        }
      }
    }
    // thread: tile wave / 2's gate (even waves) or up (odd waves) sums
    const f32x4 s = reduce_waves<2 * kTokenTiles>(acc, 2 * used, red);
    if (wave < 2 * used) red[wave * 64 + lane] = s;
    __syncthreads();
    if (wave < used) {
      const f32x4 gv = red[(2 * wave) * 64 + lane], uv = red[(2 * wave + 1) * 64 + lane];
      const int n = wave * 16 + i16;
      if (n < count) {
        const int p = base + n;
        const float w = r.weight[p];
        const int row = row0 + 4 * g;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          // past the last row of an expert: the zeros that pad `inter`
          float rest = row + v < a.inter ? gv[v] / (1.0f + expf(-gv[v])) * uv[v] * w : 0.0f;
#pragma unroll
          for (int q = 0; q < PH; ++q) {
            const unsigned b = __builtin_bit_cast(unsigned, rest);
            const u16 part = q + 1 < PH || PH == 3 ? static_cast<u16>(b >> 16) : Elem<kBf16>::put(rest);
            a.h[q * plane + static_cast<long long>(p) * IP + row + v] = part;
            rest = __builtin_isinf(rest) ? 0.0f : rest - Elem<kBf16>::get(part);
          }
        }
      }
    }
    __syncthreads();
  }
}

template <int TYPE>
__global__ __launch_bounds__(kMoeThreads) void moe_down_kernel(MoeArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int PH = Parts<TYPE>::h;
  __shared__ Routing r;
  __shared__ __attribute__((aligned(16))) f32x4 red[kMoeWaves * kTokenTiles * 64];
  route(a, r);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int IP = (a.inter + kAlign - 1) / kAlign * kAlign;
  const int chunks = IP / 128;
  const long long plane = static_cast<long long>(a.tokens) * a.top_k * IP;
  const int row0 = blockIdx.x * 16;
  const int row = min(row0 + i16, a.hidden - 1);
  const int token_tiles = (a.tokens + 15) / 16;
  f32x4 acc[kTokenTiles] = {};
  for (int s = wave; s < r.num_active * chunks; s += kMoeWaves) {
    const int ai = s / chunks, c = s - ai * chunks;
    const int e = r.active[ai];
    const long long wr = static_cast<long long>(e) * a.hidden + row;
    const uintx4 w = *reinterpret_cast<const uintx4 *>(a.w2c + wr * (IP / 2) + c * 64 + g * 16);
    const float f = scale_value(a.w2s[wr * (IP / 32) + c * 4 + g]);
    const unsigned long long m = r.lo[e] | (static_cast<unsigned long long>(r.hi[e]) << 32);
#pragma unroll
    for (int t = 0; t < kTokenTiles; ++t) {
      if (t < token_tiles && ((m >> (16 * t)) & 0xffffull)) {
        const int n = t * 16 + i16;
        const bool has = (m >> n) & 1;
        const int p = r.base[e] + __popcll(m & ((1ull << n) - 1));
        const u16 *h = a.h + static_cast<long long>(has ? p : 0) * IP + c * 128 + g * 32;
        f32x4 next = acc[t];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 v = weights8(w[j], f);
#pragma unroll
          for (int q = 0; q < PH; ++q) {
            bf16x8 hv = {};
            if (has) hv = *reinterpret_cast<const bf16x8 *>(h + q * plane + j * 8);
            next = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, hv, next, 0, 0, 0);
          }
        }
        // A token that did not choose this expert keeps its sum, also where the
        // expert's weights hold a NaN (0 * NaN is not 0).
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[t][v] = has ? next[v] : acc[t][v];
      }
    }
  }
  const f32x4 sum = reduce_waves<kTokenTiles>(acc, token_tiles, red);
  const int t = wave * 16 + i16;
  if (wave < token_tiles && t < a.tokens) {
    const bool nan = ((t < 32 ? r.nan_lo : r.nan_hi) >> (t & 31)) & 1;
    store *y = static_cast<store *>(a.y) + static_cast<long long>(t) * a.ldy + row0 + 4 * g;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (row0 + 4 * g + v < a.hidden)
        y[v] = Elem<TYPE>::put(nan ? __builtin_nanf("") : sum[v]);
  }
}

}  // namespace mx
}  // namespace gemm
