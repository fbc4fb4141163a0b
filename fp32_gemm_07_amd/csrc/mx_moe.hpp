// A mixture-of-experts layer for a few tokens on microscaled weights, in two
// kernels (the operation is described in gemm.h at gemm_mx_moe):
//   up:    route, then for each reached expert G x and U x, a = w silu(Gx) Ux
//          into the workspace;
//   down:  Y = sum over the reached experts of D a.
// Every workgroup of the first kernel works the routing out for itself from the
// logits (a few microseconds at most, and no third launch or hand-over between
// workgroups); one of them leaves the list of reached experts for the second.
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
constexpr int kDownWaves = 16;   // of the second kernel
constexpr int kDownThreads = 64 * kDownWaves;
constexpr int kMaxTokens = 64, kMaxExperts = 512, kMaxTopK = 16;   // GEMM_MX_MOE_MAX_*
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kTokenTiles = kMaxTokens / 16;
constexpr int kUpTiles = 2;   // tiles of 16 tokens that the first kernel takes at a time

template <int TYPE>
struct Parts {
  static constexpr int x = TYPE == kF32 ? 3 : TYPE == kF16 ? 2 : 1;   // of the inputs
  static constexpr int h = TYPE == kF32 ? 3 : 2;                      // of the hidden activations
};

// A reached expert: its number, the tokens that chose it (one bit each) and its
// first pair. Pairs (token, expert) are numbered by expert, then token; pair
// numbers index the rows of the hidden activations. Entry 0 of the workspace's
// list holds how many follow and the tokens whose logits hold a NaN or +inf.
struct Reached {
  unsigned expert_base;   // expert in the low, first pair in the high half
  unsigned lo, hi;
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
  u16 *h;       // workspace: Parts<TYPE>::h planes of (tokens * top_k) x IP bfloat16,
  Reached *reached;   // and what the second kernel needs of the routing
};

// What a workgroup knows after routing.
struct Routing {
  Reached reached[kMaxExperts];     // reached experts, ascending
  float weight[kMaxPairs];          // the pair's weight
  unsigned char token[kMaxPairs];   // the pair's token
  unsigned nan_lo, nan_hi;          // tokens whose logits hold a NaN or +inf
  int num_reached;
};
// What it needs on the way there.
struct RoutingScratch {
  unsigned lo[kMaxExperts], hi[kMaxExperts];   // tokens that chose the expert, one bit each
  u16 base[kMaxExperts];                       // the expert's first pair
  u16 chosen[kMaxTokens * kMaxTopK];           // token t's experts at t * kMaxTopK, 0xffff: none
  float chosen_weight[kMaxTokens * kMaxTopK];
};

template <int CTRL, int ROWS>
__device__ inline int dpp(int identity, int v) {
  return __builtin_amdgcn_update_dpp(identity, v, CTRL, ROWS, 0xf, false);
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

// The choice of 4 tokens, one to each row of 16 lanes, whose lanes hold the
// experts l, l + 16, ..: top_k rounds of a maximum over the row. Logits are
// compared as whole numbers in their order (0: not to be chosen).
template <int PER>
__device__ inline void choose(const MoeArgs &a, int t, Routing &r, RoutingScratch &s) {
  const int l16 = threadIdx.x & 15;
  const bool ok = t < a.tokens;
  const float *l = a.logits + static_cast<long long>(ok ? t : 0) * a.ld_logits;
  float val[PER];
  unsigned key[PER];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = j * 16 + l16;
    val[j] = ok && e < a.experts ? l[e] + 0.0f : -__builtin_inff();   // -0 equals +0
  }
  unsigned best = 0;
  int at = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const unsigned b = __builtin_bit_cast(unsigned, val[j]);
    if (magnitude_bits(val[j]) > 0x7f800000u || b == 0x7f800000u) bad = true;
    key[j] = b == 0xff800000u ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
    if (key[j] > best) {
      best = key[j];
      at = j;
    }
  }
  bad = row_max(bad) != 0;
  float top = 0.0f, mine = -__builtin_inff();
  int my_expert = 0xffff;
  for (int n = 0; n < a.top_k; ++n) {
    const unsigned most = row_max(best);
    const int expert = row_min(best == most ? at * 16 + l16 : kMaxExperts);
    const bool some = most != 0 && !bad;
    const float logit = __builtin_bit_cast(float, most & 0x80000000u ? most & 0x7fffffffu : ~most);
    if (n == 0) top = logit;
    if (l16 == n && some) {
      mine = logit;
      my_expert = expert;
    }
    if (expert == at * 16 + l16) {   // its lane looks for its next
      const int gone = at;
      best = 0;
      at = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (j == gone) key[j] = 0;
        if (key[j] > best) {
          best = key[j];
          at = j;
        }
      }
    }
  }
  // softmax: lane n < top_k has the n-th chosen logit, -inf behind them
  const float p = expf(mine - top);
  float sum = p;
  if (!a.renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += expf(val[j] - top);
  }
  sum = row_sum(sum);
  if (ok) {
    s.chosen[t * kMaxTopK + l16] = static_cast<u16>(my_expert);
    s.chosen_weight[t * kMaxTopK + l16] = p / sum;
    if (my_expert != 0xffff)
      atomicOr(t < 32 ? &s.lo[my_expert] : &s.hi[my_expert], 1u << (t & 31));
    if (bad && l16 == 0) atomicOr(t < 32 ? &r.nan_lo : &r.nan_hi, 1u << (t & 31));
  }
}

// Routes all tokens; ends with a barrier.
__device__ inline void route(const MoeArgs &a, Routing &r, RoutingScratch &s) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int e = threadIdx.x; e < a.experts; e += kMoeThreads) s.lo[e] = s.hi[e] = 0;
  if (threadIdx.x == 0) r.nan_lo = r.nan_hi = 0;
  __syncthreads();
  for (int t0 = wave * 4; t0 < a.tokens; t0 += kMoeWaves * 4) {
    const int t = t0 + (lane >> 4);
    if (a.experts <= 64) choose<4>(a, t, r, s);
    else if (a.experts <= 128) choose<8>(a, t, r, s);
    else if (a.experts <= 256) choose<16>(a, t, r, s);
    else choose<32>(a, t, r, s);
  }
  __syncthreads();
  if (wave == 0) {
    int pairs = 0, reached = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
      const int e = e0 + lane;
      const unsigned lo = e < a.experts ? s.lo[e] : 0, hi = e < a.experts ? s.hi[e] : 0;
      const int c = __popc(lo) + __popc(hi);
      const int upto = wave_running_sum(c);
      const unsigned long long who = __ballot(c > 0);
      const unsigned base = static_cast<unsigned>(pairs + upto - c);
      if (e < a.experts) s.base[e] = static_cast<u16>(base);
      if (c > 0)
        r.reached[reached + __popcll(who & ((1ull << lane) - 1))] =
            Reached{static_cast<unsigned>(e) | (base << 16), lo, hi};
      pairs += __builtin_amdgcn_readlane(upto, 63);
      reached += __popcll(who);
    }
    if (lane == 0) r.num_reached = reached;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * kMaxTopK; i += kMoeThreads) {
    const int e = s.chosen[i];
    if (e != 0xffff) {
      const int t = i / kMaxTopK;
      const unsigned long long m = s.lo[e] | (static_cast<unsigned long long>(s.hi[e]) << 32);
      const int p = s.base[e] + __popcll(m & ((1ull << t) - 1));
      r.token[p] = static_cast<unsigned char>(t);
      r.weight[p] = s.chosen_weight[i];
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

// 8 codes under a scale as bfloat16.
__device__ inline bf16x8 weights8(unsigned codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Sums acc over the workgroup's waves through LDS (red: WAVES * TILES * 64), in
// wave order: afterwards wave w < used holds tile w's sums, the lanes as acc.
template <int TILES, int WAVES>
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
    for (int w = 1; w < WAVES; ++w) s += red[(w * TILES + wave) * 64 + lane];
  }
  return s;
}

// 32 values of x of a lane's token as they are loaded, and their parts.
template <int TYPE>
struct RawX {
  uintx4 v[TYPE == kF32 ? 8 : 4];
  __device__ inline void parts(int j, bf16x8 (&out)[Parts<TYPE>::x]) const {
    if constexpr (TYPE == kBf16) {
      out[0] = __builtin_bit_cast(bf16x8, v[j]);
    } else {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (TYPE == kF32) {
          const unsigned w = v[2 * j + i / 4][i % 4];   // (the cast of a vector's element itself takes the first)
          f[i] = __builtin_bit_cast(float, w);
        } else
          f[i] = Elem<TYPE>::get(static_cast<u16>(v[j][i / 2] >> (16 * (i % 2))));
      }
      split8<Parts<TYPE>::x>(f, out);
    }
  }
  // From p, `left` values in range, the rest zeros.
  template <bool VEC>
  __device__ inline void load(const typename Elem<TYPE>::store *p, int left) {
    constexpr int kEach = TYPE == kF32 ? 4 : 8, kRegs = TYPE == kF32 ? 8 : 4;
    if (VEC && left >= 32) {
#pragma unroll
      for (int r = 0; r < kRegs; ++r) v[r] = reinterpret_cast<const uintx4 *>(p)[r];
    } else {
#pragma unroll
      for (int r = 0; r < kRegs; ++r) {
        uintx4 w = {};
#pragma unroll
        for (int i = 0; i < kEach; ++i)
          if (r * kEach + i < left) {
            if constexpr (TYPE == kF32)
              w[i] = __builtin_bit_cast(unsigned, p[r * kEach + i]);
            else
              w[i / 2] |= static_cast<unsigned>(p[r * kEach + i]) << (16 * (i % 2));
          }
        v[r] = w;
      }
    }
  }
};

// G x, U x and a for the reached experts. An item is 16 of an expert's gate rows
// and the same up rows; the 8 waves share its K, two chunks of 128 a wave at a
// time, and the next two's weights (of the next item where this one ends) are
// on their way meanwhile.
template <int TYPE, bool VEC>
__global__ __launch_bounds__(kMoeThreads, Parts<TYPE>::x == 1 ? 4 : 2) void moe_up_kernel(MoeArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int PX = Parts<TYPE>::x, PH = Parts<TYPE>::h;
  constexpr int kAt = 2;   // chunks of a wave at a time
  __shared__ Routing r;
  // partial sums of the waves, of two items in turn; scratch of the routing first
  constexpr int kRed = kMoeWaves * 2 * kUpTiles * 64;
  __shared__ __attribute__((aligned(16))) f32x4 red[2 * kRed];
  static_assert(sizeof(RoutingScratch) <= sizeof(red), "scratch fits");
  route(a, r, *reinterpret_cast<RoutingScratch *>(red));
  int half = 0;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int num_reached = __builtin_amdgcn_readfirstlane(r.num_reached);
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.reached[0] = Reached{static_cast<unsigned>(num_reached), r.nan_lo, r.nan_hi};
    for (int n = threadIdx.x; n < num_reached; n += kMoeThreads) a.reached[1 + n] = r.reached[n];
  }
  const int i16 = lane & 15, g = lane >> 4;
  const int HP = (a.hidden + kAlign - 1) / kAlign * kAlign;
  const int IP = (a.inter + kAlign - 1) / kAlign * kAlign;
  const int tiles = IP / 16, chunks = HP / 128;
  const long long plane = static_cast<long long>(a.tokens) * a.top_k * IP;
  const store *x = static_cast<const store *>(a.x);
  const int items = num_reached * tiles;

  struct Weights {
    uintx4 gate[kAt], up[kAt];
    unsigned gate_scale[kAt], up_scale[kAt];
  };
  auto load_weights = [&](Weights &w, int item, int c) {
    if (item >= items) return;
    const int ai = item / tiles;
    const int e = r.reached[ai].expert_base & 0xffff;
    const int row = min((item - ai * tiles) * 16 + i16, a.inter - 1);
    const long long gate = static_cast<long long>(__builtin_amdgcn_readfirstlane(e)) * 2 * a.inter + row;
    const long long up = gate + a.inter;
    const unsigned char *gc = a.w1c + gate * (HP / 2) + g * 16, *gs = a.w1s + gate * (HP / 32) + g;
    const unsigned char *uc = a.w1c + up * (HP / 2) + g * 16, *us = a.w1s + up * (HP / 32) + g;
#pragma unroll
    for (int b = 0; b < kAt; ++b) {
      const int cb = c + b * kMoeWaves;
      if (cb < chunks) {
        w.gate[b] = *reinterpret_cast<const uintx4 *>(gc + cb * 64);
        w.up[b] = *reinterpret_cast<const uintx4 *>(uc + cb * 64);
        w.gate_scale[b] = gs[cb * 4];
        w.up_scale[b] = us[cb * 4];
      }
    }
  };

  Weights cur, next;
  load_weights(cur, blockIdx.x, wave);
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int ai = item / tiles;
    const int row0 = (item - ai * tiles) * 16;
    const Reached now = r.reached[ai];
    const int base = __builtin_amdgcn_readfirstlane(now.expert_base >> 16);
    const int count = __builtin_amdgcn_readfirstlane(__popc(now.lo) + __popc(now.hi));
    for (int first = 0; first < count; first += 16 * kUpTiles) {   // tokens of the expert
      const int used = min(kUpTiles, (count - first + 15) / 16);
      const bool last = first + 16 * kUpTiles >= count;
      f32x4 acc[2 * kUpTiles] = {};   // gate and up of each tile of 16 tokens
      for (int c = wave; c < chunks || c == wave; c += kAt * kMoeWaves) {
        const bool more = c + kAt * kMoeWaves < chunks;
        load_weights(next, more || !last ? item : item + gridDim.x, more ? c + kAt * kMoeWaves : wave);
#pragma unroll
        for (int t = 0; t < kUpTiles; ++t) {
          if (t < used) {
            const int n = first + t * 16 + i16;
            const store *px = x + static_cast<long long>(n < count ? r.token[base + n] : 0) * a.ldx + g * 32;
#pragma unroll
            for (int b = 0; b < kAt; ++b) {
              const int k = (c + b * kMoeWaves) * 128;
              if (k < HP) {
                RawX<TYPE> raw = {};
                if (n < count) {
                  if (VEC && k + 128 <= a.hidden)
                    raw.template load<true>(px + k, 32);
                  else
                    raw.template load<false>(px + k, a.hidden - k - g * 32);
                }
                const float fg = scale_value(cur.gate_scale[b]), fu = scale_value(cur.up_scale[b]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  bf16x8 xv[PX];
                  raw.parts(j, xv);
                  const bf16x8 vg = weights8(cur.gate[b][j], fg), vu = weights8(cur.up[b][j], fu);
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
        cur = next;
      }
      // One barrier an item: the next one's sums go to the other half, and nobody
      // writes this half again before having passed the next barrier.
      f32x4 *mine = red + half * kRed;
      half ^= 1;
#pragma unroll
      for (int t = 0; t < 2 * kUpTiles; ++t)
        if (t < 2 * used) mine[(wave * 2 * kUpTiles + t) * 64 + lane] = acc[t];
      __syncthreads();
      if (wave < used) {
        f32x4 gv = mine[(2 * wave) * 64 + lane], uv = mine[(2 * wave + 1) * 64 + lane];
#pragma unroll
        for (int w = 1; w < kMoeWaves; ++w) {
          gv += mine[(w * 2 * kUpTiles + 2 * wave) * 64 + lane];
          uv += mine[(w * 2 * kUpTiles + 2 * wave + 1) * 64 + lane];
        }
        const int n = first + wave * 16 + i16;
        if (n < count) {
          const int p = base + n;
          const float w = r.weight[p];
          const int row = row0 + 4 * g;
          u16 parts[PH][4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            // past the last row of an expert: the zeros that pad `inter`
            float rest = row + v < a.inter ? gv[v] / (1.0f + expf(-gv[v])) * uv[v] * w : 0.0f;
#pragma unroll
            for (int q = 0; q < PH; ++q) {
              const unsigned b = __builtin_bit_cast(unsigned, rest);
              parts[q][v] = q + 1 < PH || PH == 3 ? static_cast<u16>(b >> 16) : Elem<kBf16>::put(rest);
              rest = __builtin_isinf(rest) ? 0.0f : rest - Elem<kBf16>::get(parts[q][v]);
            }
          }
#pragma unroll
          for (int q = 0; q < PH; ++q)
            *reinterpret_cast<uintx2 *>(a.h + q * plane + static_cast<long long>(p) * IP + row) =
                uintx2{parts[q][0] | (static_cast<unsigned>(parts[q][1]) << 16),
                       parts[q][2] | (static_cast<unsigned>(parts[q][3]) << 16)};
        }
      }
    }
  }
}

// Y: a workgroup takes 16 rows of every reached expert's D, its waves the
// (expert, chunk of 128) steps in turn, two a wave at a time, the next two's
// weights on their way.
template <int TYPE>
__global__ __launch_bounds__(kDownThreads, 4) void moe_down_kernel(MoeArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int PH = Parts<TYPE>::h;
  constexpr int kAt = 2;
  __shared__ Reached reached[kMaxExperts + 1];
  __shared__ __attribute__((aligned(16))) f32x4 red[kDownWaves * kTokenTiles * 64];
  const int most = min(a.experts, a.tokens * a.top_k) + 1;
  for (int n = threadIdx.x; n < most; n += kDownThreads) reached[n] = a.reached[n];
  __syncthreads();
  const int num_reached = __builtin_amdgcn_readfirstlane(reached[0].expert_base);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int IP = (a.inter + kAlign - 1) / kAlign * kAlign;
  const int chunks = IP / 128;
  const long long plane = static_cast<long long>(a.tokens) * a.top_k * IP;
  const int row0 = blockIdx.x * 16;
  const int row = min(row0 + i16, a.hidden - 1);
  const int token_tiles = (a.tokens + 15) / 16;

  // A step: reached expert `at` (num_reached: none left) and chunk c.
  struct Step {
    int at, c;
  };
  auto advance = [&](Step s) {
    s.c += kDownWaves;
    while (s.c >= chunks && s.at < num_reached) {
      s.c -= chunks;
      ++s.at;
    }
    return s;
  };
  struct Weights {
    uintx4 w[kAt];
    unsigned scale[kAt];
  };
  auto load_weights = [&](Weights &w, const Step (&s)[kAt]) {
#pragma unroll
    for (int b = 0; b < kAt; ++b) {
      if (s[b].at < num_reached) {
        const int e = __builtin_amdgcn_readfirstlane(reached[1 + s[b].at].expert_base & 0xffff);
        const long long wr = static_cast<long long>(e) * a.hidden + row;
        w.w[b] = *reinterpret_cast<const uintx4 *>(a.w2c + wr * (IP / 2) + s[b].c * 64 + g * 16);
        w.scale[b] = a.w2s[wr * (IP / 32) + s[b].c * 4 + g];
      }
    }
  };
  f32x4 acc[kTokenTiles] = {};
  Step step[kAt];
  step[0] = advance(Step{0, wave - kDownWaves});
#pragma unroll
  for (int b = 1; b < kAt; ++b) step[b] = advance(step[b - 1]);
  Weights cur, next;
  load_weights(cur, step);
  while (step[0].at < num_reached) {
    Step then[kAt];
    then[0] = advance(step[kAt - 1]);
#pragma unroll
    for (int b = 1; b < kAt; ++b) then[b] = advance(then[b - 1]);
    load_weights(next, then);
#pragma unroll
    for (int b = 0; b < kAt; ++b) {
      if (step[b].at >= num_reached) continue;
      const Reached now = reached[1 + step[b].at];
      const unsigned long long m =
          static_cast<unsigned>(__builtin_amdgcn_readfirstlane(now.lo)) |
          (static_cast<unsigned long long>(static_cast<unsigned>(__builtin_amdgcn_readfirstlane(now.hi))) << 32);
      const float f = scale_value(cur.scale[b]);
#pragma unroll
      for (int t = 0; t < kTokenTiles; ++t) {
        if (t < token_tiles && ((m >> (16 * t)) & 0xffffull)) {
          const int n = t * 16 + i16;
          const bool has = (m >> n) & 1;
          bf16x8 hv[PH][4] = {};
          if (has) {
            const int p = (now.expert_base >> 16) + __popcll(m & ((1ull << n) - 1));
            const u16 *h = a.h + static_cast<long long>(p) * IP + step[b].c * 128 + g * 32;
#pragma unroll
            for (int q = 0; q < PH; ++q)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                hv[q][j] = *reinterpret_cast<const bf16x8 *>(h + q * plane + j * 8);
          }
          f32x4 sum = acc[t];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8 v = weights8(cur.w[b][j], f);
#pragma unroll
            for (int q = 0; q < PH; ++q)
              sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, hv[q][j], sum, 0, 0, 0);
          }
          // A token that did not choose this expert keeps its sum, also where the
          // expert's weights hold a NaN (0 * NaN is not 0).
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[t][v] = has ? sum[v] : acc[t][v];
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kAt; ++b) step[b] = then[b];
    cur = next;
  }
  const f32x4 sum = reduce_waves<kTokenTiles, kDownWaves>(acc, token_tiles, red);
  const int t = wave * 16 + i16;
  if (wave < token_tiles && t < a.tokens) {
    const bool nan = ((t < 32 ? reached[0].lo : reached[0].hi) >> (t & 31)) & 1;
    store *y = static_cast<store *>(a.y) + static_cast<long long>(t) * a.ldy + row0 + 4 * g;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (row0 + 4 * g + v < a.hidden)
        y[v] = Elem<TYPE>::put(nan ? __builtin_nanf("") : sum[v]);
  }
}

}  // namespace mx
}  // namespace gemm
