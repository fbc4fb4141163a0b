// A mixture-of-experts layer for a few tokens on microscaled weights, in two
// kernels (the operation is described in gemm.h at gemm_mx_moe):
//   up:    route, then for each reached expert G x and U x, a = w silu(Gx) Ux
//          into the workspace;
//   down:  Y = sum over the reached experts of D a.
// Every workgroup of the first kernel works the routing out for itself from the
// logits (a few microseconds at most, and no third launch or hand-over between
// workgroups); one of them leaves the list of the reached experts and their tokens for the
// second.
//
// Both products stream their weights from memory once, straight into
// registers: 16 weight rows are the rows of v_mfma_f32_16x16x32_bf16, 16 tokens
// its columns. A lane loads the 16 bytes of one row's block of 32 codes and
// that block's scale, and turns 8 codes at a time into bfloat16 (exact: e2m1
// has 2 bits of mantissa) for one instruction; which k an instruction's lane
// group carries is free as long as both operands agree, so lane group g takes
// block g of a row's 128 values.
// Activations keep their precision by being split into bfloat16 parts
// whose sum is exact: a bfloat16 is one part, a half two, a float three, and so the
// hidden activations, which are FP32 whatever the type of X and Y. The
// matrix instructions are far from the bound (the weights' bytes), so the
// parts cost little that shows.
#pragma once

#include "gemm_kernels.hpp"
#include "mx_kernels.hpp"

namespace gemm {
namespace mx {

constexpr int kMoeWaves = 16;   // of the first kernel: one workgroup a CU
constexpr int kMoeThreads = 64 * kMoeWaves;
constexpr int kMaxTokens = 64, kMaxExperts = 512, kMaxTopK = 16;   // GEMM_MX_MOE_MAX_*
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
// An expert's tokens are taken in groups of GROUP = 4 or 8.
constexpr int kMaxGroups = kMaxExperts + kMaxPairs / 4;

template <int TYPE>
struct Parts {
  static constexpr int x = TYPE == kF32 ? 3 : TYPE == kF16 ? 2 : 1;   // of the inputs
  static constexpr int h = 3;                                         // of the hidden activations
  // 16-bit words of a hidden activation in the workspace: its three parts, or the
  // float, which the second kernel then splits.
  static constexpr int h_words = TYPE == kF32 ? 3 : 2;
};
// Waves of the second kernel, by the registers that the activations in flight take.
template <int TYPE>
constexpr int kDownWaves = TYPE == kF32 ? 8 : 16;

// Up to GROUP tokens of one expert: the expert, how many tokens, their first
// pair and the tokens (a byte each, the first one again where there are fewer).
// Pairs (token, expert) are numbered by expert, then token; pair numbers index the
// rows of the hidden activations. Entry 0 of the workspace's list holds how many
// follow and the tokens whose logits hold a NaN or +inf, one bit each.
struct Group {
  unsigned packed;   // expert | count << 9 | first pair << 13
  unsigned lo, hi;
  __device__ inline int expert() const { return packed & 511; }
  __device__ inline int count() const { return (packed >> 9) & 15; }
  __device__ inline int base() const { return packed >> 13; }
};
static_assert(kMaxExperts <= 512, "Group's fields");
__device__ inline Group uniform(const Group &g) {
  return Group{static_cast<unsigned>(__builtin_amdgcn_readfirstlane(g.packed)),
               static_cast<unsigned>(__builtin_amdgcn_readfirstlane(g.lo)),
               static_cast<unsigned>(__builtin_amdgcn_readfirstlane(g.hi))};
}

struct MoeArgs {
  int tokens, hidden, inter, experts, top_k, renormalize;
  const float *logits;
  int ld_logits;
  const void *x;
  int ldx;
  const unsigned char *w1c, *w1s, *w2c, *w2s;
  void *y;
  int ldy;
  u16 *h;       // workspace: (tokens * top_k) x IP hidden activations, 3 planes of their
                // bfloat16 parts (FP32 inputs) or floats,
  Group *groups;   // and what the second kernel needs of the routing
};

// What a workgroup knows after routing.
struct Routing {
  Group groups[kMaxGroups];         // of the reached experts, ascending
  float weight[kMaxPairs];          // the pair's weight
  unsigned nan_lo, nan_hi;          // tokens whose logits hold a NaN or +inf
  int num_groups;
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
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = j * 16 + l16;
    val[j] = ok && e < a.experts ? l[e] + 0.0f : -__builtin_inff();   // -0 equals +0
  }
  unsigned best = 0, largest = 0;   // largest: of the magnitudes, -inf left out
  int at = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const unsigned b = __builtin_bit_cast(unsigned, val[j]);
    largest = max(largest, b == 0xff800000u ? 0u : magnitude_bits(val[j]));
    key[j] = b == 0xff800000u ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
    if (key[j] > best) {
      best = key[j];
      at = j;
    }
  }
  const bool bad = row_max(largest) >= 0x7f800000u;   // a NaN or +inf
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
template <int GROUP>
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
    int pairs = 0, groups = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
      const int e = e0 + lane;
      unsigned long long m =
          e < a.experts ? s.lo[e] | (static_cast<unsigned long long>(s.hi[e]) << 32) : 0;
      const int c = __popcll(m);
      const int pairs_to = wave_running_sum(c);
      const int groups_to = wave_running_sum((c + GROUP - 1) / GROUP);
      int base = pairs + pairs_to - c, at = groups + groups_to - (c + GROUP - 1) / GROUP;
      if (e < a.experts) s.base[e] = static_cast<u16>(base);
      while (m) {
        unsigned tokens[2] = {};
        const int first = __builtin_ctzll(m);
        int n = 0;
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
          tokens[i / 4] |= static_cast<unsigned>(m ? __builtin_ctzll(m) : first) << (8 * (i % 4));
          n += m != 0;
          m &= m - 1;
        }
        r.groups[at++] = Group{static_cast<unsigned>(e | (n << 9) | (base << 13)), tokens[0], tokens[1]};
        base += n;
      }
      pairs += __builtin_amdgcn_readlane(pairs_to, 63);
      groups += __builtin_amdgcn_readlane(groups_to, 63);
    }
    if (lane == 0) r.num_groups = groups;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * kMaxTopK; i += kMoeThreads) {
    const int e = s.chosen[i];
    if (e != 0xffff) {
      const int t = i / kMaxTopK;
      const unsigned long long m = s.lo[e] | (static_cast<unsigned long long>(s.hi[e]) << 32);
      const int p = s.base[e] + __popcll(m & ((1ull << t) - 1));
      r.weight[p] = s.chosen_weight[i];
    }
  }
  __syncthreads();
}

// 8 floats into PARTS bfloat16 vectors whose sum is exact for PARTS = 3 (and for
// fewer bits accordingly): each part is what is left, cut off after its 8 bits.
// (Below 2^-110 the last part falls under bfloat16's smallest number: the sum is then
// cut off to a multiple of 2^-133.) Past an infinity nothing is left, or without INF,
// which saves two instructions a value and part, a NaN.
template <int PARTS, bool INF = true>
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
      w[i] = __builtin_amdgcn_perm(b, a, 0x07060302);   // the high halves
    }
    out[p] = __builtin_bit_cast(bf16x8, w);
    if (p + 1 < PARTS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float part =
            __builtin_bit_cast(float, __builtin_bit_cast(unsigned, rest[i]) & 0xffff0000u);
        rest[i] = INF && __builtin_isinf(rest[i]) ? 0.0f : rest[i] - part;
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

// Activations on their way from memory to a matrix instruction. 128 values of up
// to GROUP tokens are loaded with all lanes busy, lane (s, c) = (lane / 16,
// lane % 16) taking values 8c .. 8c + 7 of token s (and of token 4 + s), and pass
// through LDS, [part][token][16 pieces of 16 bytes], token t's piece c at c ^ t
// so that the lanes that read one piece of several tokens meet no bank twice.
// Lane (g, n) of an instruction reads pieces 4g .. 4g + 3 of one token.
template <int GROUP>
__device__ inline void stage_write(unsigned char *stage, int part, int token, int piece, bf16x8 v) {
  *reinterpret_cast<bf16x8 *>(stage + (part * GROUP + token) * 256 + ((piece ^ token) & 15) * 16) = v;
}
template <int GROUP>
__device__ inline bf16x8 stage_read(const unsigned char *stage, int part, int token, int piece) {
  return *reinterpret_cast<const bf16x8 *>(stage + (part * GROUP + token) * 256 +
                                           ((piece ^ token) & 15) * 16);
}
// Loads through a buffer resource: a uniform base and the bytes behind it (dwords
// past them read as zero), a lane's offset and a uniform one.
__device__ inline __amdgpu_buffer_rsrc_t buffer(const unsigned char *base, long long bytes) {
  const long long most = 0x7fffffff;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<unsigned char *>(base), 0,
                                           static_cast<int>(bytes < most ? bytes : most), 0x00020000);
}
__device__ inline uintx4 load16(__amdgpu_buffer_rsrc_t r, unsigned lane_off, int off) {
  return __builtin_bit_cast(uintx4, __builtin_amdgcn_raw_buffer_load_b128(r, lane_off, off, 0));
}
__device__ inline uintx2 load8(__amdgpu_buffer_rsrc_t r, unsigned lane_off, int off) {
  return __builtin_bit_cast(uintx2, __builtin_amdgcn_raw_buffer_load_b64(r, lane_off, off, 0));
}

// Waits for a load's registers here, on every path: where a branch that uses
// them is not taken the compiler would otherwise have to wait for all loads
// before it gives the registers to something else.
template <class V>
__device__ inline void arrived(const V &v) {
  asm volatile("" : : "v"(v));
}

// step(cur, next) `n` times, the two sets of registers in turn. No exit in the middle
// of the loop: loads still on their way there would be waited for at its top.
template <class F, class S>
__device__ inline void in_turn(int n, F &even, F &odd, S &&step) {
  for (; n > 1; n -= 2) {
    step(even, odd);
    step(odd, even);
  }
  if (n) step(even, odd);
}

// 8 values of x, `left` of them in range (the rest zeros), as bfloat16 parts.
template <int TYPE>
__device__ inline void load_parts(const typename Elem<TYPE>::store *p, int left,
                                  bf16x8 (&out)[Parts<TYPE>::x]) {
  if (TYPE == kBf16 && left >= 8) {
    const uintx4 v = *reinterpret_cast<const uintx4_any *>(p);
    out[0] = __builtin_bit_cast(bf16x8, v);
  } else {
    float v[8];
    load8<TYPE>(p, left, v);
    split8<Parts<TYPE>::x>(v, out);
  }
}

// The scale of chunk b (0 or 1) of two chunks' 4 scale bytes each, for lane group g.
__device__ inline float pair_scale(const uintx2 &s, int b, int g) {
  const unsigned w = b ? s[1] : s[0];
  return scale_value((w >> (8 * g)) & 255);
}

// G x, U x and a for the reached experts. An item is 16 of an expert's gate rows
// and the same up rows for one group of its tokens; a workgroup takes a run of
// items, mostly of one group, whose activations it keeps in LDS (RESIDENT; where
// all of `hidden` does not fit they are loaded again for every item). The 16
// waves share an item's K, a wave taking two neighbouring chunks of 128 at a
// time (a whole 128-byte line of a row's codes); the next two's weights (of the
// next item where this one ends) are on their way meanwhile, in the other of
// two sets of registers.
// Bound by the weights' bytes: 32 tokens on 8 of 128 experts of 4096 x 1024 (0.49 GB
// of G and U) take 118 to 125 us, 10 of them routing, so 4.2 to 4.5 TB/s. With activations
// loaded anew for each item the vector memory pipe was the bound (155 us, as long
// with the arithmetic left out).
constexpr int kUpLds = 160 * 1024;
template <int GROUP>
constexpr int kUpRed = 2 * kMoeWaves * 2 * 4 * GROUP * 16;   // partial sums, of two items in turn
// what is left for the activations
template <int GROUP>
constexpr int kUpStage = (kUpLds - kUpRed<GROUP> - static_cast<int>(sizeof(Routing))) / 1024 * 1024;

template <int TYPE, int GROUP, bool RESIDENT>
__global__ __launch_bounds__(kMoeThreads, 4) void moe_up_kernel(MoeArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int PX = Parts<TYPE>::x;
  constexpr int kAt = 2;   // chunks of a wave at a time
  constexpr int kChunkStage = PX * GROUP * 256;
  __shared__ Routing r;
  __shared__ __attribute__((aligned(16))) unsigned char red[kUpRed<GROUP>];
  // activations; scratch of the routing first
  __shared__ __attribute__((aligned(16))) unsigned char stages[RESIDENT ? kUpStage<GROUP> : kMoeWaves * kAt * kChunkStage];
  static_assert(sizeof(RoutingScratch) <= sizeof(stages), "scratch fits");
  route<GROUP>(a, r, *reinterpret_cast<RoutingScratch *>(stages));
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int num_groups = __builtin_amdgcn_readfirstlane(r.num_groups);
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) a.groups[0] = Group{static_cast<unsigned>(num_groups), r.nan_lo, r.nan_hi};
    for (int n = threadIdx.x; n < num_groups; n += kMoeThreads) a.groups[1 + n] = r.groups[n];
  }
  const int i16 = lane & 15, g = lane >> 4;
  const int HP = (a.hidden + kAlign - 1) / kAlign * kAlign;
  const int IP = (a.inter + kAlign - 1) / kAlign * kAlign;
  const int tiles = IP / 16, chunks = HP / 128;
  const int batches = (chunks + kAt * kMoeWaves - 1) / (kAt * kMoeWaves);
  const long long plane = static_cast<long long>(a.tokens) * a.top_k * IP;
  const int items = num_groups * tiles;
  const int wgs = __builtin_amdgcn_readfirstlane(gridDim.x);
  // Neighbouring runs on the workgroups of one XCD: where an expert has several
  // groups, its weights are then read at much the same time through one L2 cache.
  const int wg = xcd_order(blockIdx.x, wgs);
  int item = static_cast<int>(static_cast<long long>(items) * wg / wgs);
  const int end = static_cast<int>(static_cast<long long>(items) * (wg + 1) / wgs);
  if (item >= end) return;

  // An item: its group and tile, the tile's rows that exist (`first`: of the last tile
  // that has some, where row0 lies in the padding of `inter`) and where the gate
  // rows' codes and scales begin. Items follow each other, so the next one's are
  // a step away but for a change of group.
  const int code_row = HP / 2, scale_row = HP / 32;
  const unsigned char *scales_end = a.w1s + 2LL * a.experts * a.inter * scale_row;
  const long long up_codes = static_cast<long long>(a.inter) * code_row;
  const long long up_scales = static_cast<long long>(a.inter) * scale_row;
  struct Item {
    int gi, row0, first;
    Group group;
    const unsigned char *codes, *scales;
  };
  auto item_of = [&](int gi, int row0) __attribute__((always_inline)) {
    Item t;
    t.gi = gi;
    t.row0 = row0;
    t.first = min(row0, a.inter - 1) / 16 * 16;
    t.group = uniform(r.groups[gi]);
    const long long row = static_cast<long long>(t.group.expert()) * 2 * a.inter + t.first;
    t.codes = a.w1c + row * code_row;
    t.scales = a.w1s + row * scale_row;
    return t;
  };
  auto after = [&](const Item &s) __attribute__((always_inline)) {
    Item t = s;
    t.row0 += 16;
    if (t.row0 == IP) return item_of(s.gi + 1, 0);
    if (t.row0 < a.inter) {
      t.first = t.row0;
      t.codes += 16 * code_row;
      t.scales += 16 * scale_row;
    }
    return t;
  };
  struct Fetched {
    uintx4 gate[kAt], up[kAt];
    uintx2 gate_scale, up_scale;
  };
  auto fetch = [&](Fetched &f, const Item &t, int batch, bool wanted) __attribute__((always_inline)) {
    const int c = (batch * kMoeWaves + wave) * kAt;
    // rows past the expert's last: the last one again (their results are not kept)
    const int i = wanted ? min(i16, a.inter - 1 - t.first) : 0;
    const __amdgpu_buffer_rsrc_t gc = buffer(t.codes, 0x7fffffff), uc = buffer(t.codes + up_codes, 0x7fffffff);
    // (a pair of chunks' scales may reach past the operand's last)
    const __amdgpu_buffer_rsrc_t gs = buffer(t.scales, scales_end - t.scales);
    const __amdgpu_buffer_rsrc_t us = buffer(t.scales + up_scales, scales_end - t.scales - up_scales);
    const unsigned code_off = static_cast<unsigned>(i * code_row + (wanted ? g * 16 : 0));
    const unsigned scale_off = static_cast<unsigned>(i * scale_row);
#pragma unroll
    for (int b = 0; b < kAt; ++b) {
      const int cb = min(c + b, chunks - 1);   // past the end: the last chunk again, not used
      f.gate[b] = load16(gc, code_off, cb * 64);
      f.up[b] = load16(uc, code_off, cb * 64);
    }
    const int cs = min(c, chunks - 1);
    f.gate_scale = load8(gs, scale_off, cs * 4);
    f.up_scale = load8(us, scale_off, cs * 4);
  };
  // The wave's chunks of batch of the group's activations into LDS.
  auto stage_of = [&](int batch, int b) {
    return stages + (RESIDENT ? (batch * kMoeWaves + wave) * kAt + b : wave * kAt + b) * kChunkStage;
  };
  auto stage_x = [&](unsigned lo, unsigned hi, int batch) __attribute__((always_inline)) {
    const store *x = static_cast<const store *>(a.x) + i16 * 8;
    const store *x0 = x + static_cast<long long>((lo >> (8 * g)) & 255) * a.ldx;
    const store *x1 = x + static_cast<long long>((hi >> (8 * g)) & 255) * a.ldx;
    const int c = (batch * kMoeWaves + wave) * kAt;
    wave_order();
#pragma unroll
    for (int b = 0; b < kAt; ++b) {
      if (c + b < chunks) {
        const int left = a.hidden - (c + b) * 128 - i16 * 8;
        unsigned char *stage = stage_of(batch, b);
        bf16x8 parts[PX];
        load_parts<TYPE>(x0 + (c + b) * 128, left, parts);
#pragma unroll
        for (int p = 0; p < PX; ++p) stage_write<GROUP>(stage, p, g, i16, parts[p]);
        if constexpr (GROUP > 4) {
          load_parts<TYPE>(x1 + (c + b) * 128, left, parts);
#pragma unroll
          for (int p = 0; p < PX; ++p) stage_write<GROUP>(stage, p, 4 + g, i16, parts[p]);
        }
      }
    }
    wave_order();
  };

  int batch = 0, turn = 0;
  bool fresh = true;   // the group's activations are not in LDS yet
  Item now = item_of(item / tiles, item % tiles * 16);
  f32x4 acc_gate = {}, acc_up = {};
  // One batch of an item from one set of registers, the next one's loads into the
  // other.
  auto step = [&](Fetched &cur, Fetched &next) __attribute__((always_inline)) {
    const bool last = batch + 1 == batches;
    const bool more = !last || item + 1 < end;
    Item then = now;
    if (last && more) then = after(now);
    // Also after the last one (then all lanes load the same bytes): a branch
    // around the loads would make the compiler wait for them at its end.
    fetch(next, then, last ? 0 : batch + 1, more);
    __builtin_amdgcn_sched_barrier(0);
    if (fresh || !RESIDENT) stage_x(now.group.lo, now.group.hi, batch);
    const int c = (batch * kMoeWaves + wave) * kAt;
    arrived(cur.gate_scale);
    arrived(cur.up_scale);
#pragma unroll
    for (int b = 0; b < kAt; ++b) {
      arrived(cur.gate[b]);
      arrived(cur.up[b]);
      if (c + b < chunks) {
        const unsigned char *stage = stage_of(batch, b);
        const float fg = pair_scale(cur.gate_scale, b, g), fu = pair_scale(cur.up_scale, b, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 vg = weights8(cur.gate[b][j], fg), vu = weights8(cur.up[b][j], fu);
#pragma unroll
          for (int p = 0; p < PX; ++p) {
            const bf16x8 xv = stage_read<GROUP>(stage, p, i16 & (GROUP - 1), 4 * g + j);
            acc_gate = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vg, xv, acc_gate, 0, 0, 0);
            acc_up = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vu, xv, acc_up, 0, 0, 0);
          }
        }
      }
    }
    if (!last) {
      ++batch;
      return;
    }
    // One barrier an item: the next one's sums go to the other half, and nobody
    // writes this half again before having passed the next barrier. Of the 16
    // columns the group's are kept: [wave][gate, up][g][column].
    f32x4 *sums = reinterpret_cast<f32x4 *>(red) + (turn & 1) * (kMoeWaves * 2 * 4 * GROUP);
    const int at = g * GROUP + i16;
    if (i16 < GROUP) {
      sums[wave * (8 * GROUP) + at] = acc_gate;
      sums[wave * (8 * GROUP) + 4 * GROUP + at] = acc_up;
    }
    __syncthreads();
    // One wave finishes the item, a lane for each output. The others wait for it at the
    // next barrier: with four outputs a lane the layer above took 131 us, and with
    // four outputs for each wave, which all of them then wait for, 128.
    if (wave == (turn & (kMoeWaves - 1))) {
      const float *s = reinterpret_cast<const float *>(sums);
#pragma unroll
      for (int e = 0; e < GROUP / 4; ++e) {
        const int col = (lane + 64 * e) % GROUP, row = (lane + 64 * e) / GROUP;
        const int from = (row / 4 * GROUP + col) * 4 + row % 4;
        float gv[kMoeWaves], uv[kMoeWaves];
#pragma unroll
        for (int w = 0; w < kMoeWaves; ++w) {
          gv[w] = s[w * (32 * GROUP) + from];
          uv[w] = s[w * (32 * GROUP) + 16 * GROUP + from];
        }
#pragma unroll
        for (int w = 1; w < kMoeWaves; ++w) {
          gv[0] += gv[w];
          uv[0] += uv[w];
        }
        if (col < now.group.count()) {
          const int p = now.group.base() + col;
          // past the last row of an expert: the zeros that pad `inter`
          float rest = now.row0 + row < a.inter
                           ? gv[0] / (1.0f + expf(-gv[0])) * uv[0] * r.weight[p] : 0.0f;
          const long long at_h = static_cast<long long>(p) * IP + now.row0 + row;
          if constexpr (TYPE == kF32) {
#pragma unroll
            for (int q = 0; q < 3; ++q) {
              const u16 part = static_cast<u16>(__builtin_bit_cast(unsigned, rest) >> 16);
              a.h[q * plane + at_h] = part;
              rest = __builtin_isinf(rest) ? 0.0f : rest - Elem<kBf16>::get(part);
            }
          } else {
            reinterpret_cast<float *>(a.h)[at_h] = rest;
          }
        }
      }
    }
    acc_gate = f32x4{};
    acc_up = f32x4{};
    ++item;
    batch = 0;
    ++turn;
    fresh = then.group.packed != now.group.packed;
    now = then;
  };
  Fetched even, odd;
  fetch(even, now, 0, true);
  in_turn((end - item) * batches, even, odd, step);
}

// Y: a workgroup takes 16 rows of every reached expert's D. Its waves take the
// steps (group of tokens, two neighbouring chunks of 128) in turn, the next
// step's weights and activations on their way. An instruction's columns are the three
// parts of four tokens' activations (columns 4 part + token; the last four repeat
// the third part): all parts at the price of one instruction and one read from
// LDS, where a column for each token would take three. A step's sums over the
// parts are added to the wave's own sums of those tokens, in LDS; at the end
// the waves' sums are added in order. Where the first part's sum is not finite it is the
// result: the other parts of an infinity are NaN.
// 32 tokens on 8 of 128 experts of 4096 x 1024 (0.25 GB of D) take 69 to 73 us, 3.4 to 3.6
// TB/s; the activations, as many bytes for a workgroup as its weights, cost the rest.
template <int TYPE, int GROUP>
__global__ __launch_bounds__(64 * kDownWaves<TYPE>, kDownWaves<TYPE> / 4) void moe_down_kernel(
    MoeArgs a) {
  typedef typename Elem<TYPE>::store store;
  constexpr int PH = Parts<TYPE>::h, W = kDownWaves<TYPE>, THREADS = 64 * W;
  constexpr int kLoads = Parts<TYPE>::h_words;   // of 16 bytes, for 8 hidden activations
  constexpr int kAt = 2, kHalves = GROUP / 4;   // chunks at a time; fours of tokens
  constexpr int kChunkStage = PH * 4 * 256;
  __shared__ Group groups[kMaxGroups + 1];
  __shared__ __attribute__((aligned(16))) unsigned char stages[W * kChunkStage];
  __shared__ __attribute__((aligned(16))) float sums[W * kMaxTokens * 16];   // [wave][token][row]
  const int most = min(a.experts, a.tokens * a.top_k) + a.tokens * a.top_k / GROUP + 1;
  for (int n = threadIdx.x; n < most; n += THREADS) groups[n] = a.groups[n];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  unsigned char *stage = stages + wave * kChunkStage;
  float *mine = sums + wave * (kMaxTokens * 16);
  for (int n = lane; n < a.tokens * 4; n += 64) reinterpret_cast<f32x4 *>(mine)[n] = f32x4{};
  __syncthreads();
  const int num_groups = __builtin_amdgcn_readfirstlane(groups[0].packed);
  const int IP = (a.inter + kAlign - 1) / kAlign * kAlign;
  const int chunks = IP / 128, batches = (chunks + kAt - 1) / kAt;
  const long long plane = static_cast<long long>(a.tokens) * a.top_k * IP;
  const int row0 = blockIdx.x * 16;
  const int row = min(i16, a.hidden - 1 - row0);
  const unsigned code_off = static_cast<unsigned>(row * (IP / 2) + g * 16);
  const unsigned scale_off = static_cast<unsigned>(row * (IP / 32));
  const long long expert_codes = static_cast<long long>(a.hidden) * (IP / 2);
  const long long expert_scales = static_cast<long long>(a.hidden) * (IP / 32);
  const unsigned char *codes0 = a.w2c + static_cast<long long>(row0) * (IP / 2);
  const unsigned char *scales0 = a.w2s + static_cast<long long>(row0) * (IP / 32);
  const unsigned char *scales_end = a.w2s + a.experts * expert_scales;

  struct Fetched {
    uintx4 w[kAt];
    uintx2 scale;
    uintx4 h[kAt][kLoads][kHalves];
  };
  auto fetch = [&](Fetched &f, const Group &now, int batch, bool wanted) __attribute__((always_inline)) {
    const unsigned char *scale_rows = scales0 + now.expert() * expert_scales;
    const __amdgpu_buffer_rsrc_t codes = buffer(codes0 + now.expert() * expert_codes, 0x7fffffff);
    // (a pair of chunks' scales may reach past the operand's last)
    const __amdgpu_buffer_rsrc_t scales = buffer(scale_rows, scales_end - scale_rows);
    // of a plane's parts, or of the floats
    constexpr int kBytes = TYPE == kF32 ? 2 : 4;
    const unsigned char *h = reinterpret_cast<const unsigned char *>(a.h) + static_cast<long long>(now.base()) * IP * kBytes;
    unsigned h_off[kHalves];   // (tokens past the group's last: the last one again)
#pragma unroll
    for (int s = 0; s < kHalves; ++s)
      h_off[s] = static_cast<unsigned>((min(4 * s + g, now.count() - 1) * IP + i16 * 8) * kBytes);
    f.scale = load8(scales, wanted ? scale_off : 0, min(batch * kAt, chunks - 1) * 4);
#pragma unroll
    for (int b = 0; b < kAt; ++b) {
      const int c = min(batch * kAt + b, chunks - 1);   // past the end: not used
      f.w[b] = load16(codes, wanted ? code_off : 0, c * 64);
#pragma unroll
      for (int q = 0; q < kLoads; ++q)
#pragma unroll
        for (int s = 0; s < kHalves; ++s)
          f.h[b][q][s] = load16(buffer(h + (TYPE == kF32 ? 2 * q * plane : 16 * q), 0x7fffffff), h_off[s],
                                c * 128 * kBytes);
    }
  };
  int at = 0, batch = wave;   // the step: group and batch
  auto wrap = [&](int &to, int &bt) {
    if (bt < batches) return;
    to += bt / batches;
    bt %= batches;
  };
  wrap(at, batch);
  Group now = uniform(groups[1 + min(at, kMaxGroups - 1)]);
  auto step = [&](Fetched &cur, Fetched &next) __attribute__((always_inline)) {
    int next_at = at, next_batch = batch + W;
    wrap(next_at, next_batch);
    const bool more = next_at < num_groups;
    const Group then = uniform(groups[1 + (more ? next_at : at)]);
    fetch(next, then, more ? next_batch : batch, more);
    __builtin_amdgcn_sched_barrier(0);
    f32x4 acc[kHalves] = {};
    arrived(cur.scale);
#pragma unroll
    for (int b = 0; b < kAt; ++b) {
      arrived(cur.w[b]);
#pragma unroll
      for (int q = 0; q < kLoads; ++q)
#pragma unroll
        for (int s = 0; s < kHalves; ++s) arrived(cur.h[b][q][s]);
      if (batch * kAt + b < chunks) {
        const float f = pair_scale(cur.scale, b, g);
        bf16x8 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = weights8(cur.w[b][j], f);
#pragma unroll
        for (int s = 0; s < kHalves; ++s) {
          bf16x8 parts[PH];
          if constexpr (TYPE == kF32) {
#pragma unroll
            for (int q = 0; q < PH; ++q) {
              const uintx4 h = cur.h[b][q][s];
              parts[q] = __builtin_bit_cast(bf16x8, h);
            }
          } else {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const unsigned h = cur.h[b][i / 4][s][i % 4];
              v[i] = __builtin_bit_cast(float, h);
            }
            split8<PH, false>(v, parts);   // (the sums below look after infinities)
          }
          // The third part's pieces lie 8 further on (c ^ t ^ 8): lanes 0 .. 3, 12 .. 15, 20 ..
          // 27, which LDS serves at one time, then meet no bank twice (with c ^ row a layer of
          // 32 tokens on 8 of 128 experts had 4.5e6 cycles of conflicts, so 0.55e6).
          wave_order();
#pragma unroll
          for (int q = 0; q < PH; ++q) stage_write<4>(stage, q, g, i16 ^ (q == 2 ? 8 : 0), parts[q]);
          wave_order();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                w[j], stage_read<4>(stage, min(i16 / 4, PH - 1), i16 & 3, (4 * g + j) ^ (i16 & 8)), acc[s], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int s = 0; s < kHalves; ++s) {
      f32x4 sum;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float first = acc[s][v], rest = from_lane<4>(first) + from_lane<8>(first);
        sum[v] = __builtin_isfinite(first) ? first + rest : first;
      }
      if (i16 < 4 && 4 * s + i16 < now.count()) {
        const unsigned t = ((s == 0 ? now.lo : now.hi) >> (8 * i16)) & 255;
        *reinterpret_cast<f32x4 *>(mine + t * 16 + g * 4) += sum;
      }
    }
    at = next_at;
    batch = next_batch;
    now = then;
  };
  if (at < num_groups) {
    Fetched even, odd;
    fetch(even, now, batch, true);
    in_turn((num_groups * batches - wave + W - 1) / W, even, odd, step);
  }
  __syncthreads();
  for (int n = threadIdx.x; n < a.tokens * 16; n += THREADS) {
    const int t = n >> 4, i = n & 15;
    float s = sums[n];
#pragma unroll
    for (int w = 1; w < W; ++w) s += sums[w * (kMaxTokens * 16) + n];
    const bool nan = ((t < 32 ? groups[0].lo : groups[0].hi) >> (t & 31)) & 1;
    if (row0 + i < a.hidden)
      static_cast<store *>(a.y)[static_cast<long long>(t) * a.ldy + row0 + i] =
          Elem<TYPE>::put(nan ? __builtin_nanf("") : s);
  }
}

}  // namespace mx
}  // namespace gemm
