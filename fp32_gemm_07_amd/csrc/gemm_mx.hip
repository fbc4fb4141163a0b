// The gemm_mx* entry points (declared and documented in gemm.h): argument checks,
// choice of kernel, launches.
#include "gemm.h"

#include <algorithm>
#include <cstdint>

#include "host_checks.hpp"
#include "host_shared.hpp"
#include "mx_kernels.hpp"
#include "mx_moe.hpp"
#include "mx_tile.hpp"

namespace {

using namespace gemm::mx;
using namespace gemm::host;

static_assert(kF32 == GEMM_TYPE_F32 && kBf16 == GEMM_TYPE_BF16 && kF16 == GEMM_TYPE_F16,
              "element types");
static_assert(kMaxTokens == GEMM_MX_MOE_MAX_TOKENS && kMaxExperts == GEMM_MX_MOE_MAX_EXPERTS &&
                  kMaxTopK == GEMM_MX_MOE_MAX_TOP_K,
              "layer limits");

int padded(int K) { return static_cast<int>(ceil_div(K, kAlign) * kAlign); }
size_t codes_bytes(long long rows, int K) { return static_cast<size_t>(rows) * (padded(K) / 2); }
size_t scales_bytes(long long rows, int K) { return static_cast<size_t>(rows) * (padded(K) / 32); }
// Rows and K of an operand.
bool valid_operand(long long rows, int K) {
  return rows >= 0 && K >= 0 && K <= GEMM_MX_MAX_K && rows * static_cast<long long>(padded(K)) <= kMaxElements;
}

// ---------------------------------------------------------------------------
// Conversion.

// The checks shared by both directions; `mat` is the float matrix.
int check_convert(int trans, int rows, int K, const void *mat, int type, int ld, const void *codes,
                  const void *scales, bool to_codes) {
  const int cols = trans ? rows : K;
  const long long stored = trans ? K : rows;
  if (!valid_operand(rows, K) || ld < std::max(1, cols) || stored * ld > kMaxElements)
    return GEMM_ERR_INVALID_DIM;
  if (!valid_type(type)) return GEMM_ERR_INVALID_TYPE;
  if (rows == 0 || K == 0) return GEMM_OK;
  if (!mat || !codes || !scales) return GEMM_ERR_NULL_PTR;
  if (!aligned(mat, elem_size(type)) || !aligned(codes, 16) || !aligned(scales, 4))
    return GEMM_ERR_ALIGNMENT;
  const size_t mb = extent(stored, cols, ld, type), cb = codes_bytes(rows, K), sb = scales_bytes(rows, K);
  if (gemm::host_overlaps(mat, mb, codes, cb) || gemm::host_overlaps(mat, mb, scales, sb) ||
      (to_codes && gemm::host_overlaps(codes, cb, scales, sb)))
    return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

// Workgroups of the kernels along rows, which take whole groups of group_rows rows.
struct RowLaunch {
  RowMap map;
  long long group_rows;
  dim3 grid(int rows) const { return dim3(static_cast<unsigned>(ceil_div(rows, group_rows) * map.col_groups)); }
  // Rows of one launch.
  long long most() const { return max_blocks(256) / map.col_groups * group_rows; }
};
RowLaunch row_launch(int KP) {
  const int chunks = KP / 8;
  int log2 = 4;
  while (log2 < 8 && (1 << log2) < chunks) ++log2;
  return RowLaunch{RowMap{log2, static_cast<int>(ceil_div(chunks, 1 << log2))}, (256 >> log2) * kRowPasses};
}

// The same for the kernels across the stored rows.
struct ColumnLaunch {
  int k_tiles;
  dim3 grid(int rows) const { return dim3(static_cast<unsigned>(ceil_div(rows, kColRows) * k_tiles)); }
  long long most() const { return max_blocks(kColThreads) / k_tiles * kColRows; }
};
ColumnLaunch column_launch(int KP) { return ColumnLaunch{static_cast<int>(ceil_div(KP, kColK))}; }

// ---------------------------------------------------------------------------
// Product.
struct Product {
  int M, N, K;
  float alpha, beta;
  const unsigned char *ac, *as, *bc, *bs;
  void *C;
  int type, ldc;
};

// How a product is computed: tiles of bm x bn through a ring of `stages`, or with no
// stages the kernel for few rows of A; K cut into `splits` ranges of k_chunk.
struct ProductPlan {
  int bm, bn, stages;
  int splits, k_chunk;
};

constexpr size_t kMaxWorkspace = size_t(64) << 20;

// The time of a tile on one CU: us of a 128-value stretch of K when it has the CU to
// itself, when it shares it (or follows others on it), and of its start and end.
// Fitted on an MI355X over 20 shapes (M 1 .. 6000, K 128 .. 131072), where the
// tiles take 43, 49, 46 and 75 us in this order at 4096^3 and 37, 27, 25 and
// 39 us at 2048 x 4096 x 4096.
struct TileCost {
  int bm, bn;
  double alone, shared, ends;
};
constexpr TileCost kTiles[] = {
    {256, 256, 0.94, 0.94, 8.8},
    {256, 128, 0.55, 0.55, 5.5},
    {128, 128, 0.33, 0.31, 1.2},
    {64, 64, 0.125, 0.12, 0.9},
};
// The sum of split partial sums: its launch, and bytes a us.
constexpr double kSumUs = 3.0, kSumBytesPerUs = 4.5e6;

ProductPlan plan_product(int M, int N, int K, int cus) {
  const int KP = padded(K);
  ProductPlan best{};
  double best_us = 1e30;
  for (const TileCost &c : kTiles) {
    const long long tiles = ceil_div(M, c.bm) * ceil_div(N, c.bn);
    for (int s = 1; s <= 64; s *= 2) {
      // ranges of whole stages of 256
      const int chunk = s == 1 ? KP : static_cast<int>(ceil_div(ceil_div(KP, s), 256) * 256);
      const int splits = static_cast<int>(ceil_div(KP, chunk));
      const double partial = 4.0 * splits * M * static_cast<double>(N);
      if (s > 1 && (chunk < 512 || partial > kMaxWorkspace)) break;
      const long long rounds = ceil_div(tiles * splits, cus);
      double us = rounds * (chunk / kAlign * (rounds > 1 ? c.shared : c.alone) + c.ends);
      if (splits > 1) us += kSumUs + 2 * partial / kSumBytesPerUs;
      if (us < best_us * 0.99) {
        best_us = us;
        // Two workgroups of 128 x 128 share a CU; where there is one for each CU at most
        // it takes twice the stages instead (512 x 512 x 131072: 34 us against 39).
        const int stages = c.bm == 64 || (c.bm == 128 && tiles * splits <= cus) ? 4 : 2;
        best = ProductPlan{c.bm, c.bn, stages, splits, chunk};
      }
    }
  }
  // Few rows: a round of one workgroup (16 rows of B) a CU takes 2.2 us for each 4
  // chunks of its 8 waves, 4.5 with two tiles of A's rows, less a little (no stages
  // to fill). 1 x 4096 x 4096: 5.2 us against 7.4 (64 x 64, 4 splits); 32 x 4096 x
  // 4096: 7.6 against 8.3; 24 x 8192 x 4096: 11.6 against 9.5 (64 x 64, whole).
  if (M <= 32) {
    const long long rounds = ceil_div(ceil_div(N, 16), cus);
    const double us = rounds * ceil_div(KP / kAlign, kSkinnyWaves * kSkinnyAt) * (M <= 16 ? 2.2 : 4.5) - 0.3;
    if (us < best_us) best = ProductPlan{M <= 16 ? 16 : 32, 16, 0, 1, KP};
  }
  return best;
}

size_t product_workspace(int M, int N, int K, int cus) {
  const ProductPlan plan = plan_product(M, N, K, cus);
  return plan.splits > 1 ? size_t(4) * plan.splits * M * N : 0;
}

template <int BM, int BN, int NS, int WPE>
int launch_tile(const Product &p, const ProductPlan &plan, void *ws, hipStream_t stream) {
  const int KP = padded(p.K);
  if (plan.splits > 1) {   // few tiles: the partial sums fit the workspace
    const long long tm = ceil_div(p.M, BM), tn = ceil_div(p.N, BN);
    const TileArgs a{p.ac, p.as, p.bc, p.bs, ws, p.M, p.N, KP, p.ldc, p.alpha, p.beta, plan.k_chunk,
                     static_cast<int>(tm), static_cast<int>(tn), plan.splits};
    hipLaunchKernelGGL((tile_kernel<BM, BN, NS, kF32, true, WPE>),
                       dim3(static_cast<unsigned>(tm * tn * plan.splits)), dim3(256), 0, stream, a);
    return launched();
  }
  // A launch takes as many columns of C as it can, and as many rows of those.
  const long long wide = std::min(ceil_div(p.N, BN), max_blocks(256));
  return in_ranges(p.N, wide * BN, [&](long long n0, int N) {
    return in_ranges(p.M, max_blocks(256) / wide * BM, [&](long long m0, int M) {
      const long long tm = ceil_div(M, BM), tn = ceil_div(N, BN);
      const TileArgs a{p.ac + m0 * (KP / 2), p.as + m0 * (KP / 32), p.bc + n0 * (KP / 2), p.bs + n0 * (KP / 32),
                       static_cast<char *>(p.C) + (m0 * p.ldc + n0) * static_cast<long long>(elem_size(p.type)),
                       M, N, KP, p.ldc, p.alpha, p.beta, plan.k_chunk, static_cast<int>(tm),
                       static_cast<int>(tn), 1};
      with_type(p.type, [&](auto t) {
        hipLaunchKernelGGL((tile_kernel<BM, BN, NS, decltype(t)::value, false, WPE>),
                           dim3(static_cast<unsigned>(tm * tn)), dim3(256), 0, stream, a);
      });
      return launched();
    });
  });
}

int launch_product(const Product &p, void *ws, int cus, hipStream_t stream) {
  ProductPlan plan = plan_product(p.M, p.N, p.K, cus);
  if (plan.splits > 1 && !ws) {   // no workspace to be had: no split
    plan.splits = 1;
    plan.k_chunk = padded(p.K);
  }
  int st = GEMM_OK;
  if (plan.bn == 256) st = launch_tile<256, 256, 2, 1>(p, plan, ws, stream);
  else if (plan.bm == 256) st = launch_tile<256, 128, 2, 1>(p, plan, ws, stream);
  else if (plan.bm == 128 && plan.stages == 4) st = launch_tile<128, 128, 4, 1>(p, plan, ws, stream);
  else if (plan.bm == 128) st = launch_tile<128, 128, 2, 2>(p, plan, ws, stream);
  else if (plan.bm == 64) st = launch_tile<64, 64, 4, 2>(p, plan, ws, stream);
  else {
    // (One launch: with more workgroups than one takes a tile is always chosen above.)
    with_type(p.type, [&](auto t) {
      constexpr int T = decltype(t)::value;
      auto *kernel = plan.bm == 16 ? skinny_kernel<T, 1> : skinny_kernel<T, 2>;
      hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(ceil_div(p.N, 16))),
                         dim3(64 * kSkinnyWaves), 0, stream, p.ac, p.as, p.bc, p.bs,
                         static_cast<typename Elem<T>::store *>(p.C), p.M, p.N, padded(p.K), p.ldc,
                         p.alpha, p.beta);
    });
    st = launched();
  }
  if (st != GEMM_OK || plan.splits == 1) return st;
  const long long count = static_cast<long long>(p.M) * p.N;
  const unsigned blocks = static_cast<unsigned>(std::min<long long>(ceil_div(count, 256), 8LL * cus));
  with_type(p.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    hipLaunchKernelGGL(split_reduce_kernel<T>, dim3(blocks), dim3(256), 0, stream,
                       static_cast<const float *>(ws), static_cast<typename Elem<T>::store *>(p.C),
                       count, p.N, p.ldc, plan.splits, p.alpha, p.beta);
  });
  return launched();
}

int launch_scale(const Product &p, int cus, hipStream_t stream) {
  const long long count = static_cast<long long>(p.M) * p.N;
  const unsigned blocks = static_cast<unsigned>(std::min<long long>(ceil_div(count, 256), 4LL * cus));
  with_type(p.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    hipLaunchKernelGGL(scale_kernel<T>, dim3(blocks), dim3(256), 0, stream,
                       static_cast<typename Elem<T>::store *>(p.C), count, p.N, p.ldc, p.beta);
  });
  return launched();
}

int check_product(const Product &p) {
  if (p.M < 0 || p.N < 0 || p.K < 0) return GEMM_ERR_INVALID_DIM;
  if (!valid_operand(p.M, p.K) || !valid_operand(p.N, p.K) || p.ldc < std::max(1, p.N) ||
      static_cast<long long>(p.M) * p.ldc > kMaxElements)
    return GEMM_ERR_INVALID_DIM;
  if (!valid_type(p.type)) return GEMM_ERR_INVALID_TYPE;
  if (p.M == 0 || p.N == 0) return GEMM_OK;
  if (!p.C) return GEMM_ERR_NULL_PTR;
  const bool uses = p.K > 0 && p.alpha != 0.0f;
  if (uses && (!p.ac || !p.as || !p.bc || !p.bs)) return GEMM_ERR_NULL_PTR;
  if (!aligned(p.C, elem_size(p.type))) return GEMM_ERR_ALIGNMENT;
  if (!uses) return GEMM_OK;
  if (!aligned(p.ac, 16) || !aligned(p.bc, 16) || !aligned(p.as, 4) || !aligned(p.bs, 4))
    return GEMM_ERR_ALIGNMENT;
  const size_t c = extent(p.M, p.N, p.ldc, p.type);
  if (gemm::host_overlaps(p.C, c, p.ac, codes_bytes(p.M, p.K)) ||
      gemm::host_overlaps(p.C, c, p.as, scales_bytes(p.M, p.K)) ||
      gemm::host_overlaps(p.C, c, p.bc, codes_bytes(p.N, p.K)) ||
      gemm::host_overlaps(p.C, c, p.bs, scales_bytes(p.N, p.K)))
    return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

// ---------------------------------------------------------------------------
// The mixture-of-experts layer.
constexpr size_t kGroupBytes = (kMaxGroups + 1) * sizeof(Group) / 16 * 16 + 16;   // the workspace's head

size_t moe_workspace(int tokens, int inter, int top_k, int type) {
  const size_t words = type == kF32 ? Parts<kF32>::h_words : Parts<kBf16>::h_words;
  const size_t hidden = words * sizeof(u16) * static_cast<size_t>(tokens) * top_k * padded(inter);
  return hidden + kGroupBytes;
}

// Both kernels for groups of GROUP tokens, RESIDENT: their activations kept in LDS.
template <int TYPE, int GROUP, bool RESIDENT>
int launch_moe_groups(const MoeArgs &a, int cus, hipStream_t stream) {
  const long long pairs = static_cast<long long>(a.tokens) * a.top_k;
  const long long groups = std::min<long long>(pairs, a.experts) + pairs / GROUP;
  const dim3 up(static_cast<unsigned>(std::min<long long>(groups * (padded(a.inter) / 16), cus)));
  const dim3 down(static_cast<unsigned>(ceil_div(a.hidden, 16)));
  hipLaunchKernelGGL((moe_up_kernel<TYPE, GROUP, RESIDENT>), up, dim3(kMoeThreads), 0, stream, a);
  const int st = launched();
  if (st != GEMM_OK) return st;
  hipLaunchKernelGGL((moe_down_kernel<TYPE, GROUP>), down, dim3(64 * kDownWaves<TYPE>), 0, stream, a);
  return launched();
}

template <int TYPE, int GROUP>
bool activations_fit(const MoeArgs &a) {
  return static_cast<long long>(padded(a.hidden)) / 128 * Parts<TYPE>::x * GROUP * 256 <= kUpStage<GROUP>;
}

int launch_moe(const MoeArgs &a, int type, int cus, hipStream_t stream) {
  int st = GEMM_OK;
  with_type(type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    // Groups of 8 where an expert has more than 3 tokens on average (its weights are
    // then read once for 8 of them), else of 4 (fewer activations to move and split):
    // with 2, 2.5, 3 and 4 tokens for each of 128 experts of 4096 x 1024 (bfloat16) groups
    // of 4 take 177, 200, 220 and 261 us, of 8 202, 214, 218 and 233; with 2, 3, 4 and 16
    // for each of 8 of 4096 x 2048 32, 38, 40 and 104 us against 38, 39, 41 and 81; with 3
    // and 6 for each of 16 of 2048 x 1024 32 and 45 us against 35 and 41 in half, 33 and 46
    // against 37 and 44 in FP32.
    if (static_cast<long long>(a.tokens) * a.top_k > 3LL * a.experts && activations_fit<T, 8>(a))
      st = launch_moe_groups<T, 8, true>(a, cus, stream);
    else if (activations_fit<T, 4>(a))
      st = launch_moe_groups<T, 4, true>(a, cus, stream);
    else
      st = launch_moe_groups<T, 4, false>(a, cus, stream);
  });
  return st;
}

int check_moe(const MoeArgs &a, int type, bool routed) {
  if (a.tokens < 0 || a.tokens > kMaxTokens || a.hidden < 1 || a.inter < 1 || a.experts < 1 ||
      a.experts > kMaxExperts || a.top_k < 1 || a.top_k > std::min(kMaxTopK, a.experts) ||
      (!routed && a.ld_logits < a.experts) || a.ldx < a.hidden || a.ldy < a.hidden)
    return GEMM_ERR_INVALID_DIM;
  const long long rows1 = 2LL * a.experts * a.inter, rows2 = static_cast<long long>(a.experts) * a.hidden;
  if (!valid_operand(rows1, a.hidden) || !valid_operand(rows2, a.inter)) return GEMM_ERR_INVALID_DIM;
  if (!valid_type(type)) return GEMM_ERR_INVALID_TYPE;
  if (a.tokens == 0) return GEMM_OK;
  if ((routed ? !a.chosen || !a.weights : !a.logits) || !a.x || !a.y || !a.w1c || !a.w1s || !a.w2c || !a.w2s) return GEMM_ERR_NULL_PTR;
  const size_t es = elem_size(type);
  if (!aligned(a.logits, 4) || !aligned(a.chosen, 4) || !aligned(a.weights, 4) || !aligned(a.x, es) || !aligned(a.y, es) || !aligned(a.w1c, 16) ||
      !aligned(a.w2c, 16) || !aligned(a.w1s, 4) || !aligned(a.w2s, 4))
    return GEMM_ERR_ALIGNMENT;
  const size_t y = extent(a.tokens, a.hidden, a.ldy, type);
  const size_t logits = routed ? 0 : extent(a.tokens, a.experts, a.ld_logits, kF32);
  const size_t choices = routed ? 4 * static_cast<size_t>(a.tokens) * a.top_k : 0;
  if (gemm::host_overlaps(a.y, y, a.logits, logits) || gemm::host_overlaps(a.y, y, a.chosen, choices) ||
      gemm::host_overlaps(a.y, y, a.weights, choices) ||
      gemm::host_overlaps(a.y, y, a.x, extent(a.tokens, a.hidden, a.ldx, type)) ||
      gemm::host_overlaps(a.y, y, a.w1c, codes_bytes(rows1, a.hidden)) ||
      gemm::host_overlaps(a.y, y, a.w1s, scales_bytes(rows1, a.hidden)) ||
      gemm::host_overlaps(a.y, y, a.w2c, codes_bytes(rows2, a.inter)) ||
      gemm::host_overlaps(a.y, y, a.w2s, scales_bytes(rows2, a.inter)))
    return GEMM_ERR_ALIAS;
  return GEMM_OK;
}

int run_moe(MoeArgs a, int type, bool routed, void *workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_moe(a, type, routed);
  if (st != GEMM_OK || a.tokens == 0) return st;
  const size_t need = moe_workspace(a.tokens, a.inter, a.top_k, type);
  const long long rows1 = 2LL * a.experts * a.inter, rows2 = static_cast<long long>(a.experts) * a.hidden;
  const size_t choices = routed ? 4 * static_cast<size_t>(a.tokens) * a.top_k : 0;
  st = check_workspace(workspace, workspace_bytes, need,
                       {{a.y, extent(a.tokens, a.hidden, a.ldy, type)}, {a.x, extent(a.tokens, a.hidden, a.ldx, type)},
                        {a.logits, routed ? 0 : extent(a.tokens, a.experts, a.ld_logits, kF32)},
                        {a.chosen, choices}, {a.weights, choices},
                        {a.w1c, codes_bytes(rows1, a.hidden)}, {a.w1s, scales_bytes(rows1, a.hidden)},
                        {a.w2c, codes_bytes(rows2, a.inter)}, {a.w2s, scales_bytes(rows2, a.inter)}});
  if (st != GEMM_OK) return st;
  int dev = 0, cus = 0;
  st = gemm::host_check_device(&dev, &cus);
  if (st != GEMM_OK) return st;
  struct Call {
    MoeArgs *a;
    int type, cus;
    hipStream_t stream;
  } call{&a, type, cus, stream};
  auto body = [](void *c, void *ws) {
    const Call *k = static_cast<const Call *>(c);
    if (!ws) return static_cast<int>(GEMM_ERR_WORKSPACE);
    k->a->groups = static_cast<Group *>(ws);
    k->a->h = reinterpret_cast<u16 *>(static_cast<char *>(ws) + kGroupBytes);
    return launch_moe(*k->a, k->type, k->cus, k->stream);
  };
  if (workspace) return body(&call, workspace);
  return gemm::host_with_library_workspace(dev, need, stream, body, &call);
}

}  // namespace

extern "C" {

size_t gemm_mx_codes_bytes(int rows, int K) {
  return valid_operand(rows, K) ? codes_bytes(rows, K) : 0;
}

size_t gemm_mx_scales_bytes(int rows, int K) {
  return valid_operand(rows, K) ? scales_bytes(rows, K) : 0;
}

int gemm_mx_quantize(int trans, int rows, int K, const void *X, int x_type, int ldx, void *codes,
                     void *scales, hipStream_t stream) {
  int st = check_convert(trans, rows, K, X, x_type, ldx, codes, scales, true);
  if (st != GEMM_OK || rows == 0 || K == 0) return st;
  int dev = 0, cus = 0;
  st = gemm::host_check_device(&dev, &cus);
  if (st != GEMM_OK) return st;
  const int KP = padded(K);
  with_type(x_type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    const typename Elem<T>::store *x = static_cast<const typename Elem<T>::store *>(X);
    // codes and scales of row r
    auto c = [&](long long r) { return static_cast<unsigned *>(codes) + r * (KP / 8); };
    auto s = [&](long long r) { return static_cast<unsigned char *>(scales) + r * (KP / 32); };
    if (trans) {
      const ColumnLaunch l = column_launch(KP);
      st = in_ranges(rows, l.most(), [&](long long r, int n) {
        hipLaunchKernelGGL(quantize_columns_kernel<T>, l.grid(n), dim3(kColThreads), 0, stream, x + r, ldx,
                           c(r), reinterpret_cast<unsigned *>(s(r)), n, K, KP, l.k_tiles);
        return launched();
      });
    } else {
      const RowLaunch l = row_launch(KP);
      st = in_ranges(rows, l.most(), [&](long long r, int n) {
        hipLaunchKernelGGL(quantize_rows_kernel<T>, l.grid(n), dim3(256), 0, stream, x + r * ldx, ldx,
                           c(r), s(r), n, K, KP, l.map);
        return launched();
      });
    }
  });
  return st;
}

int gemm_mx_dequantize(int trans, int rows, int K, const void *codes, const void *scales, void *Y,
                       int y_type, int ldy, hipStream_t stream) {
  int st = check_convert(trans, rows, K, Y, y_type, ldy, codes, scales, false);
  if (st != GEMM_OK || rows == 0 || K == 0) return st;
  int dev = 0, cus = 0;
  st = gemm::host_check_device(&dev, &cus);
  if (st != GEMM_OK) return st;
  const int KP = padded(K);
  with_type(y_type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    typename Elem<T>::store *y = static_cast<typename Elem<T>::store *>(Y);
    auto c = [&](long long r) { return static_cast<const unsigned *>(codes) + r * (KP / 8); };
    auto s = [&](long long r) { return static_cast<const unsigned char *>(scales) + r * (KP / 32); };
    if (trans) {
      const ColumnLaunch l = column_launch(KP);
      st = in_ranges(rows, l.most(), [&](long long r, int n) {
        hipLaunchKernelGGL(dequantize_columns_kernel<T>, l.grid(n), dim3(kColThreads), 0, stream, c(r), s(r),
                           y + r, ldy, n, K, KP, l.k_tiles);
        return launched();
      });
    } else {
      const RowLaunch l = row_launch(KP);
      st = in_ranges(rows, l.most(), [&](long long r, int n) {
        hipLaunchKernelGGL(dequantize_rows_kernel<T>, l.grid(n), dim3(256), 0, stream, c(r), s(r),
                           y + r * ldy, ldy, n, K, KP, l.map);
        return launched();
      });
    }
  });
  return st;
}

size_t gemm_mx_workspace_bytes(int M, int N, int K) {
  if (M <= 0 || N <= 0 || K <= 0 || !valid_operand(M, K) || !valid_operand(N, K)) return 0;
  return product_workspace(M, N, K, gemm::host_planning_cus());
}

int gemm_mx_plan(int M, int N, int K, gemm_mx_plan_t *out) {
  if (!out) return GEMM_ERR_NULL_PTR;
  if (M < 1 || N < 1 || K < 1 || !valid_operand(M, K) || !valid_operand(N, K)) return GEMM_ERR_INVALID_DIM;
  const ProductPlan plan = plan_product(M, N, K, gemm::host_planning_cus());
  *out = gemm_mx_plan_t{plan.bm, plan.bn, plan.stages, plan.splits, plan.k_chunk};
  return GEMM_OK;
}

int gemm_mx(int M, int N, int K, float alpha, const void *A_codes, const void *A_scales,
            const void *B_codes, const void *B_scales, float beta, void *C, int c_type, int ldc,
            void *workspace, size_t workspace_bytes, hipStream_t stream) {
  const Product p{M, N, K, alpha, beta,
                  static_cast<const unsigned char *>(A_codes), static_cast<const unsigned char *>(A_scales),
                  static_cast<const unsigned char *>(B_codes), static_cast<const unsigned char *>(B_scales),
                  C, c_type, ldc};
  int st = check_product(p);
  if (st != GEMM_OK || M == 0 || N == 0) return st;
  const bool uses = K > 0 && alpha != 0.0f;
  const int cus = gemm::host_planning_cus();
  const size_t need = uses ? product_workspace(M, N, K, cus) : 0;
  st = check_workspace(workspace, workspace_bytes, need,
                       {{C, extent(M, N, ldc, c_type)}, {A_codes, codes_bytes(M, K)},
                        {A_scales, scales_bytes(M, K)}, {B_codes, codes_bytes(N, K)},
                        {B_scales, scales_bytes(N, K)}});
  if (st != GEMM_OK) return st;
  int dev = 0, dev_cus = 0;
  st = gemm::host_check_device(&dev, &dev_cus);
  if (st != GEMM_OK) return st;
  if (!uses) return launch_scale(p, cus, stream);
  if (workspace || need == 0) return launch_product(p, workspace, cus, stream);
  struct Call {
    const Product *p;
    int cus;
    hipStream_t stream;
  } call{&p, cus, stream};
  return gemm::host_with_library_workspace(
      dev, need, stream,
      [](void *c, void *ws) {
        const Call *k = static_cast<const Call *>(c);
        return launch_product(*k->p, ws, k->cus, k->stream);
      },
      &call);
}

size_t gemm_mx_moe_workspace_bytes(int tokens, int inter, int top_k, int x_type) {
  if (tokens < 1 || tokens > kMaxTokens || top_k < 1 || top_k > kMaxTopK || inter < 1 ||
      inter > GEMM_MX_MAX_K || !valid_type(x_type))
    return 0;
  return moe_workspace(tokens, inter, top_k, x_type);
}

int gemm_mx_moe(int tokens, int hidden, int inter, int experts, int top_k, int renormalize,
                const float *logits, int ld_logits, const void *X, int x_type, int ldx,
                const void *W1_codes, const void *W1_scales, const void *W2_codes,
                const void *W2_scales, void *Y, int ldy, void *workspace, size_t workspace_bytes,
                hipStream_t stream) {
  const MoeArgs a{tokens, hidden, inter, experts, top_k, renormalize != 0, logits, ld_logits, nullptr, nullptr, X, ldx,
                  static_cast<const unsigned char *>(W1_codes), static_cast<const unsigned char *>(W1_scales),
                  static_cast<const unsigned char *>(W2_codes), static_cast<const unsigned char *>(W2_scales),
                  Y, ldy, nullptr, nullptr};
  return run_moe(a, x_type, false, workspace, workspace_bytes, stream);
}

int gemm_mx_moe_routed(int tokens, int hidden, int inter, int experts, int top_k,
                       const int *chosen, const float *weights, const void *X, int x_type, int ldx,
                       const void *W1_codes, const void *W1_scales, const void *W2_codes,
                       const void *W2_scales, void *Y, int ldy, void *workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  const MoeArgs a{tokens, hidden, inter, experts, top_k, 0, nullptr, 0, chosen, weights, X, ldx,
                  static_cast<const unsigned char *>(W1_codes), static_cast<const unsigned char *>(W1_scales),
                  static_cast<const unsigned char *>(W2_codes), static_cast<const unsigned char *>(W2_scales),
                  Y, ldy, nullptr, nullptr};
  return run_moe(a, x_type, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
