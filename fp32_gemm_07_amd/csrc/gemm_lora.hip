// The gemm_lora* entry points (declared and documented in gemm.h): argument checks,
// choice of kernel, launches.
#include "gemm.h"

#include "host_checks.hpp"
#include "host_shared.hpp"
#include "lora_launch.hpp"

namespace {

using namespace gemm::mx;
using namespace gemm::host;

static_assert(kLoraMaxRank == GEMM_LORA_MAX_RANK && kLoraMaxAdapters == GEMM_LORA_MAX_ADAPTERS, "adapter limits");

size_t up16(size_t bytes) { return (bytes + 15) / 16 * 16; }

int check_set(int rows, const gemm_lora_t *s) {
  if (!s) return GEMM_ERR_NULL_PTR;
  if (rows < 0 || rows > GEMM_LORA_MAX_ROWS || s->K < 1 || s->K > GEMM_LORA_MAX_DIM || s->N < 1 ||
      s->N > GEMM_LORA_MAX_DIM || s->rank < 1 || s->rank > kLoraMaxRank || s->adapters < 1 ||
      s->adapters > kLoraMaxAdapters)
    return GEMM_ERR_INVALID_DIM;
  if (!valid_type(s->type)) return GEMM_ERR_INVALID_TYPE;
  return GEMM_OK;
}
Range range_a(const gemm_lora_t &s) {
  return {s.A, elem_size(s.type) * static_cast<size_t>(s.adapters) * s.rank * s.K};
}
Range range_b(const gemm_lora_t &s) {
  return {s.B, elem_size(s.type) * static_cast<size_t>(s.adapters) * s.rank * s.N};
}
Range range_ranks(const gemm_lora_t &s) { return {s.ranks, s.ranks ? 4 * static_cast<size_t>(s.adapters) : 0}; }
Range range_scales(const gemm_lora_t &s) { return {s.scales, s.scales ? 4 * static_cast<size_t>(s.adapters) : 0}; }
bool aligned_set(const gemm_lora_t &s, const int *ids) {
  return aligned(s.A, elem_size(s.type)) && aligned(s.B, elem_size(s.type)) && aligned(s.ranks, 4) &&
         aligned(s.scales, 4) && aligned(ids, 4);
}
LoraRows rows_of(int rows, const gemm_lora_t &s, const int *ids) {
  return LoraRows{rows, s.rank, s.adapters, ids, s.ranks, s.scales};
}

// How shrink is launched: 16-row tiles of a unit, waves of a workgroup, workgroups among
// which the units of a window are dealt out, and ranges that the columns are cut into. A
// window has from 4 / tiles units (one adapter) to 64 (all different).
// Many rows: units of two tiles, which halve the reads of A (8192 x 4096 bfloat16, rank 32: 20 us,
// of one tile 29; rank 16: 18 and 21), dealt out among 4 for the windows where one adapter's
// rows end and another's begin. Fewer rows: one tile, dealt out among 8. Up to 64 rows (a
// window, `few`): as many workgroups as there may be units, of 8 waves (4 above rank 64, whose
// operands take the registers), and where that leaves CUs idle ranges of 512 columns at least,
// whose sums the expand adds up (48 rows on 32 adapters of rank 64, 4096 columns: 8 ranges 11
// us, 4 14, one 25).
ShrinkPlan shrink_plan(int rows, const gemm_lora_t &s, int cus) {
  if (rows >= 16 * cus) return {2, 4, 4, 1, false};
  if (rows > 64) return {1, 4, 8, 1, false};
  const int units = std::max(1, std::min(rows, 32));
  const int splits = static_cast<int>(std::max<long long>(1, std::min<long long>({4LL * cus / units, s.K / 512, 8})));
  return {1, s.rank > 64 ? 4 : 8, units, splits, true};
}
Shrink shrink_of(const void *z, long long ldz, const void *w, int rank, int K, int splits, void *h, bool floats, void *parts) {
  const int k_split = static_cast<int>(ceil_div(ceil_div(K, splits), 64) * 64);
  return Shrink{z, ldz, w, static_cast<long long>(rank) * K, K, K, k_split, splits, h, floats, parts};
}

// Whether one kernel makes both products: where its waves' shares of K are short, and the adapters'
// A, read again for every 128 columns of Y, come to 16 MB at most if every row has another.
// In graphs, bfloat16, rank 16: 1 row of 4096 x 4096 takes 8.0 us so and 7.6 by two kernels
// (8.8 and 11.9 launched one by one), of 8192 x 8192 12.3 and 7.9, of 1024 x 1024 4.8 and 7.1;
// 8 rows of 2048 x 2048 6.7 and 8.5, 32 of 1024 x 1024 7.3 and 12.4, 16 of 4096 x 1024 7.9 and
// 9.5; rank 32, 1 row of 4096 x 4096 11.4 and 8.1.
bool one_kernel(int rows, const gemm_lora_t &s) {
  const double again = static_cast<double>(ceil_div(s.N, kSmallCols)) * rows * s.rank * s.K * elem_size(s.type);
  return rows <= 64 && s.rank <= 32 && s.K * rank_tiles(s.rank) <= 4096 && again <= 16 << 20;
}

// Bytes of what shrink leaves for expand.
size_t hidden_bytes(int rows, const gemm_lora_t &s, const ShrinkPlan &plan) {
  const size_t each = s.type != GEMM_TYPE_F32 && !plan.few ? 6 : 4 * static_cast<size_t>(plan.splits);
  return up16(each * rows * 16 * rank_tiles(s.rank));
}

// Runs body(workspace) on the caller's workspace or the library's.
template <class F>
int with_workspace(void *workspace, size_t need, int dev, hipStream_t stream, F &&body) {
  if (workspace) return body(workspace);
  return gemm::host_with_library_workspace(
      dev, need, stream,
      [](void *f, void *ws) { return ws ? (*static_cast<F *>(f))(ws) : static_cast<int>(GEMM_ERR_WORKSPACE); }, &body);
}

// ---------------------------------------------------------------------------
// Backward.

// Rows of a slot, the stretch of an adapter's rows that one workgroup sums over: as few as
// give each CU two workgroups (a slot's sums are written and read once more), 128 at least.
int slot_rows(int rows, const gemm_lora_t &s, int cus) {
  const int lane = s.type == GEMM_TYPE_F32 ? 4 : 8;
  const long long blocks = ceil_div(s.K, 16 * lane) + ceil_div(s.N, 16 * lane);
  int n = 128;
  while (n < rows && ceil_div(rows, n) * blocks > 2LL * cus) n *= 2;
  return n;
}

struct Backward {
  size_t plan, slots, sums, order, position, g, parts_h, parts_g, at, bt, partial_a, partial_b, bytes;
  int slot_rows, most_slots, positions;
};
Backward backward_layout(int rows, const gemm_lora_t &s, int cus) {
  Backward l{};
  const size_t rp = 16 * rank_tiles(s.rank), used = std::min(rows, s.adapters);
  l.slot_rows = slot_rows(rows, s, cus);
  l.most_slots = static_cast<int>(rows / l.slot_rows + used);
  l.positions = static_cast<int>((rows + 31 * used + 31) / 32 * 32);
  // partial sums of adapters with more rows than a slot
  const size_t partials = 2 * static_cast<size_t>(rows) / l.slot_rows;
  const size_t part = s.type == GEMM_TYPE_F32 ? 4 : 6;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += up16(bytes);
    return here;
  };
  l.plan = take(sizeof(LoraPlan));
  l.slots = take(sizeof(Slot) * l.most_slots);
  l.sums = take(sizeof(int2) * s.adapters);
  l.order = take(sizeof(int) * l.positions);
  l.position = take(sizeof(int) * rows);
  ShrinkPlan whole = shrink_plan(rows, s, cus);
  whole.splits = 1;
  l.g = take(hidden_bytes(rows, s, whole));
  l.parts_h = take(part * rp * l.positions);
  l.parts_g = take(part * rp * l.positions);
  l.at = take(range_a(s).bytes);
  l.bt = take(range_b(s).bytes);
  l.partial_a = take(sizeof(float) * partials * s.rank * s.K);
  l.partial_b = take(sizeof(float) * partials * s.rank * s.N);
  l.bytes = at;
  return l;
}

const LoraLaunches &lora_launches(int type) {
  return type == kF32 ? lora_launches_f32() : type == kBf16 ? lora_launches_bf16() : lora_launches_f16();
}

}  // namespace

extern "C" {

size_t gemm_lora_workspace_bytes(int rows, const gemm_lora_t *set) {
  if (check_set(rows, set) != GEMM_OK || rows == 0) return 0;
  if (one_kernel(rows, *set)) return 0;
  return hidden_bytes(rows, *set, shrink_plan(rows, *set, gemm::host_planning_cus()));
}

int gemm_lora(int rows, const gemm_lora_t *set, const int *ids, const void *X, int ldx,
              const void *C, int ldc, void *Y, int ldy, void *workspace, size_t workspace_bytes,
              hipStream_t stream) {
  int st = check_set(rows, set);
  if (st != GEMM_OK) return st;
  const gemm_lora_t &s = *set;
  if (ldx < s.K || (C && ldc < s.N) || ldy < s.N) return GEMM_ERR_INVALID_DIM;
  if (rows == 0) return GEMM_OK;
  if (!s.A || !s.B || !ids || !X || !Y) return GEMM_ERR_NULL_PTR;
  const size_t es = elem_size(s.type);
  if (!aligned_set(s, ids) || !aligned(X, es) || !aligned(C, es) || !aligned(Y, es)) return GEMM_ERR_ALIGNMENT;
  const bool in_place = C == Y && ldc == ldy;
  const Range x = {X, extent(rows, s.K, ldx, s.type)}, c = {C, C ? extent(rows, s.N, ldc, s.type) : 0};
  const Range y = {Y, extent(rows, s.N, ldy, s.type)}, id = {ids, 4 * static_cast<size_t>(rows)};
  const Range in[] = {x, range_a(s), range_b(s), range_ranks(s), range_scales(s), id, {C, in_place ? 0 : c.bytes}};
  const Range out[] = {y};
  st = check_outputs(out, in);
  if (st != GEMM_OK) return st;
  const int cus = gemm::host_planning_cus();
  const ShrinkPlan plan = shrink_plan(rows, s, cus);
  const bool one = one_kernel(rows, s);
  const size_t need = one ? 0 : hidden_bytes(rows, s, plan);
  st = check_workspace(workspace, workspace_bytes, need,
                       {x, c, y, id, range_a(s), range_b(s), range_ranks(s), range_scales(s)});
  if (st != GEMM_OK) return st;
  int dev = 0, dev_cus = 0;
  st = gemm::host_check_device(&dev, &dev_cus);
  if (st != GEMM_OK) return st;
  const LoraLaunches &launches = lora_launches(s.type);
  if (one)
    return launches.small(SmallArgs{rows_of(rows, s, ids), X, ldx, s.A, s.B, C, ldc, Y, ldy, s.N, s.K, std::min(rows, 64),
                                    in_place},
                          stream);
  return with_workspace(workspace, need, dev, stream, [&](void *ws) {
    const LoraRows r = rows_of(rows, s, ids);
    ShrinkArgs sa{};
    sa.r = r;
    sa.p[0] = shrink_of(X, ldx, s.A, s.rank, s.K, plan.splits, ws, plan.few, nullptr);
    const int launch_st = launches.shrink(sa, 1, plan, stream);
    if (launch_st != GEMM_OK) return launch_st;
    const ExpandArgs ea{r, ws, plan.splits, s.B, static_cast<long long>(s.rank) * s.N, s.rank,
                        C, ldc, Y, ldy, s.N, 1, 1, in_place};
    return launches.expand(ea, plan.few, cus, stream);
  });
}

size_t gemm_lora_backward_workspace_bytes(int rows, const gemm_lora_t *set) {
  if (check_set(rows, set) != GEMM_OK) return 0;
  return backward_layout(rows, *set, gemm::host_planning_cus()).bytes;
}

int gemm_lora_backward(int rows, const gemm_lora_t *set, const int *ids, const void *X, int ldx,
                       const void *dY, int lddy, const void *C, int ldc, void *dX, int lddx,
                       float *dA, float *dB, void *workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  int st = check_set(rows, set);
  if (st != GEMM_OK) return st;
  const gemm_lora_t &s = *set;
  const bool weights = dA || dB;   // (X is for these alone)
  if ((weights && ldx < s.K) || lddy < s.N || (dX && C && ldc < s.K) || (dX && lddx < s.K)) return GEMM_ERR_INVALID_DIM;
  if (!dX && !weights) return GEMM_OK;
  if (!dA != !dB) return GEMM_ERR_NULL_PTR;
  if (rows == 0 && !dA) return GEMM_OK;
  if (rows > 0 && (!s.A || !s.B || !ids || (weights && !X) || !dY)) return GEMM_ERR_NULL_PTR;
  const size_t es = elem_size(s.type);
  if (!aligned_set(s, ids) || (weights && !aligned(X, es)) || !aligned(dY, es) || !aligned(C, es) || !aligned(dX, es) ||
      !aligned(dA, 4) || !aligned(dB, 4))
    return GEMM_ERR_ALIGNMENT;
  const bool in_place = C == dX && ldc == lddx;
  const Range x = {X, weights ? extent(rows, s.K, ldx, s.type) : 0}, dy = {dY, extent(rows, s.N, lddy, s.type)};
  const Range c = {C, dX && C ? extent(rows, s.K, ldc, s.type) : 0}, dx = {dX, dX ? extent(rows, s.K, lddx, s.type) : 0};
  const Range id = {ids, 4 * static_cast<size_t>(rows)};
  const size_t grads = sizeof(float) * static_cast<size_t>(s.adapters) * s.rank;
  const Range da = {dA, dA ? grads * s.K : 0}, db = {dB, dB ? grads * s.N : 0};
  const Range in[] = {x, dy, range_a(s), range_b(s), range_ranks(s), range_scales(s), id, {C, in_place ? 0 : c.bytes}};
  const Range out[] = {dx, da, db};
  st = check_outputs(out, in);
  if (st != GEMM_OK) return st;
  if (in_place && (gemm::host_overlaps(C, c.bytes, dA, da.bytes) || gemm::host_overlaps(C, c.bytes, dB, db.bytes)))
    return GEMM_ERR_ALIAS;
  const int cus = gemm::host_planning_cus();
  const Backward l = backward_layout(rows, s, cus);
  st = check_workspace(workspace, workspace_bytes, l.bytes,
                       {x, dy, c, dx, da, db, id, range_a(s), range_b(s), range_ranks(s), range_scales(s)});
  if (st != GEMM_OK) return st;
  int dev = 0, dev_cus = 0;
  st = gemm::host_check_device(&dev, &dev_cus);
  if (st != GEMM_OK) return st;
  const LoraLaunches &launches = lora_launches(s.type);
  return with_workspace(workspace, l.bytes, dev, stream, [&](void *ws) {
    char *w = static_cast<char *>(ws);
    const LoraRows r = rows_of(rows, s, ids);
    ShrinkPlan plan = shrink_plan(rows, s, cus);
    plan.splits = 1;   // (the gradients' parts are of whole sums)
    LoraPlan *header = reinterpret_cast<LoraPlan *>(w + l.plan);
    Slot *slots = reinterpret_cast<Slot *>(w + l.slots);
    int2 *sums = reinterpret_cast<int2 *>(w + l.sums);
    int *order = reinterpret_cast<int *>(w + l.order), *position = reinterpret_cast<int *>(w + l.position);
    const int a_tiles = dX ? static_cast<int>(ceil_div(s.K, kTransRows)) : 0, b_tiles = static_cast<int>(ceil_div(s.N, kTransRows));
    const long long tiles = static_cast<long long>(std::min(rows, s.adapters)) * (a_tiles + b_tiles);   // at most
    const PrepareArgs pa{r, l.slot_rows, s.N, header, slots, sums, order, position, s.A, s.B, w + l.at, w + l.bt,
                         s.K, a_tiles, b_tiles};
    int launch_st = launches.prepare(pa, 1 + static_cast<int>(std::min(tiles, 2LL * cus)), stream);
    if (launch_st != GEMM_OK) return launch_st;
    void *g = w + l.g;
    if (rows > 0) {
      ShrinkArgs sa{};
      sa.r = r;
      sa.position = position;
      sa.positions = l.positions;
      sa.p[0] = shrink_of(dY, lddy, w + l.bt, s.rank, s.N, 1, dX ? g : nullptr, plan.few, dA ? w + l.parts_g : nullptr);
      if (dA) sa.p[1] = shrink_of(X, ldx, s.A, s.rank, s.K, 1, nullptr, false, w + l.parts_h);
      launch_st = launches.shrink(sa, dA ? 2 : 1, plan, stream);
      if (launch_st != GEMM_OK) return launch_st;
      if (dX) {
        const ExpandArgs ea{r, g, 1, w + l.at, static_cast<long long>(s.rank) * s.K, s.rank, C, ldc, dX, lddx, s.K, 1, 1,
                            in_place};
        launch_st = launches.expand(ea, plan.few, cus, stream);
        if (launch_st != GEMM_OK) return launch_st;
      }
    }
    if (!dA) return launch_st;
    float *partial_a = reinterpret_cast<float *>(w + l.partial_a), *partial_b = reinterpret_cast<float *>(w + l.partial_b);
    if (rows > 0) {
      const int lane = s.type == kF32 ? 4 : 8;
      const int blocks0 = static_cast<int>(ceil_div(s.K, 16 * lane)), blocks = blocks0 + static_cast<int>(ceil_div(s.N, 16 * lane));
      GradArgs ga{r, header, slots, order, l.positions,
                  {{X, ldx, s.K, w + l.parts_g, partial_a, dA}, {dY, lddy, s.N, w + l.parts_h, partial_b, dB}},
                  blocks0, blocks, 0, 16 * rank_tiles(s.rank), s.rank > 64 ? 2 : 1};
      launch_st = launches.grads(ga, l.most_slots, stream);
      if (launch_st != GEMM_OK) return launch_st;
    }
    const long long size_a = static_cast<long long>(s.rank) * s.K, size_b = static_cast<long long>(s.rank) * s.N;
    const int blocks = static_cast<int>(std::min<long long>(ceil_div(std::max(size_a, size_b), 1024), 64));
    const GradSumArgs ga{sums, {partial_a, partial_b}, {dA, dB}, {size_a, size_b}, blocks};
    return launches.sum(ga, 2 * blocks * s.adapters, stream);
  });
}

}  // extern "C"
