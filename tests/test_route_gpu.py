"""gemm_route, gemm_route_backward and gemm_mx_moe_routed on the GPU against
tests/rows_reference.py and tests/mx_reference.py (NumPy, float64): choices and counts
equal, weights and gradients within bounds derived beside them.

Inputs lie inside NaN-filled buffers, outputs inside ones filled with a sentinel that has
to survive."""
import numpy as np
import pytest

import mx_reference as mxref
import rows_reference as ref
from fp32_gemm_07_amd import binding as lib
from gpu_util import say, torch

pytestmark = pytest.mark.gpu

KINDS = {"f32": 0, "bf16": 1, "f16": 2}
SENTINEL = -77


@pytest.fixture(scope="module", autouse=True)
def _setup():
    lib.load()
    torch()


def dtype(kind):
    t = torch()
    return {"f32": t.float32, "bf16": t.bfloat16, "f16": t.float16}[kind]


def stream():
    return torch().cuda.current_stream().cuda_stream


def dev(x, kind="f32"):
    return torch().from_numpy(np.ascontiguousarray(x, np.float32)).to("cuda:0").to(dtype(kind))


def padded(x, kind, pad, offset=0):
    """x stored with `pad` NaN elements behind every row, `offset` elements into its buffer."""
    rows, cols = x.shape
    buf = np.full(offset + rows * (cols + pad), np.nan, np.float32)
    buf[offset:].reshape(rows, cols + pad)[:, :cols] = x
    return dev(buf, kind)[offset:], cols + pad


def ints(n):
    return torch().full((n + 8,), SENTINEL, dtype=torch().int32, device="cuda:0")


def floats(n):
    return torch().full((n + 8,), float(SENTINEL), device="cuda:0")


def run_route(l, kind, bias, r, pad=0, offset=0, counts=True):
    """(chosen, weights, counts) NumPy, sentinels checked."""
    T, E = l.shape
    x, ld = padded(l, kind, pad, offset)
    router = lib.gemm_route_t(E, r.top_k, r.score, r.groups, r.top_groups, r.group_top, r.renormalize, r.scale)
    c, w, n = ints(T * r.top_k), floats(T * r.top_k), ints(E)
    lib.gemm_route(T, router, x, KINDS[kind], ld, None if bias is None else dev(bias), c, w, n if counts else None, stream())
    c, w, n = c.cpu().numpy(), w.cpu().numpy(), n.cpu().numpy()
    k = T * r.top_k
    assert (c[k:] == SENTINEL).all() and (w[k:] == SENTINEL).all() and (n[E:] == SENTINEL).all()
    if not counts:
        assert (n == SENTINEL).all()
    return c[:k].reshape(T, -1), w[:k].reshape(T, -1), n[:E]


def weight_bound(l, chosen, weights):
    """Bound on a weight's error. A quotient of an exponential and a sum of at most 512 of them: an
    exponential of x, its argument one rounding off, has |x| 2^-24 + 2 steps of its own; the terms that
    make up the sum have |x| < 21 (smaller ones come to less than 512 e^-21 < 2^-21 of it, whatever their error, here taken
    at |x| 2^-24 of that); 36 additions, a division, a product and the sigmoid's own 1 + e^-x."""
    top = np.where(np.isfinite(l), l, -np.inf).max(axis=1, keepdims=True)
    picked = np.take_along_axis(l, np.maximum(chosen, 0), axis=1)
    span = np.where(chosen >= 0, np.abs(top) + np.abs(picked), 0)
    return np.abs(weights) * (np.minimum(span, 200) + 100) * 2.0 ** -24 + 2.0 ** -126


def check_route(l, kind, bias, r, what, **more):
    say(what)
    chosen, weights, counts = run_route(l, kind, bias, r, **more)
    ec, ew, en = ref.route(l.astype(np.float64), None if bias is None else bias.astype(np.float64), r)
    assert np.array_equal(chosen, ec), what
    assert np.array_equal(np.isnan(weights), np.isnan(ew)), what
    fine = ~np.isnan(ew)
    bound = weight_bound(l.astype(np.float64), ec, ew)
    assert (np.abs(weights - ew)[fine] <= bound[fine]).all(), (what, np.nanmax(np.abs(weights - ew) / bound))
    if more.get("counts", True):
        assert np.array_equal(counts, en), what
    return chosen


def logits(rng, T, E, kind):
    return mxref.to_type(rng.normal(size=(T, E)) * 1.5 + rng.normal(size=(1, E)) * 0.5, KINDS[kind])


CASES = [  # tokens, experts, top_k, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 128, 8, 1, 1, 1), (3, 5, 5, 1, 1, 1), (17, 64, 4, 1, 1, 1), (64, 65, 16, 1, 1, 1), (65, 96, 6, 6, 3, 1),
    (130, 256, 8, 8, 4, 2), (33, 512, 16, 64, 7, 2), (70, 510, 9, 3, 2, 2), (31, 60, 3, 60, 3, 2), (50, 129, 4, 43, 2, 2), (1030, 24, 2, 2, 1, 1),
    (64, 300, 7, 10, 9, 2), (8, 16, 16, 4, 4, 2)]


@pytest.mark.parametrize("T,E,k,g,tg,gt", CASES)
@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("kind", KINDS)
def test_route(T, E, k, g, tg, gt, score, kind):
    rng = np.random.default_rng(T * 1000 + E + k)
    l = logits(rng, T, E, kind)
    for bias in (None, (0.1 * rng.normal(size=E)).astype(np.float32)):
        for renormalize in (False, True):
            r = ref.Router(E, k, score, g, tg, gt, renormalize, 2.5)
            check_route(l, kind, bias, r, f"route {T}x{E} top {k} groups {g}/{tg}/{gt} {score} {kind} bias {bias is not None} renorm {renormalize}",
                        pad=T % 3, offset=E % 2)


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
def test_many_tokens(score):
    """More tokens than the grid has rows, and the counts of several workgroups."""
    rng = np.random.default_rng(3)
    l = logits(rng, 40000, 12, "f32")
    check_route(l, "f32", None, ref.Router(12, 2, score, renormalize=True), f"route 40000x12 {score}")
    check_route(l, "f32", (0.1 * rng.normal(size=12)).astype(np.float32), ref.Router(12, 3, score, 4, 2, 2), f"route 40000x12 bias {score}", counts=False)


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("bias", [False, True])
def test_ties_and_masks(score, bias):
    """Ties go to the lowest index; -inf is never chosen, the type's lowest value is; rows with
    too few experts, none, a NaN, +inf."""
    rng = np.random.default_rng(8)
    T, E = 64, 48
    l = rng.integers(-2, 3, (T, E)).astype(np.float32)
    l[0] = 0.0
    l[1, ::2] = -0.0
    l[2] = -np.inf
    l[3] = -np.inf
    l[3, [7, 40]] = 1.0
    l[4, 9] = np.nan
    l[5, 11] = np.inf
    l[6] = np.finfo(np.float32).min
    l[7] = -np.inf
    l[7, 5] = np.finfo(np.float32).min
    l[8] = np.where(np.arange(E) < 20, -np.inf, l[8])
    l[9] = 80.0 + rng.integers(0, 3, E)
    l[10] = -80.0 - rng.integers(0, 3, E)
    l[11] = np.where(np.arange(E) % 16 == 3, 0.5, -np.inf)
    b = np.zeros(E, np.float32) if bias else None
    for g, tg, gt in ((1, 1, 1), (4, 2, 1), (4, 2, 2), (16, 4, 2)):
        for renormalize in (False, True):
            check_route(l, "f32", b, ref.Router(E, 6, score, g, tg, gt, renormalize), f"ties {score} bias {bias} groups {g} {tg} {gt}")
    if bias:
        b[3] = -np.inf
        b[20] = np.inf
        b[21] = np.inf
        check_route(l, "f32", b, ref.Router(E, 6, score, 1, 1, 1, True), "an infinite bias")
        check_route(l, "f32", b, ref.Router(E, 6, score, 4, 2, 2, True), "an infinite bias, groups")
        b[5] = np.nan
        check_route(l, "f32", b, ref.Router(E, 6, score), "a NaN in the bias")


def test_values_next_to_each_other():
    """Scores plus bias that FP32 would call equal, or order the other way round, are told apart."""
    E = 32
    l = np.full((1, E), -4.0, np.float32)
    l[0, 3], l[0, 17] = 12.0, 12.000001          # sigmoids 1 - 6e-6, 6e-12 apart
    b = np.zeros(E, np.float32)
    check_route(l, "f32", b, ref.Router(E, 1, ref.SIGMOID), "sigmoids 6e-12 apart")
    l[0, 3], l[0, 17] = 12.000001, 12.0
    check_route(l, "f32", b, ref.Router(E, 2, ref.SIGMOID), "and in the other order")
    b[17] = 2.0 ** -36                            # more than they differ by
    check_route(l, "f32", b, ref.Router(E, 2, ref.SIGMOID), "a bias of 2^-36")
    b[:] = 1000.0                                 # FP32 sums would all round alike
    check_route(l, "f32", b, ref.Router(E, 2, ref.SOFTMAX), "a large bias")


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
def test_logits_next_to_each_other(score):
    """Logits that differ by less than FP64 scores tell are told apart where there is no bias; groups
    whose two best scores are the same tie, to the lowest."""
    E = 24
    l = np.full((3, E), -2.0, np.float32)
    l[0, [5, 11]] = [1e-30, 2e-30]                # groups of 6: two in the first two
    l[0, [12, 18]] = 2e-30
    l[1, [3, 9, 15, 21]] = [40.0, 41.0, 42.0, 40.5]
    l[2] = 0.0
    for g, tg, gt in ((1, 1, 1), (4, 2, 1), (4, 2, 2), (4, 3, 2)):
        check_route(l, "f32", None, ref.Router(E, 4, score, g, tg, gt, True), f"logits next to each other {score} groups {g} {tg} {gt}")


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
def test_near_ties_everywhere(score):
    """Values a few FP32 steps apart in every token: estimates settle nothing, by groups or by experts, with
    more near each other than there are candidates."""
    rng = np.random.default_rng(12)
    T, E = 40, 96
    l = (1.0 + rng.integers(0, 9, (T, E)) * 2.0 ** -22).astype(np.float32)
    b = (rng.integers(-3, 4, E) * 2.0 ** -23).astype(np.float32)
    for g, tg, gt in ((1, 1, 1), (8, 3, 1), (8, 3, 2), (48, 20, 2)):
        for k in (1, 6, 16):
            check_route(l, "f32", b, ref.Router(E, k, score, g, tg, gt, True), f"near ties {score} groups {g} {tg} {gt} top {k}")


def test_no_tokens_zero_the_counts():
    n = ints(16)
    lib.gemm_route(0, lib.gemm_route_t(16, 2), None, 0, 16, None, None, None, n, stream())
    n = n.cpu().numpy()
    assert (n[:16] == 0).all() and (n[16:] == SENTINEL).all()


def run_backward(l, kind, chosen, dw, r, pad=0, offset=0):
    T, E = l.shape
    x, ld = padded(l, kind, pad, offset)
    router = lib.gemm_route_t(E, r.top_k, r.score, r.groups, r.top_groups, r.group_top, r.renormalize, r.scale)
    ldd = E + pad + 1
    out = torch().full((T * ldd + 8,), float(SENTINEL), device="cuda:0").to(dtype(kind))
    lib.gemm_route_backward(T, router, x, KINDS[kind], ld, torch().from_numpy(np.ascontiguousarray(chosen, np.int32)).to("cuda:0"), dev(dw), out, ldd,
                            stream())
    out = out.float().cpu().numpy()
    assert (out[T * ldd:] == SENTINEL).all()
    out = out[:T * ldd].reshape(T, ldd)
    assert (out[:, E:] == SENTINEL).all()
    return out[:, :E]


def check_backward(l, kind, chosen, dw, r, what, **more):
    say(what)
    got = run_backward(l, kind, chosen, dw, r, **more)
    l64 = l.astype(np.float64)
    d, mag = ref.route_backward(l64, chosen, dw.astype(np.float64), r)
    # every factor is off as a weight is (see weight_bound), three of them and 20 additions; then
    # the rounding to the type, at its smallest numbers half a step of those
    top = np.where(np.isfinite(l64), l64, -np.inf).max(axis=1, keepdims=True)
    span = np.where(np.isfinite(l64), np.abs(l64) + np.abs(top), 0)
    bound = mag * (3 * (np.minimum(span, 200) + 100) + 20) * 2.0 ** -24 + 2.0 ** -126
    k = KINDS[kind]
    bound += (np.abs(d) + bound) * mxref.HALF_STEP[k] + (2.0 ** -25 if k == 2 else 0)
    assert (np.abs(got - d) <= bound).all(), (what, np.max(np.abs(got - d) / bound))


@pytest.mark.parametrize("T,E,k,g,tg,gt", CASES)
@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("kind", KINDS)
def test_backward(T, E, k, g, tg, gt, score, kind):
    rng = np.random.default_rng(T * 1000 + E + k)
    l = logits(rng, T, E, kind)
    dw = rng.normal(size=(T, k)).astype(np.float32)
    for renormalize in (False, True):
        r = ref.Router(E, k, score, g, tg, gt, renormalize, 2.5)
        chosen, _, _ = ref.route(l.astype(np.float64), None, r)
        check_backward(l, kind, chosen, dw, r, f"gradient {T}x{E} top {k} {score} {kind} renorm {renormalize}", pad=T % 3, offset=E % 2)


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("renormalize", [False, True])
def test_backward_of_odd_choices(score, renormalize):
    """Entries outside the experts count nothing, an expert named twice counts twice, masked
    logits get zeros, and so does a token without a choice."""
    rng = np.random.default_rng(4)
    T, E, k = 40, 33, 4
    l = logits(rng, T, E, "f32")
    chosen = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    l[5, rng.permutation(E)[:20]] = -np.inf
    l[5, chosen[5]] = 0.25
    chosen[0] = -1
    chosen[1] = [4, -1, 2 ** 30, 7]
    chosen[2] = [-2 ** 31, E, E - 1, 0]
    chosen[3] = [6, 6, 9, 6]
    l[4] = 1e30
    l[6] = np.nan
    chosen[6] = -1
    dw = rng.normal(size=(T, k)).astype(np.float32)
    check_backward(l, "f32", chosen, dw, ref.Router(E, k, score, renormalize=renormalize), f"odd choices {score} {renormalize}")


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_against_differences(score, renormalize):
    """Differences of the weights that the library itself gives, a step of 2^-6: the third derivative
    (at most 1) leaves h^2 / 6 < 5e-5, the weights' roundings (less than 2^-17 each by
    weight_bound) 2^-17 / h = 2^-11 for each of the choices summed, whose dw are at most 1."""
    rng = np.random.default_rng(11)
    E, k, h = 12, 3, 2.0 ** -6
    base = rng.integers(-64, 64, E).astype(np.float32) / 32
    base[[2, 5, 8]] = [4.0, 3.5, 3.0]   # far enough ahead to stay chosen
    r = ref.Router(E, k, score, renormalize=renormalize)
    l = np.repeat(base[None], 2 * E, axis=0)
    for e in range(E):
        l[2 * e, e] += h
        l[2 * e + 1, e] -= h
    chosen, weights, _ = run_route(l, "f32", None, r)
    assert (np.sort(chosen, axis=1) == [2, 5, 8]).all()
    dw = rng.uniform(-1, 1, (1, k)).astype(np.float32)
    slope = ((weights[0::2] - weights[1::2]) * dw).sum(axis=1) / (2 * h)
    got = run_backward(base[None], "f32", chosen[:1], dw, r)[0]
    assert np.abs(got - slope).max() < k * (2.0 ** -11 + 5e-5)


# ---------------------------------------------------------------------------
# The layer on a given choice.

def operand(rng, rows, K):
    KP = mxref.padded(K)
    codes = rng.integers(0, 256, (rows, KP // 2), dtype=np.uint8)
    scales = rng.integers(122, 127, (rows, KP // 32)).astype(np.uint8)
    nib = np.arange(KP).reshape(-1, 2)
    codes &= (np.where(nib[:, 0] < K, 15, 0) | np.where(nib[:, 1] < K, 240, 0)).astype(np.uint8)
    t = torch()
    return codes, scales, t.from_numpy(codes).to("cuda:0"), t.from_numpy(scales).to("cuda:0")


def run_layer(T, H, I, E, k, chosen, weights, x, kind, w1, w2, workspace=True):
    t = torch()
    ws = t.empty(lib.gemm_mx_moe_workspace_bytes(T, I, k, KINDS[kind]), dtype=t.uint8, device="cuda:0") if workspace else None
    y = t.full((T * H + 8,), float(SENTINEL), device="cuda:0").to(dtype(kind))
    xd, ldx = padded(x, kind, 3)
    lib.gemm_mx_moe_routed(T, H, I, E, k, t.from_numpy(np.ascontiguousarray(chosen, np.int32)).to("cuda:0"), dev(weights), xd, KINDS[kind], ldx,
                           w1[2], w1[3], w2[2], w2[3], y, H, ws, ws.numel() if workspace else 0, stream())
    y = y.float().cpu().numpy()
    assert (y[T * H:] == SENTINEL).all()
    return y[:T * H].reshape(T, H)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 64, 4, 2), (5, 200, 100, 7, 3), (16, 256, 96, 8, 8), (33, 130, 40, 32, 5), (64, 300, 70, 16, 16)])
@pytest.mark.parametrize("kind", KINDS)
def test_layer_on_a_choice(T, H, I, E, k, kind):
    rng = np.random.default_rng(T + H + I)
    w1, w2 = operand(rng, E * 2 * I, H), operand(rng, E * H, I)
    x = mxref.to_type(rng.normal(size=(T, H)), KINDS[kind])
    chosen = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    weights = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    odd = rng.integers(0, 10, (T, k))
    chosen = np.where(odd == 0, -1, np.where(odd == 1, E + 3, chosen))
    if T > 4:
        chosen[0] = -1                     # no expert: zeros
        chosen[1, :] = chosen[1, 0] = 2    # one expert in every place
        chosen[2, :2] = 1                  # named twice
        chosen[3, 0], weights[3, 0] = -1, np.nan
    say(f"layer on a choice {T} tokens {k} of {E} {H}x{I} {kind}")
    y = run_layer(T, H, I, E, k, chosen, weights, x, kind, w1, w2, workspace=T != 5)
    dense = np.zeros((T, E))
    for t in range(T):
        if np.isnan(weights[t]).any():
            dense[t] = np.nan
            continue
        for e, w in zip(chosen[t], weights[t].astype(np.float64)):
            if 0 <= e < E:
                dense[t, e] += w
    want, bound = mxref.moe(x.astype(np.float64), dense, mxref.decode(w1[0], w1[1], H), mxref.decode(w2[0], w2[1], I), I,
                            {"f32": 3, "f16": 2, "bf16": 1}[kind], 3)
    # (the sum of an expert's up to 16 weights has as many roundings; they are inside the 16 + E of a weight)
    bound = bound + (np.abs(want) + bound) * mxref.HALF_STEP[KINDS[kind]]
    assert np.array_equal(np.isnan(y), np.isnan(want))
    fine = ~np.isnan(want)
    assert (np.abs(y - want)[fine] <= bound[fine]).all(), np.nanmax(np.abs(y - want) / np.maximum(bound, 1e-300))
    if T > 4:
        assert (y[0] == 0).all() and np.isnan(y[3]).all()


def test_layer_on_the_layers_own_choice():
    """The choice that gemm_route makes without a bias is gemm_mx_moe's: the same result within the weights'
    roundings (both layers' bound, twice)."""
    rng = np.random.default_rng(2)
    T, H, I, E, k = 12, 256, 128, 32, 4
    w1, w2 = operand(rng, E * 2 * I, H), operand(rng, E * H, I)
    x = rng.normal(size=(T, H)).astype(np.float32)
    l = rng.normal(size=(T, E)).astype(np.float32)
    chosen, weights, _ = run_route(l, "f32", None, ref.Router(E, k, renormalize=True))
    y = run_layer(T, H, I, E, k, chosen, weights, x, "f32", w1, w2)
    t = torch()
    z = t.empty(T, H, device="cuda:0")
    lib.gemm_mx_moe(T, H, I, E, k, True, dev(l), E, dev(x), 0, H, w1[2], w1[3], w2[2], w2[3], z, H, None, 0, stream())
    want, bound = mxref.moe(x.astype(np.float64), mxref.route(l, k, True), mxref.decode(w1[0], w1[1], H), mxref.decode(w2[0], w2[1], I), I, 3, 3)
    assert (np.abs(y - z.cpu().numpy()) <= 2 * bound).all()


LOWEST = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("E,g,tg,gt,k", [(8, 4, 2, 2, 4), (16, 4, 2, 2, 6), (16, 4, 3, 2, 9), (96, 8, 3, 2, 16), (300, 10, 2, 2, 5), (48, 16, 5, 1, 12)])
def test_bias_of_a_types_lowest_and_largest_values(E, g, tg, gt, k, score):
    """Finite biases whose sums of two pass float32: a group of such experts is worth what 64 bits say, and its
    experts fill up where the others do not suffice. Only a bias of -inf takes an expert out."""
    rng = np.random.default_rng(E + k)
    l = logits(rng, 24, E, "f32")
    l[0] = 0.25
    size = E // g
    masks = [np.where(np.arange(E) < size, 0.0, LOWEST),             # all groups but the first
             np.where(np.arange(E) < E - size, LOWEST, 0.0),         # all but the last
             np.full(E, LOWEST), np.full(E, -LOWEST),
             np.where(np.arange(E) // size % 2 == 1, -LOWEST, 0.0),  # sums past the largest value
             np.where(np.arange(E) % size == 0, 0.0, LOWEST),        # one expert left in each group
             np.where(np.arange(E) % size < 2, LOWEST, -np.inf)]
    masks += [rng.choice([0.0, LOWEST, -LOWEST, -2e38, 2e38, -1e38, -1e9, -np.inf, np.inf], E) for _ in range(12)]
    for n, b in enumerate(masks):
        check_route(l, "f32", b.astype(np.float32), ref.Router(E, k, score, g, tg, gt, True),
                    f"bias of lowest values {n}: {E} experts groups {g} {tg} {gt} top {k} {score}")


def logit_of(score, sign, off):
    """The float32 logit whose sigmoid lies nearest behind score + sign * off, on that side (float64), and how far."""
    at = score + sign * off
    l = np.float32(np.log(at / (1.0 - at)))
    for _ in range(8):
        far = sign * (1.0 / (1.0 + np.exp(-np.float64(l))) - score)
        if far >= off:
            return l, far
        l = np.nextafter(l, np.float32(sign * np.inf), dtype=np.float32)
    return l, -1.0


@pytest.mark.parametrize("largest", [16, 64, 1024])
@pytest.mark.parametrize("last", [False, True])
def test_groups_next_to_each_other_under_a_large_bias(largest, last):
    """Two groups of two experts under biases near a power of two, so that a value in float32 is a whole number of
    `unit`. One group's values lie next to half a unit and round down, and so does their sum; the other's
    round up: their float32 sums are 4 units apart, while in 64 bits the first is worth a little more."""
    rng = np.random.default_rng(largest)
    unit = largest * 2.0 ** -23
    many = 0
    for _ in range(30):
        score = rng.uniform(0.55, 0.9)                       # of the expert that gets most of its value from there
        whole = int(score / unit)
        one, two = rng.integers(0, 40, 2)
        add = np.array([0, one, whole // 2 + two, whole - whole // 2 + one - two])   # units above `largest`: both sums the same
        rows = []
        for _ in range(400):
            t = np.array([whole + rng.integers(-3, 4), *rng.integers(0, 4, 3)])
            m = add + t                                      # the units below each value
            if m[0] % 2 or not m[1] % 2 or (m[0] + m[1]) % 4 != 1 or m[0] + m[1] != m[2] + m[3]:
                continue
            small = [logit_of((t[n] + 0.5) * unit, -1 if n == 1 else 1, 2.0 ** -19 * (t[n] + 0.5) * unit) for n in (1, 2, 3)]
            lost = sum(far for _, far in small)
            l, far = logit_of((t[0] + 0.5) * unit, 1, 1.5 * lost + 2.0 ** -29)
            if min(far for _, far in small) > 0 and 0 < far < 2.0 ** -25:
                rows.append([l] + [v for v, _ in small])
        if not rows:
            continue
        many += len(rows)
        l = np.array(rows, np.float32)
        b = (largest + add * unit).astype(np.float32)
        if last:
            l, b = l[:, ::-1].copy(), b[::-1].copy()
        chosen = check_route(l, "f32", b, ref.Router(4, 2, ref.SIGMOID, 2, 1, 2, True), f"groups next to each other, biases near {largest} {last}")
        assert (chosen // 2 == int(last)).all()
    assert many > 20


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("mask", [-1e9, LOWEST, -np.inf, 1e9, -LOWEST, np.inf])
def test_masked_experts_beside_near_ties(mask, score):
    """How far estimates are trusted goes by the values that are compared: beside experts that a bias masks
    (or forces), values a few FP32 steps apart, and others far apart, are told apart as without them."""
    rng = np.random.default_rng(21)
    T, E = 40, 96
    near = (1.0 + rng.integers(0, 9, (T, E)) * 2.0 ** -22).astype(np.float32)
    far = logits(rng, T, E, "f32")
    b = (rng.integers(-3, 4, E) * 2.0 ** -23).astype(np.float32)
    for l in (near, far):
        for at in ([50], [3, 4, 60], list(range(12, 24)), list(range(12, 23)), list(range(0, 96, 2))):
            masked = b.copy()
            masked[at] = mask
            for g, tg, gt in ((1, 1, 1), (8, 3, 1), (8, 3, 2), (48, 20, 2)):
                check_route(l, "f32", masked, ref.Router(E, 7, score, g, tg, gt, True), f"masks {mask} at {len(at)} {score} groups {g} {tg} {gt}")


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("T,E,k,g,tg,gt,kind", [
    (4097, 64, 4, 1, 1, 1, "f32"), (20001, 24, 3, 4, 2, 2, "f32"), (5000, 128, 6, 8, 3, 2, "bf16"), (5000, 250, 8, 10, 4, 1, "f16"),
    (4500, 256, 8, 8, 4, 2, "bf16"), (4200, 512, 5, 16, 5, 2, "f32")])
def test_counts_of_many_tokens_by_values(T, E, k, g, tg, gt, kind, score):
    """A bias (and sums of two) over more tokens than a workgroup of 256 a CU takes, counted by several workgroups:
    every width of a lane's experts."""
    rng = np.random.default_rng(T + E)
    l = logits(rng, T, E, kind)
    check_route(l, kind, (0.1 * rng.normal(size=E)).astype(np.float32), ref.Router(E, k, score, g, tg, gt, True), f"counts of {T}x{E} by values {score}")
    if gt == 2:
        check_route(l, kind, None, ref.Router(E, k, score, g, tg, gt), f"counts of {T}x{E} by sums {score}")
