"""The operators whose rows choose their own matrices as a program runs them: together in a
decoding step, captured into graphs, on several streams at once, on
buffers past 32-bit offsets."""
import numpy as np
import pytest

import mx_reference as mxref
import rows_reference as ref
from fp32_gemm_07_amd import binding as lib
from gpu_util import say, torch
from test_lora_gpu import Case, half_step
from test_route_gpu import operand

pytestmark = pytest.mark.gpu

KINDS = {"f32": 0, "bf16": 1, "f16": 2}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    lib.load()
    torch()


def dtype(kind):
    t = torch()
    return {"f32": t.float32, "bf16": t.bfloat16, "f16": t.float16}[kind]


def dev(x, kind="f32"):
    return torch().from_numpy(np.ascontiguousarray(x, np.float32)).to("cuda:0").to(dtype(kind))


def ints(x):
    return torch().from_numpy(np.ascontiguousarray(x, np.int32)).to("cuda:0")


def host(x):
    return x.float().cpu().numpy()


def stream():
    return torch().cuda.current_stream().cuda_stream


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 24, 64])
def test_decoding_step(kind, T):
    """A block's shared projection with microscaled weights, each request's adapter on its result, the
    router's logits from the FP32 product, its choice, and the experts on it."""
    t = torch()
    rng = np.random.default_rng(T)
    H, N, I, E, k, R, A = 256, 320, 96, 32, 4, 12, 7
    x = mxref.to_type(rng.normal(size=(T, H)), KINDS[kind])
    w, w1, w2 = operand(rng, N, H), operand(rng, E * 2 * I, H), operand(rng, E * H, I)
    router = rng.normal(size=(H, E)).astype(np.float32) / 16
    bias = (0.05 * rng.normal(size=E)).astype(np.float32)
    a = mxref.to_type(rng.normal(size=(A, R, H)) / 16, KINDS[kind])
    b = mxref.to_type(rng.normal(size=(A, N, R)) / 4, KINDS[kind])
    ids = rng.integers(-1, A, T).astype(np.int32)
    scales = rng.uniform(0.5, 2, A).astype(np.float32)
    say(f"decoding step of {T} tokens {kind}")
    xd, s = dev(x, kind), stream()
    codes = t.empty(lib.gemm_mx_codes_bytes(T, H), dtype=t.uint8, device="cuda:0")
    cscales = t.empty(lib.gemm_mx_scales_bytes(T, H), dtype=t.uint8, device="cuda:0")
    y = t.empty(T, N, device="cuda:0").to(dtype(kind))
    lib.gemm_mx_quantize(False, T, H, xd, KINDS[kind], H, codes, cscales, s)
    lib.gemm_mx(T, N, H, 1.0, codes, cscales, w[2], w[3], 0.0, y, KINDS[kind], N, None, 0, s)
    shared = host(y).astype(np.float64)
    da, db, ds = dev(a, kind), dev(b, kind), dev(scales)
    adapters = lib.gemm_lora_t(KINDS[kind], N, H, R, A, da, db, None, ds)
    lib.gemm_lora(T, adapters, ints(ids), xd, H, y, N, y, N, None, 0, s)
    x32, rw = xd.float().contiguous(), dev(router)
    logits = t.empty(T, E, device="cuda:0")
    lib.gemm_f32(x32, rw, logits, T, E, H, s)
    r = ref.Router(E, k, ref.SIGMOID, 4, 2, 2, True, 1.5)
    rt = lib.gemm_route_t(E, k, r.score, r.groups, r.top_groups, r.group_top, r.renormalize, r.scale)
    chosen, weights = t.empty(T, k, dtype=t.int32, device="cuda:0"), t.empty(T, k, device="cuda:0")
    counts = t.empty(E, dtype=t.int32, device="cuda:0")
    lib.gemm_route(T, rt, logits, 0, E, dev(bias), chosen, weights, counts, s)
    out = t.empty(T, H, device="cuda:0").to(dtype(kind))
    lib.gemm_mx_moe_routed(T, H, I, E, k, chosen, weights, xd, KINDS[kind], H, w1[2], w1[3], w2[2], w2[3], out, H, None, 0, s)

    qc, qs = mxref.quantize(x)
    p, pmag = mxref.product(mxref.decode(qc, qs, H), mxref.decode(w[0], w[1], H))
    pb = pmag * (H + 8) * 2.0 ** -23
    assert (np.abs(shared - p) <= pb + half_step(kind, np.abs(p) + pb)).all()
    want, mag = ref.lora(x.astype(np.float64), shared, a.astype(np.float64), b.astype(np.float64), ids, None, scales)
    bound = mag * (H + 5 * R + 40) * 2.0 ** -23
    assert (np.abs(host(y) - want) <= bound + half_step(kind, np.abs(want) + bound)).all()
    l = host(logits)
    exact = x.astype(np.float64) @ router.astype(np.float64)
    assert (np.abs(l - exact) <= (np.abs(x).astype(np.float64) @ np.abs(router)) * (H + 8) * 2.0 ** -23).all()
    ec, ew, en = ref.route(l.astype(np.float64), bias.astype(np.float64), r)
    assert np.array_equal(chosen.cpu().numpy(), ec) and np.array_equal(counts.cpu().numpy(), en)
    gw = weights.cpu().numpy()
    assert (np.abs(gw - ew) <= np.abs(ew) * 120 * 2.0 ** -24).all()   # logits within 5 of each other: see weight_bound
    dense = np.zeros((T, E))
    np.put_along_axis(dense, ec, gw.astype(np.float64), axis=1)
    want, bound = mxref.moe(x.astype(np.float64), dense, mxref.decode(w1[0], w1[1], H), mxref.decode(w2[0], w2[1], I), I,
                            {"f32": 3, "f16": 2, "bf16": 1}[kind], 3)
    assert (np.abs(host(out) - want) <= bound + (np.abs(want) + bound) * mxref.HALF_STEP[KINDS[kind]]).all()


# ---------------------------------------------------------------------------
# Graphs.

def route_call(rng, T=700, E=64, k=4):
    t = torch()
    l, dw = dev(rng.normal(size=(T, E))), dev(rng.normal(size=(T, k)))
    b = dev(0.1 * rng.normal(size=E))
    c, w = t.empty(T, k, dtype=t.int32, device="cuda:0"), t.empty(T, k, device="cuda:0")
    n, dl = t.empty(E, dtype=t.int32, device="cuda:0"), t.empty(T, E, device="cuda:0")
    r = lib.gemm_route_t(E, k, lib.GEMM_ROUTE_SIGMOID, 8, 4, 2, True, 2.5)

    def call(s):
        lib.gemm_route(T, r, l, 0, E, b, c, w, n, s)
        lib.gemm_route_backward(T, r, l, 0, E, c, dw, dl, E, s)
    return call, [l, dw], [c, w, n, dl]


def lora_call(rng, rows=300, N=260, K=520, R=20, A=5, kind="bf16"):
    t = torch()
    x, c, dy = (dev(rng.normal(size=(rows, m)), kind) for m in (K, N, N))
    a, b = dev(rng.normal(size=(A, R, K)) / 16, kind), dev(rng.normal(size=(A, N, R)) / 4, kind)
    ids = ints(rng.integers(-1, A, rows))
    y, dx = t.empty_like(c), t.empty_like(x)
    da, db = t.empty(A, R, K, device="cuda:0"), t.empty(A, N, R, device="cuda:0")
    s_ = lib.gemm_lora_t(KINDS[kind], N, K, R, A, a, b)
    need = max(lib.gemm_lora_workspace_bytes(rows, s_), lib.gemm_lora_backward_workspace_bytes(rows, s_))
    ws = t.empty(need, dtype=t.uint8, device="cuda:0")

    def call(s):
        lib.gemm_lora(rows, s_, ids, x, K, c, N, y, N, ws, need, s)
        lib.gemm_lora_backward(rows, s_, ids, x, K, dy, N, None, K, dx, K, da, db, ws, need, s)
    call.keep = (a, b, ids)
    return call, [x, c, dy], [y, dx, da, db]


def experts_call(rng, T=30, H=256, I=96, E=16, k=4):
    t = torch()
    w1, w2 = operand(rng, E * 2 * I, H), operand(rng, E * H, I)
    x, weights = dev(rng.normal(size=(T, H)), "bf16"), dev(rng.uniform(0.1, 1, (T, k)))
    chosen = ints(np.stack([rng.permutation(E)[:k] for _ in range(T)]))
    y = t.empty(T, H, dtype=t.bfloat16, device="cuda:0")
    need = lib.gemm_mx_moe_workspace_bytes(T, I, k, 1)
    ws = t.empty(need, dtype=t.uint8, device="cuda:0")

    def call(s):
        lib.gemm_mx_moe_routed(T, H, I, E, k, chosen, weights, x, 1, H, w1[2], w1[3], w2[2], w2[3], y, H, ws, need, s)
    call.keep = (w1, w2, chosen)
    return call, [x, weights], [y]


CALLS = {"route": route_call, "lora": lora_call, "few_rows": lambda rng: lora_call(rng, rows=9), "experts": experts_call}


@pytest.mark.parametrize("what", CALLS)
def test_graph_replays_match_eager(what):
    t = torch()
    rng = np.random.default_rng(5)
    say(f"graph {what}")
    call, inputs, outputs = CALLS[what](rng)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        call(side.cuda_stream)
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        call(t.cuda.current_stream().cuda_stream)
    for turn in range(4):
        for x in inputs:
            x.copy_(x.roll(1 + turn, 0))
        call(stream())
        eager = [o.clone() for o in outputs]
        for o in outputs:
            o.fill_(-1)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        for o, e in zip(outputs, eager):
            assert t.equal(o, e), (what, turn)


def test_library_workspace_is_refused_while_capturing():
    t = torch()
    c = Case(np.random.default_rng(1), 70, 64, 64, 8, 2, "f32", True)   # (a few rows need no workspace)
    s_ = c.set()
    x, y = dev(c.x), t.empty(70, 64, device="cuda:0")
    da, db = t.empty(c.a.size, device="cuda:0"), t.empty(c.b.size, device="cuda:0")
    t.cuda.synchronize()
    for call in (lambda s: lib.gemm_lora(70, s_, c.di, x, 64, None, 64, y, 64, None, 0, s),
                 lambda s: lib.gemm_lora_backward(70, s_, c.di, x, 64, x, 64, None, 64, y, 64, da, db, None, 0, s)):
        with pytest.raises(lib.GemmError) as e:
            graph = t.cuda.CUDAGraph()
            with t.cuda.graph(graph):
                call(t.cuda.current_stream().cuda_stream)
        assert e.value.status == lib.GEMM_ERR_CAPTURING
        t.cuda.synchronize()


def test_streams_at_once():
    """Calls on three streams at the same time, with the library's workspaces: each as if alone."""
    t = torch()
    rng = np.random.default_rng(8)
    cases = []
    for n in range(3):
        rows, N, K, R, A, kind = (400, 300, 500, 16, 3, "bf16") if n < 2 else (31, 700, 1030, 30, 6, "f32")
        c = Case(rng, rows, N, K, R, A, kind, n == 1)
        c.a, c.b = np.nan_to_num(c.a), np.nan_to_num(c.b)
        s_ = c.set()
        x, cc, dy = dev(c.x, kind), dev(c.c, kind), dev(c.dy, kind)
        out = [t.empty_like(cc), t.empty_like(x), t.empty(c.a.size, device="cuda:0"), t.empty(c.b.size, device="cuda:0")]

        def call(s, c=c, s_=s_, x=x, cc=cc, dy=dy, out=out):
            lib.gemm_lora(c.rows, s_, c.di, x, c.k, cc, c.n, out[0], c.n, None, 0, s)
            lib.gemm_lora_backward(c.rows, s_, c.di, x, c.k, dy, c.n, None, c.k, out[1], c.k, out[2], out[3], None, 0, s)
        call(stream())
        t.cuda.synchronize()
        cases.append((call, out, [o.clone() for o in out]))
    streams = [t.cuda.Stream() for _ in cases]
    t.cuda.synchronize()
    for _ in range(10):
        for (call, _, _), s in zip(cases, streams):
            call(s.cuda_stream)
    t.cuda.synchronize()
    for _, out, alone in cases:
        for o, a in zip(out, alone):
            assert t.equal(o, a)


# ---------------------------------------------------------------------------
# Offsets past 32 bits.

def test_adapters_past_32_bits():
    """70 adapters of 128 x 262144 bfloat16: the last lies 2.3e9 elements from the first."""
    t = torch()
    rng = np.random.default_rng(3)
    rows, N, K, R, A = 7, 16, 1 << 18, 128, 70
    say("adapters past 32 bits")
    a = t.empty(A, R, K, dtype=t.bfloat16, device="cuda:0")
    b = t.empty(A, N, R, dtype=t.bfloat16, device="cuda:0")
    x = mxref.to_type(rng.normal(size=(rows, K)), 1)
    wa, wb = mxref.to_type(rng.normal(size=(R, K)) / 512, 1), mxref.to_type(rng.normal(size=(N, R)) / 8, 1)
    a[69].copy_(dev(wa, "bf16"))
    b[69].copy_(dev(wb, "bf16"))
    s_ = lib.gemm_lora_t(1, N, K, R, A, a, b)
    y = t.empty(rows, N, dtype=t.bfloat16, device="cuda:0")
    ids = ints(np.full(rows, 69))
    lib.gemm_lora(rows, s_, ids, dev(x, "bf16"), K, None, N, y, N, None, 0, stream())
    want, mag = ref.lora(x.astype(np.float64), None, wa[None].astype(np.float64), wb[None].astype(np.float64), np.zeros(rows, int), None, None)
    # (K terms in ranges of at most 4096 a lane group: the bound counts the longest chain)
    bound = mag * (K // 8 + 5 * R + 40) * 2.0 ** -23
    assert (np.abs(host(y) - want) <= bound + half_step("bf16", np.abs(want) + bound)).all()


def test_rows_past_32_bits():
    """Row strides of 2^30 elements: the third row begins past 2^31."""
    t = torch()
    rng = np.random.default_rng(4)
    ld, T, E = (1 << 30) + 8, 3, 40
    say("rows past 32 bits")
    buf = t.empty(2 * ld + 64, dtype=t.bfloat16, device="cuda:0")
    l = mxref.to_type(rng.normal(size=(T, E)), 1)
    for i in range(T):
        buf[i * ld:i * ld + E].copy_(dev(l[i], "bf16"))
    r = lib.gemm_route_t(E, 3, 0, 1, 1, 1, True, 1.0)
    c, w = t.empty(T, 3, dtype=t.int32, device="cuda:0"), t.empty(T, 3, device="cuda:0")
    lib.gemm_route(T, r, buf, 1, ld, None, c, w, None, stream())
    chosen, _, _ = ref.route(l.astype(np.float64), None, ref.Router(E, 3, renormalize=True))
    assert np.array_equal(c.cpu().numpy(), chosen)
    a, b = mxref.to_type(rng.normal(size=(1, 4, E)), 1), mxref.to_type(rng.normal(size=(1, 24, 4)), 1)
    da, db = dev(a, "bf16"), dev(b, "bf16")
    s_ = lib.gemm_lora_t(1, 24, E, 4, 1, da, db)
    out = t.empty(2 * ld + 64, dtype=t.bfloat16, device="cuda:0")
    lib.gemm_lora(T, s_, ints([0, 0, 0]), buf, ld, None, 24, out, ld, None, 0, stream())
    want, mag = ref.lora(l.astype(np.float64), None, a.astype(np.float64), b.astype(np.float64), np.zeros(T, int), None, None)
    for i in range(T):
        got = host(out[i * ld:i * ld + 24])
        bound = mag[i] * 100 * 2.0 ** -23
        assert (np.abs(got - want[i]) <= bound + half_step("bf16", np.abs(want[i]) + bound)).all()
