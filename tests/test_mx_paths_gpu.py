"""The gemm_mx* entry points on the GPU: what tests/test_mx_gpu.py leaves open, against
the same reference (tests/mx_reference.py) and by the same rules."""
import numpy as np
import pytest

import mx_reference as ref
from fp32_gemm_07_amd import binding as lib
from gpu_util import say, torch
from mx_plans import IDS, PLANS, is_plan
from test_mx_gpu import KINDS, bytes_dev, check_layer, dtype, layer_case, operand, run_layer, stream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    lib.load()
    torch()


def packed(values, scales):
    """e2m1 values rows x KP (a multiple of 128) and scale bytes rows x KP / 32 -> an
    operand: (codes, scales) NumPy and on the device."""
    code = np.searchsorted(ref.E2M1, np.abs(values)).astype(np.uint8) | (np.signbit(values).astype(np.uint8) << 3)
    assert (ref.E2M1[code & 7] == np.abs(values)).all()
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    scales = np.ascontiguousarray(scales, np.uint8)
    return codes, scales, bytes_dev(codes), bytes_dev(scales)


# ---------------------------------------------------------------------------
# The layer's hidden activations.

def wide_layer(rng, T, H, I, kind):
    """One expert whose hidden activations need 24 bits, and outputs in which the high
    ones cancel. Gates are 32 for every token, so that silu(gate) is 32 (1 + exp(-32)
    is 1 in FP32, 32 (1 - 1.3e-14) in real numbers); ups are 2^17 + b with b a sum of
    a few half numbers, |b| < 60; a row of D holds +d and -d in two columns, so
    y = 32 d (b_i - b_j). Every product and partial sum is a multiple of 2^3
    (b and d are multiples of 2^-1) and below 2^27, hence exact in FP32 in any order."""
    HP, IP = ref.padded(H), ref.padded(I)
    x = np.zeros((T, H))
    x[:, 0] = 1.0
    at = rng.choice(np.arange(32, H), 5, replace=False)
    x[:, at] = rng.integers(-2, 3, (T, 5))
    w1 = np.zeros((2 * I, HP))
    w1[:I, 0] = 1.0                                              # gates: 1 under 2^5
    w1[I:, 0] = 1.0                                              # ups: 1 under 2^17
    w1[I:, at] = rng.choice([0.5, -1.0, 1.5, -3.0, 4.0, 6.0], (I, 5))
    s1 = np.full((2 * I, HP // 32), 127)
    s1[:I, 0], s1[I:, 0] = 127 + 5, 127 + 17
    w2 = np.zeros((H, IP))
    for h in range(H):
        i, j = rng.choice(I, 2, replace=False)
        w2[h, i] = rng.choice([0.5, 1.0, 3.0])
        w2[h, j] = -w2[h, i]
    s2 = np.full((H, IP // 32), 127)
    b = x[:, at] @ w1[I:, at].T
    want = 32.0 * (b @ w2[:, :I].T)
    assert np.abs(b).max() < 60 and want.any()
    return x, packed(w1, s1), packed(w2, s2), want


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 6, 31])   # one group of 4; a partial group of 8; four groups of 8
@pytest.mark.parametrize("H,I", [(160, 40), (300, 300), (96, 1000)])
def test_layer_hidden_activations_keep_24_bits(kind, T, H, I):
    say(f"layer hidden activations {kind} tokens {T} hidden {H} inter {I}")
    x, w1, w2, want = wide_layer(np.random.default_rng(T + H + I), T, H, I, kind)
    got = run_layer(x, np.zeros((T, 1), np.float32), w1, w2, I, 1, True, kind)
    np.testing.assert_array_equal(got, ref.to_type(want, ref.TYPES[kind]))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [3, 20])
def test_layer_infinite_hidden_activations(kind, T):
    """A hidden activation past the largest float is an infinity: outputs whose weight
    of it is a zero are NaN, the others infinite with the weight's sign, other tokens
    untouched."""
    say(f"layer infinite hidden activations {kind} tokens {T}")
    rng = np.random.default_rng(T)
    H, I = 140, 200
    x, w1, w2, want = wide_layer(rng, T, H, I, kind)
    hot, col = T // 2, 77
    x[:, H - 1] = 0.0
    x[hot, H - 1] = 1.0
    last = (H - 1) // 32
    codes, scales = w1[0].copy(), w1[1].copy()
    for row in (col, I + col):   # gate and up of one column: 2^100 more for one token
        scales[row, last] = 127 + 100
        codes[row, 16 * last:16 * last + 16] = 0
        codes[row, (H - 1) // 2] = 2 << (4 * ((H - 1) % 2))
    w1 = (codes, scales, bytes_dev(codes), bytes_dev(scales))
    d = np.zeros((H, ref.padded(I)))
    d[:, col] = rng.choice([0.0, -0.0, 0.5, -6.0, 2.0], H)
    codes = w2[0].copy()
    full = ref.decode(w2[0], np.full(w2[1].shape, 127, np.uint8), ref.padded(I))
    full[:, col] = d[:, col]
    w2 = packed(full, w2[1])
    got = run_layer(x, np.zeros((T, 1), np.float32), w1, w2, I, 1, True, kind)
    g, v = x @ ref.decode(w1[0], w1[1], H)[:I].T, x @ ref.decode(w1[0], w1[1], H)[I:].T
    with np.errstate(over="ignore", invalid="ignore"):
        a = (g / (1 + np.exp(-g)) * v).astype(np.float32).astype(np.float64)
        want = a @ full[:, :I].T
    assert np.isinf(a[hot, col]) and np.isfinite(np.delete(a, hot, 0)).all()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(got[hot][np.isinf(want[hot])], want[hot][np.isinf(want[hot])])
    rest = np.arange(T) != hot
    assert np.isfinite(got[rest]).all() if kind != "f16" else not np.isnan(got[rest]).any()


# ---------------------------------------------------------------------------
# More workgroups than one launch takes (2^32 threads).

@pytest.fixture
def room():
    """The card's memory without what earlier tests left in torch's pool, and given back."""
    t = torch()
    t.cuda.empty_cache()
    yield
    t.cuda.synchronize()
    t.cuda.empty_cache()


@pytest.mark.parametrize("trans", [False, True], ids=["rows", "columns"])
def test_conversion_of_more_rows_than_a_launch_takes(trans, room):
    """2^30 + 130 rows of one value (64 rows of it are a workgroup, 128 down columns):
    1 to 7 by row, which stand for 1, 2, 3, 4, 4 (a tie, to the even code), 6 and 6."""
    t = torch()
    rows = (1 << 30) + 130
    say(f"conversion of {rows} rows, trans {trans}")
    x = (t.arange(rows, dtype=t.int32, device="cuda:0") % 7 + 1).to(t.bfloat16)
    c = t.full((lib.gemm_mx_codes_bytes(rows, 1),), 0xA5, dtype=t.uint8, device="cuda:0")
    s = t.full((lib.gemm_mx_scales_bytes(rows, 1),), 0xA5, dtype=t.uint8, device="cuda:0")
    ld = rows if trans else 1
    lib.gemm_mx_quantize(trans, rows, 1, x, ref.BF16, ld, c, s, stream())
    codes, scales = ref.quantize(np.arange(1.0, 8.0)[:, None])
    for first in (0, (1 << 29) - 70, (1 << 30) - 150, rows - 140):   # whole periods of 7 rows
        first -= first % 7
        n = min(140, rows - first)
        got_c = c.view(rows, 64)[first:first + n].cpu().numpy()
        got_s = s.view(rows, 4)[first:first + n].cpu().numpy()
        np.testing.assert_array_equal(got_c, codes[np.arange(n) % 7])
        np.testing.assert_array_equal(got_s, scales[np.arange(n) % 7])
    y = t.full((rows,), float("nan"), dtype=t.bfloat16, device="cuda:0")
    lib.gemm_mx_dequantize(trans, rows, 1, c, s, y, ref.BF16, ld, stream())
    del c, s
    stands_for = t.tensor([1, 2, 3, 4, 4, 6, 6], dtype=t.bfloat16, device="cuda:0")
    step = 7 << 24
    for first in range(0, rows, step):
        n = min(step, rows - first)
        want = stands_for.repeat(-(-n // 7))[:n]
        assert t.equal(y[first:first + n], want), first


def test_product_of_more_tiles_than_a_launch_takes(room):
    """2^31 - 1 rows of A by one of B: 2^24 tiles of 128 x 128, one more than a launch
    of 256 threads each takes. Every row's value has its own code."""
    t = torch()
    M = (1 << 31) - 1
    say(f"product {M}x1x1")
    c = t.zeros((M, 64), dtype=t.uint8, device="cuda:0")
    s = t.full((M, 4), 127, dtype=t.uint8, device="cuda:0")
    step = 1 << 27
    for first in range(0, M, step):
        n = min(step, M - first)
        c[first:first + n, 0] = (t.arange(first, first + n, dtype=t.int64, device="cuda:0") % 16).to(t.uint8)
    b = packed(np.full((1, 128), 1.0) * (np.arange(128) == 0), np.full((1, 4), 128))
    out = t.full((M,), float("nan"), dtype=t.bfloat16, device="cuda:0")
    lib.gemm_mx(M, 1, 1, 1.0, c, s, b[2], b[3], 0.0, out, ref.BF16, 1, None, 0, stream())
    table = t.tensor(np.concatenate((2 * ref.E2M1, -2 * ref.E2M1)), dtype=t.bfloat16, device="cuda:0")
    for first in range(0, M, step):
        n = min(step, M - first)
        assert t.equal(out[first:first + n], table.repeat(n // 16 + 1)[:n]), first


def test_product_of_more_columns_than_a_launch_takes(room):
    """The same with the operands exchanged: the columns of C in two launches."""
    t = torch()
    N = (1 << 31) - 1
    say(f"product 3x{N}x1")
    c = t.zeros((N, 64), dtype=t.uint8, device="cuda:0")
    s = t.full((N, 4), 127, dtype=t.uint8, device="cuda:0")
    c[:, 0] = 2                      # 1.0, and the last tile 6.0
    c[N - 100:, 0] = 7
    a = packed(np.array([[1.0], [-2.0], [0.5]]) * (np.arange(128) == 0), np.full((3, 4), 127))
    out = t.full((3, N), float("nan"), dtype=t.bfloat16, device="cuda:0")
    lib.gemm_mx(3, N, 1, 1.0, a[2], a[3], c, s, 0.0, out, ref.BF16, N, None, 0, stream())
    for row, v in enumerate((1.0, -2.0, 0.5)):
        assert (out[row, :N - 100] == v).all().item() and (out[row, N - 100:] == 6 * v).all().item()


# ---------------------------------------------------------------------------
# The product through every kernel it chooses between.

def decode_on_device(codes, scales, K):
    """An operand as float64 on the device (exact)."""
    t = torch()
    table = t.tensor(np.concatenate((ref.E2M1, -ref.E2M1)), dtype=t.float64, device="cuda:0")
    v = t.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), dim=-1).view(*scales.shape, 32)
    powers = t.tensor([2.0 ** (n - 127) for n in range(255)] + [float("nan")], dtype=t.float64, device="cuda:0")
    v *= powers[scales.long()][..., None]
    return v.view(codes.shape[0], -1)[:, :K].contiguous()


@pytest.mark.parametrize("M,N,K,tile,split", PLANS, ids=IDS)
def test_product_through_every_kernel(M, N, K, tile, split):
    """Bit for bit in every type, with alpha, beta and row strides, aligned and not. Scales
    within a factor of 4 of each other: products are multiples of 2^-4, with a root mean
    square of 15 under random signs, so that sums stay below 100 sqrt(K) 15 < 2^20 and FP32
    sums of them are exact in any order; so are the powers of two alpha and beta with
    whole numbers in C, and one rounding to the type is left."""
    t = torch()
    plan = lib.gemm_mx_plan(M, N, K)
    say(f"product {M}x{N}x{K}: {plan}")
    assert is_plan(plan, tile, split), "other sizes are needed to reach this kernel"
    rng = np.random.default_rng(M + N + K)
    a, b = operand(rng, M, K, 126, 128), operand(rng, N, K, 126, 128)
    s = decode_on_device(a[2], a[3], K) @ decode_on_device(b[2], b[3], K).t().contiguous()
    assert s.abs().max().item() < 2 ** 20
    need = lib.gemm_mx_workspace_bytes(M, N, K)
    ws = t.full((max(need, 16),), 0xff, dtype=t.uint8, device="cuda:0")
    c0 = t.randint(-99, 100, (M, N), device="cuda:0")
    for kind in KINDS:
        # alpha small enough for half's range; strides of 16 bytes, and odd ones one element off
        for alpha, beta, ldc, off in ((0.125, 0.0, N + -N % 8, 0), (-0.25, 0.5, N + -N % 8 + 8, 0),
                                      (0.0625, -2.0, N + 1 + N % 2, 1)):
            C = t.full((off + M * ldc + 8,), 7.0, dtype=dtype(kind), device="cuda:0")
            view = C[off:off + M * ldc].view(M, ldc)
            view[:, :N] = c0.to(dtype(kind)) if beta else float("nan")
            lib.gemm_mx(M, N, K, alpha, a[2], a[3], b[2], b[3], beta, C[off:], ref.TYPES[kind], ldc, ws, need, stream())
            want = (alpha * s + beta * c0).float().to(dtype(kind))
            assert t.equal(view[:, :N], want), (kind, alpha, (view[:, :N] != want).sum().item())
            assert (view[:, N:] == 7).all().item() and (C[off + M * ldc:] == 7).all().item() and (C[:off] == 7).all().item()
    # a NaN block in the last stretch of a row of A and in the first of B's last row
    a[3][M // 2, -(-K // 32) - 1] = 255
    b[3][N - 1, 0] = 255
    out = t.zeros((M, N), device="cuda:0")
    lib.gemm_mx(M, N, K, 1.0, a[2], a[3], b[2], b[3], 0.0, out, ref.F32, N, ws, need, stream())
    want = s.float()
    want[M // 2], want[:, N - 1] = float("nan"), float("nan")
    assert t.equal(t.isnan(out), t.isnan(want)) and t.equal(out.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("M,N,K,tile,split", [PLANS[n] for n in (1, 6, 10, 16, 21, 24, 27)],
                         ids=[IDS[n] for n in (1, 6, 10, 16, 21, 24, 27)])
def test_product_kernels_captured_and_on_streams(M, N, K, tile, split):
    """Replays of a captured call with operands changed between them, and calls on three
    streams at once with the library's workspace, all against the exact product."""
    t = torch()
    say(f"product {M}x{N}x{K} captured and on streams")
    assert is_plan(lib.gemm_mx_plan(M, N, K), tile, split)
    rng = np.random.default_rng(M * N + K)
    a, bs = operand(rng, M, K, 126, 128), [operand(rng, N, K, 126, 128) for _ in range(2)]
    av = decode_on_device(a[2], a[3], K)
    want = [(av @ decode_on_device(b[2], b[3], K).t().contiguous()).float() for b in bs]
    del av
    need = lib.gemm_mx_workspace_bytes(M, N, K)
    ws = t.empty(max(need, 16), dtype=t.uint8, device="cuda:0")
    bc, bsc, out = bs[0][2].clone(), bs[0][3].clone(), t.zeros((M, N), device="cuda:0")
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        lib.gemm_mx(M, N, K, 1.0, a[2], a[3], bc, bsc, 0.0, out, ref.F32, N, ws, need, stream())
    for n in range(4):
        bc.copy_(bs[n % 2][2])
        bsc.copy_(bs[n % 2][3])
        out.fill_(float("nan"))
        g.replay()
        t.cuda.synchronize()
        assert t.equal(out, want[n % 2]), n
    streams = [t.cuda.Stream() for _ in range(3)]
    outs = [t.full((M, N), float("nan"), device="cuda:0") for _ in range(6)]
    t.cuda.synchronize()
    for i, o in enumerate(outs):
        b = bs[i % 2]
        lib.gemm_mx(M, N, K, 1.0, a[2], a[3], b[2], b[3], 0.0, o, ref.F32, N, None, 0, streams[i % 3].cuda_stream)
    t.cuda.synchronize()
    for i, o in enumerate(outs):
        assert t.equal(o, want[i % 2]), i


# ---------------------------------------------------------------------------
# More of the layer.

@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "plain"])
@pytest.mark.parametrize("kind,T,H,I,E,k", [
    # groups of 8 tokens whose activations fill several batches of K in LDS
    ("bf16", 40, 5120, 48, 8, 2), ("bf16", 64, 7000, 20, 6, 3), ("bf16", 25, 4225, 130, 4, 1),
    # the same sizes where more parts leave room for groups of 4 only
    ("f16", 40, 5120, 48, 8, 2), ("f32", 40, 5120, 48, 8, 2),
    # groups of 8 in one batch, every type
    ("f16", 30, 1700, 70, 5, 2), ("f32", 30, 1100, 70, 5, 2)])
def test_layer_with_many_tokens_an_expert(kind, T, H, I, E, k, renorm):
    say(f"layer {kind} tokens {T} hidden {H} inter {I} experts {E} top {k} renorm {renorm}")
    x, logits, w1, w2 = layer_case(T + H + E, T, H, I, E, kind)
    check_layer(run_layer(x, logits, w1, w2, I, k, renorm, kind), x, logits, w1, w2, I, k, renorm, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [4, 30])
def test_layer_inputs_near_the_largest_value(kind, T):
    """Inputs near the type's largest value, both signs, under weights that bring the gates
    back to ordinary size: what the split into parts leaves of them is in the bound."""
    say(f"layer large inputs {kind}, {T} tokens")
    H, I, E, k = 260, 64, 4, 2
    x, logits, w1, w2 = layer_case(T, T, H, I, E, kind)
    top = torch().finfo(dtype(kind)).max
    rng = np.random.default_rng(T)
    big = rng.random(x.shape) < 0.3
    x[big] = ref.to_type(top * rng.choice([-1.0, -0.75, 0.5, 1.0], big.sum()), ref.TYPES[kind])
    assert np.isfinite(x).all() and np.abs(x).max() == top
    w1 = operand(rng, E * 2 * I, H, *((103, 106) if kind == "f16" else (0, 2)))   # from 2^-24 or 2^-127 on
    got = run_layer(x, logits, w1, w2, I, k, True, kind)
    want, _ = check_layer(got, x, logits, w1, w2, I, k, True, kind)
    assert np.isfinite(want).all() and (np.abs(want) > 0).all()
