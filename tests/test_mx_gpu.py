"""The gemm_mx* entry points on the GPU against tests/mx_reference.py (NumPy,
float64): conversion bit for bit, products and the mixture-of-experts layer
within bounds derived beside them, and bit for bit where every sum is exact.

Outputs lie inside larger buffers filled with a sentinel that has to survive,
inputs inside NaN-filled ones."""
import numpy as np
import pytest

import mx_reference as ref
from fp32_gemm_07_amd import binding as lib
from gpu_util import say, torch

pytestmark = pytest.mark.gpu

KINDS = ["f32", "bf16", "f16"]
GUARD = 0xA5


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
    """float32 array (already rounded to `kind`) -> a device tensor of that type."""
    return torch().from_numpy(np.ascontiguousarray(x, np.float32)).to("cuda:0").to(dtype(kind))


def bytes_dev(x):
    return torch().from_numpy(np.ascontiguousarray(x, np.uint8)).to("cuda:0")


def host(t):
    return t.float().cpu().numpy()


def matrix(x, kind, pad, offset=0):
    """Stored matrix with rows padded by `pad` NaN elements, `offset` elements into
    its buffer. Returns (view to pass, ld)."""
    rows, cols = x.shape
    ld = cols + pad
    buf = np.full(offset + rows * ld, np.nan, np.float32)
    buf[offset:].reshape(rows, ld)[:, :cols] = x
    return dev(buf, kind)[offset:], ld


def operand_buffers(rows, K, extra=64):
    t = torch()
    c = t.full((lib.gemm_mx_codes_bytes(rows, K) + extra,), GUARD, dtype=t.uint8, device="cuda:0")
    s = t.full((lib.gemm_mx_scales_bytes(rows, K) + extra,), GUARD, dtype=t.uint8, device="cuda:0")
    return c, s


def operand(rng, rows, K, low=120, high=130):
    """Random codes under scales 2^(low - 127 .. high - 127), the padding zero:
    (codes, scales) NumPy and on the device."""
    KP = ref.padded(K)
    codes = rng.integers(0, 256, (rows, KP // 2), dtype=np.uint8)
    scales = rng.integers(low, high + 1, (rows, KP // 32)).astype(np.uint8)
    nib = np.arange(KP).reshape(-1, 2)
    codes &= (np.where(nib[:, 0] < K, 15, 0) | np.where(nib[:, 1] < K, 240, 0)).astype(np.uint8)
    return codes, scales, bytes_dev(codes), bytes_dev(scales)


# ---------------------------------------------------------------------------
# Conversion.

SIZES = [(1, 1), (1, 32), (3, 33), (5, 127), (64, 128), (65, 129), (17, 255), (130, 257), (63, 2049), (4, 4100), (300, 511)]


def values(rng, rows, K, kind):
    x = rng.standard_normal((rows, K)) * np.exp(2 * rng.standard_normal((1, K)))
    x[rng.random((rows, K)) < 0.05] = 0.0
    # values on and next to the borders of e2m1
    pick = rng.random((rows, K)) < 0.2
    x[pick] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, -0.25, -5.0, -0.0], pick.sum())
    return ref.to_type(x, ref.TYPES[kind])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("trans", [False, True], ids=["rows", "columns"])
@pytest.mark.parametrize("rows,K", SIZES, ids=[f"{r}x{k}" for r, k in SIZES])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1), (8, 0)], ids=["dense", "odd", "even"])
def test_quantize(kind, trans, rows, K, pad, offset):
    say(f"quantize {kind} trans {trans} {rows}x{K} pad {pad} offset {offset}")
    rng = np.random.default_rng(rows * 7919 + K + pad)
    x = values(rng, rows, K, kind)
    X, ld = matrix(x.T if trans else x, kind, pad, offset)
    c, s = operand_buffers(rows, K)
    lib.gemm_mx_quantize(trans, rows, K, X, ref.TYPES[kind], ld, c, s, stream())
    codes, scales = ref.quantize(x)
    got_c, got_s = c.cpu().numpy(), s.cpu().numpy()
    assert (got_c[codes.size:] == GUARD).all() and (got_s[scales.size:] == GUARD).all()
    np.testing.assert_array_equal(got_s[:scales.size].reshape(scales.shape), scales)
    np.testing.assert_array_equal(got_c[:codes.size].reshape(codes.shape), codes)


@pytest.mark.parametrize("trans", [False, True], ids=["rows", "columns"])
def test_quantize_special_values(trans):
    """Infinities and NaN (their block NaN, the neighbours untouched), subnormals,
    the largest and smallest values, powers of two and their neighbours."""
    say(f"quantize specials trans {trans}")
    f = np.float32
    rng = np.random.default_rng(5)
    x = rng.standard_normal((12, 256)).astype(f)
    x[0, 5], x[0, 40], x[0, 70], x[0, 255] = np.inf, -np.inf, np.nan, -np.nan
    x[1] = 0.0
    x[2] = -0.0
    x[3] = np.ldexp(f(1), rng.integers(-149, -120, 256))
    x[4] = np.finfo(f).max
    x[5] = -np.finfo(f).tiny
    x[6] = np.ldexp(f(1), rng.integers(-126, 127, 256))
    x[7] = np.nextafter(np.ldexp(f(1), rng.integers(-120, 120, 256)), f(0))
    x[8] = np.nextafter(np.ldexp(f(1), rng.integers(-120, 120, 256)), f(np.inf))
    x[9] = f(2.0 ** -149)
    x[10] = x[0][::-1]
    x[11] = rng.standard_normal(256) * f(2.0 ** -127)
    X, ld = matrix(x.T if trans else x, "f32", 0)
    c, s = operand_buffers(12, 256)
    lib.gemm_mx_quantize(trans, 12, 256, X, ref.F32, ld, c, s, stream())
    codes, scales = ref.quantize(x)
    np.testing.assert_array_equal(s.cpu().numpy()[:scales.size].reshape(scales.shape), scales)
    np.testing.assert_array_equal(c.cpu().numpy()[:codes.size].reshape(codes.shape), codes)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("trans", [False, True], ids=["rows", "columns"])
@pytest.mark.parametrize("rows,K,pad,offset", [(1, 1, 0, 0), (257, 256, 0, 0), (65, 129, 3, 1), (33, 300, 8, 0), (4, 4100, 0, 0), (130, 511, 1, 0)])
def test_dequantize(kind, trans, rows, K, pad, offset):
    """Every scale byte and code (257 x 256 has them all in its first rows)."""
    say(f"dequantize {kind} trans {trans} {rows}x{K} pad {pad}")
    t = torch()
    rng = np.random.default_rng(rows + K)
    codes, scales, c, s = operand(rng, rows, K, 0, 255)
    if rows == 257:
        scales[:256] = np.arange(256, dtype=np.uint8)[:, None]
        codes[:256] = np.arange(codes.shape[1], dtype=np.uint8)[None, :]
        c, s = bytes_dev(codes), bytes_dev(scales)
    want = ref.decode(codes, scales, K)
    with np.errstate(over="ignore"):
        want = ref.to_type(want.astype(np.float32), ref.TYPES[kind])
    shape = (K, rows) if trans else (rows, K)
    ld = shape[1] + pad
    y = t.full((offset + shape[0] * ld + 16,), 7.0, dtype=dtype(kind), device="cuda:0")
    lib.gemm_mx_dequantize(trans, rows, K, c, s, y[offset:], ref.TYPES[kind], ld, stream())
    flat = host(y)
    assert (flat[:offset] == 7).all() and (flat[offset + shape[0] * ld:] == 7).all()
    got = flat[offset:offset + shape[0] * ld].reshape(shape[0], ld)
    assert (got[:, shape[1]:] == 7).all()
    got = got[:, :shape[1]]
    np.testing.assert_array_equal(got.T if trans else got, want)


def test_conversion_past_32_bits():
    """An operand whose codes pass 2^32 bytes: the last rows are quantised and read
    back where they belong (the first and last rows of 2^20 + 3 by 8192)."""
    t = torch()
    rows, K = (1 << 20) + 3, 8192
    say(f"quantize {rows}x{K} bf16: {lib.gemm_mx_codes_bytes(rows, K) >> 20} MiB of codes")
    x = t.zeros((rows, K), dtype=t.bfloat16, device="cuda:0")
    g = t.Generator(device="cuda:0")
    g.manual_seed(3)
    for part in (slice(0, 64), slice(rows - 64, rows)):
        x[part] = t.randn((64, K), generator=g, device="cuda:0").to(t.bfloat16)
    c = t.empty(lib.gemm_mx_codes_bytes(rows, K), dtype=t.uint8, device="cuda:0")
    s = t.empty(lib.gemm_mx_scales_bytes(rows, K), dtype=t.uint8, device="cuda:0")
    lib.gemm_mx_quantize(False, rows, K, x, ref.BF16, K, c, s, stream())
    y = t.empty_like(x)
    lib.gemm_mx_dequantize(False, rows, K, c, s, y, ref.BF16, K, stream())
    for part in (slice(0, 64), slice(rows - 64, rows)):
        codes, scales = ref.quantize(host(x[part]))
        np.testing.assert_array_equal(c.view(rows, -1)[part].cpu().numpy(), codes)
        np.testing.assert_array_equal(s.view(rows, -1)[part].cpu().numpy(), scales)
        np.testing.assert_array_equal(host(y[part]), ref.decode(codes, scales, K))
    assert not t.any(y[64:rows - 64].view(t.int16)).item()


# ---------------------------------------------------------------------------
# Product.

def run_product(M, N, K, a, b, kind, alpha=1.0, beta=0.0, c0=None, pad=0, workspace="caller"):
    """C (float32 NumPy) through gemm_mx, the padding of its rows checked."""
    t = torch()
    ldc = N + pad
    C = t.full((M * ldc + 8,), 7.0, dtype=dtype(kind), device="cuda:0")
    view = C[:M * ldc].view(M, ldc)
    if c0 is None:
        view[:, :N] = float("nan")
    else:
        view[:, :N] = dev(c0, kind)
    need = lib.gemm_mx_workspace_bytes(M, N, K)
    ws, wb = None, 0
    if workspace == "caller":
        ws, wb = t.full((max(need, 16),), 0xff, dtype=t.uint8, device="cuda:0"), max(need, 16)
    lib.gemm_mx(M, N, K, alpha, a[2], a[3], b[2], b[3], beta, C, ref.TYPES[kind], ldc, ws, wb, stream())
    got = host(C)
    assert (got[M * ldc:] == 7).all() and (got[:M * ldc].reshape(M, ldc)[:, N:] == 7).all(), "padding of C written"
    return got[:M * ldc].reshape(M, ldc)[:, :N]


def check_product(got, a, b, K, kind, alpha=1.0, beta=0.0, c0=None):
    """|C - ref| <= (K + 4) 2^-23 sum|a b| (an FP32 sum of K exact products, each
    addition off by at most 2^-23 of the magnitudes, and the epilogue's
    roundings) + half a step of the type."""
    A, B = ref.decode(a[0], a[1], K), ref.decode(b[0], b[1], K)
    want, S = ref.product(A, B, alpha, beta, c0)
    bound = (K + 4) * 2.0 ** -23 * S + ref.HALF_STEP[ref.TYPES[kind]] * np.abs(want) * 1.01 + (2.0 ** -25 if kind == "f16" else 0)
    bad = ~(np.abs(got.astype(np.float64) - want) <= bound)
    assert not bad.any(), f"{bad.sum()} outside, worst {np.nanmax(np.abs(got - want) / bound)}"


SHAPES = [(1, 1, 1), (1, 33, 64), (1, 4096, 512), (2, 31, 129), (7, 100, 1000), (15, 17, 33), (16, 64, 128), (17, 257, 383), (31, 16, 4096),
          (33, 65, 255), (64, 64, 256), (65, 129, 511), (100, 2000, 127), (128, 128, 1024), (129, 255, 640), (255, 257, 1025), (300, 70, 8192),
          (512, 384, 256), (513, 1000, 300), (40, 24, 65536), (1001, 777, 513)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", SHAPES, ids=[f"{m}x{n}x{k}" for m, n, k in SHAPES])
def test_product(kind, M, N, K):
    say(f"product {kind} {M}x{N}x{K}")
    rng = np.random.default_rng(M + 3 * N + 7 * K)
    a, b = operand(rng, M, K, 117, 125), operand(rng, N, K, 117, 125)
    check_product(run_product(M, N, K, a, b, kind), a, b, K, kind)


@pytest.mark.parametrize("M,N,K", SHAPES + [(4096, 128, 512), (2048, 2048, 1024), (200, 8192, 128)],
                         ids=lambda v: str(v))
def test_product_exact(M, N, K):
    """Scales within a factor of 4 of one: every product is a multiple of 2^-6 and
    every sum below 2^18 in magnitude (K 36 4 < 2^24 2^-6 needs K <= 1820; beyond,
    random signs keep the partial sums far below), so FP32 sums are exact in any
    order and the bits must match; a wrong lane, scale or row shows."""
    say(f"product exact {M}x{N}x{K}")
    rng = np.random.default_rng(K + M)
    a, b = operand(rng, M, K, 126, 128), operand(rng, N, K, 126, 128)
    got = run_product(M, N, K, a, b, "f32")
    want = ref.product(ref.decode(a[0], a[1], K), ref.decode(b[0], b[1], K))[0].astype(np.float32)
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(1, 100, 300), (33, 257, 1000), (300, 520, 384), (64, 48, 32768)])
@pytest.mark.parametrize("alpha,beta", [(2.0, -0.5), (-1.0, 1.0), (0.5, 0.0)])
def test_product_alpha_beta_strides(kind, M, N, K, alpha, beta):
    say(f"product {kind} {M}x{N}x{K} alpha {alpha} beta {beta}")
    rng = np.random.default_rng(M + N + K)
    a, b = operand(rng, M, K, 122, 126), operand(rng, N, K, 122, 126)
    c0 = ref.to_type(rng.standard_normal((M, N)), ref.TYPES[kind]) if beta else None
    for pad in (0, 3):
        check_product(run_product(M, N, K, a, b, kind, alpha, beta, c0, pad), a, b, K, kind, alpha, beta, c0)


@pytest.mark.parametrize("kind", KINDS)
def test_product_without_a_sum(kind):
    say(f"product {kind} alpha 0 and K 0")
    t = torch()
    c0 = np.arange(35, dtype=np.float32).reshape(5, 7)
    C = dev(c0, kind)
    lib.gemm_mx(5, 7, 64, 0.0, None, None, None, None, -2.0, C, ref.TYPES[kind], 7, None, 0, stream())
    np.testing.assert_array_equal(host(C), -2 * c0)
    C.fill_(float("nan"))
    lib.gemm_mx(5, 7, 0, 1.0, None, None, None, None, 0.0, C, ref.TYPES[kind], 7, None, 0, stream())
    assert not t.any(C != 0).item()


@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (20, 100, 4096), (300, 260, 512), (512, 512, 512), (32, 32, 65536)])
def test_product_nan_blocks_and_extreme_scales(M, N, K):
    """A NaN block of A makes its row of C NaN, one of B its column, nothing else;
    scales 2^-127 and 2^127 meet without harm."""
    say(f"product NaN blocks {M}x{N}x{K}")
    rng = np.random.default_rng(9)
    a, b = operand(rng, M, K, 127, 127), operand(rng, N, K, 127, 127)
    a[1][M // 2, (K // 32) // 2] = 255
    b[1][N - 1, 0] = 255
    a[1][0, 0], b[1][:N - 1, 0] = 0, 252      # 2^-127 by 2^125
    a, b = (*a[:2], bytes_dev(a[0]), bytes_dev(a[1])), (*b[:2], bytes_dev(b[0]), bytes_dev(b[1]))
    got = run_product(M, N, K, a, b, "f32")
    nan = np.zeros((M, N), bool)
    nan[M // 2], nan[:, N - 1] = True, True
    np.testing.assert_array_equal(np.isnan(got), nan)
    if M > 1:   # row 0: its first block is scaled by 2^-2 in all
        A, B = ref.decode(a[0], a[1], K), ref.decode(b[0], b[1], K)
        want = (A[0] * B[:N - 1]).sum(axis=1)
        assert (np.abs(got[0, :N - 1] - want) <= (K + 4) * 2.0 ** -23 * (np.abs(A[0]) * np.abs(B[:N - 1])).sum(axis=1)).all()


def test_product_library_workspace_and_streams_agree():
    """The library's workspace gives the caller's workspace's bits, also from two
    other streams at once, and twice the same."""
    t = torch()
    rng = np.random.default_rng(1)
    for M, N, K in [(40, 24, 65536), (1, 4096, 4096), (512, 512, 16384)]:
        say(f"product workspaces {M}x{N}x{K} need {lib.gemm_mx_workspace_bytes(M, N, K)}")
        a, b = operand(rng, M, K, 117, 125), operand(rng, N, K, 117, 125)
        want = run_product(M, N, K, a, b, "f32")
        np.testing.assert_array_equal(run_product(M, N, K, a, b, "f32", workspace="library"), want)
        streams = [t.cuda.Stream() for _ in range(3)]
        outs = [t.full((M, N), float("nan"), device="cuda:0") for _ in range(6)]
        t.cuda.synchronize()
        for i, o in enumerate(outs):
            lib.gemm_mx(M, N, K, 1.0, a[2], a[3], b[2], b[3], 0.0, o, ref.F32, N, None, 0, streams[i % 3].cuda_stream)
        t.cuda.synchronize()
        for o in outs:
            np.testing.assert_array_equal(host(o), want)


def test_product_captured_and_replayed():
    t = torch()
    rng = np.random.default_rng(2)
    for M, N, K in [(40, 24, 65536), (1, 4096, 4096), (300, 300, 300)]:
        need = lib.gemm_mx_workspace_bytes(M, N, K)
        say(f"product graph {M}x{N}x{K} need {need}")
        a, b, b2 = operand(rng, M, K, 117, 125), operand(rng, N, K, 117, 125), operand(rng, N, K, 117, 125)
        want = [run_product(M, N, K, a, x, "f32") for x in (b, b2)]
        bc, bs = b[2].clone(), b[3].clone()
        out = t.zeros((M, N), device="cuda:0")
        ws = t.empty(max(need, 16), dtype=t.uint8, device="cuda:0")
        g = t.cuda.CUDAGraph()
        if need:
            with pytest.raises(lib.GemmError) as e:
                with t.cuda.graph(t.cuda.CUDAGraph()):
                    lib.gemm_mx(M, N, K, 1.0, a[2], a[3], bc, bs, 0.0, out, ref.F32, N, None, 0, stream())
            assert e.value.status == lib.GEMM_ERR_CAPTURING
        with t.cuda.graph(g):
            lib.gemm_mx(M, N, K, 1.0, a[2], a[3], bc, bs, 0.0, out, ref.F32, N, ws, max(need, 16), stream())
        for n in range(4):
            src = (b, b2)[n % 2]
            bc.copy_(src[2])
            bs.copy_(src[3])
            out.fill_(float("nan"))
            g.replay()
            t.cuda.synchronize()
            np.testing.assert_array_equal(host(out), want[n % 2])


# ---------------------------------------------------------------------------
# The mixture-of-experts layer.

def layer_case(seed, T, H, I, E, kind, spread=(119, 122)):
    rng = np.random.default_rng(seed)
    x = ref.to_type(rng.standard_normal((T, H)), ref.TYPES[kind])
    w1, w2 = operand(rng, E * 2 * I, H, *spread), operand(rng, E * H, I, *spread)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    return x, logits, w1, w2


def run_layer(x, logits, w1, w2, I, top_k, renorm, kind, pad=0, workspace="caller", offset=0, s=None):
    t = torch()
    T, H = x.shape
    E = logits.shape[1]
    X, ldx = matrix(x, kind, pad, offset)
    L, ldl = matrix(logits, "f32", pad)
    ldy = H + pad
    y = t.full((T * ldy + 8,), 7.0, dtype=dtype(kind), device="cuda:0")
    need = lib.gemm_mx_moe_workspace_bytes(T, I, top_k, ref.TYPES[kind])
    ws, wb = None, 0
    if workspace == "caller":
        # NaN bits: what is read has to be written first
        ws, wb = t.full((need,), 0xff, dtype=t.uint8, device="cuda:0"), need
    lib.gemm_mx_moe(T, H, I, E, top_k, renorm, L, ldl, X, ref.TYPES[kind], ldx, w1[2], w1[3], w2[2], w2[3], y, ldy, ws, wb, stream())
    got = host(y)
    assert (got[T * ldy:] == 7).all() and (got[:T * ldy].reshape(T, ldy)[:, H:] == 7).all(), "padding of Y written"
    return got[:T * ldy].reshape(T, ldy)[:, :H]


PARTS = {"f32": (3, 3), "bf16": (1, 2), "f16": (2, 2)}


def check_layer(got, x, logits, w1, w2, I, top_k, renorm, kind):
    H, E = x.shape[1], logits.shape[1]
    weights = ref.route(logits, top_k, renorm)
    want, bound = ref.moe(x.astype(np.float64), weights, ref.decode(w1[0], w1[1], H), ref.decode(w2[0], w2[1], I), I, *PARTS[kind])
    bound = bound + ref.HALF_STEP[ref.TYPES[kind]] * (np.abs(want) + bound) + (2.0 ** -24 if kind == "f16" else 0)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    bad = ~(np.abs(got.astype(np.float64) - want) <= bound) & ~np.isnan(want)
    assert not bad.any(), f"{bad.sum()} outside, worst {np.nanmax(np.abs(got - want) / bound)}"
    return want, bound


LAYERS = [  # tokens, hidden, inter, experts, top_k
    (1, 128, 128, 4, 1), (1, 512, 256, 64, 4), (1, 100, 72, 3, 3), (2, 257, 129, 8, 2), (3, 33, 17, 512, 16), (7, 640, 200, 33, 5),
    (16, 256, 128, 16, 4), (17, 130, 255, 5, 5), (31, 384, 96, 128, 8), (48, 200, 130, 6, 2), (64, 256, 128, 2, 1), (64, 144, 64, 65, 8), (5, 1, 1, 1, 1),
    # activations that do not fit LDS: loaded again for every item
    (2, 17408, 40, 2, 1), (20, 7704, 33, 2, 1), (3, 6001, 20, 2, 2),
    # several batches of K a wave, experts in every width of the routing
    (9, 9000, 24, 20, 3), (40, 5120, 16, 200, 4), (33, 96, 4200, 300, 2)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,H,I,E,k", LAYERS, ids=["x".join(map(str, c)) for c in LAYERS])
@pytest.mark.parametrize("renorm", [True, False], ids=["renorm", "plain"])
def test_layer(kind, T, H, I, E, k, renorm):
    say(f"layer {kind} tokens {T} hidden {H} inter {I} experts {E} top {k} renorm {renorm}")
    x, logits, w1, w2 = layer_case(T + H + E, T, H, I, E, kind)
    pad = 0 if renorm else 3
    got = run_layer(x, logits, w1, w2, I, k, renorm, kind, pad, "caller", pad // 3)
    check_layer(got, x, logits, w1, w2, I, k, renorm, kind)


@pytest.mark.parametrize("T", [5, 40])
def test_layer_ties_and_masked_experts(T):
    """Equal logits go to the lowest index (-0 and +0 are equal); -inf is never
    chosen; a row of nothing else gives zeros; NaN and +inf make their row NaN and
    no other; the type's lowest value is an ordinary logit."""
    say(f"layer ties and masks, {T} tokens")
    H, I, E, k = 160, 64, 70, 4
    x, logits, w1, w2 = layer_case(3, T, H, I, E, "f32")
    logits = np.round(logits * 2) / 2 + 0.0
    logits[0, ::2] = -0.0
    logits[0, 1::2] = 0.0
    logits[1, :] = -np.inf
    logits[2, 3:] = -np.inf
    logits[3, :] = np.finfo(np.float32).min
    logits[4, 10] = np.nan
    if T > 30:
        logits[33, 69] = np.inf
        logits[35, 1:] = -np.inf
        logits[36, :] = 3.0
    for renorm in (True, False):
        got = run_layer(x, logits, w1, w2, I, k, renorm, "f32")
        check_layer(got, x, logits, w1, w2, I, k, renorm, "f32")
        assert (got[1] == 0).all() and np.isnan(got[4]).all()


def test_layer_nan_weights_stay_with_their_expert():
    say("layer NaN weights")
    T, H, I, E, k = 20, 192, 128, 6, 2
    x, logits, w1, w2 = layer_case(4, T, H, I, E, "bf16")
    for where in ("w1", "w2"):
        u1, u2 = w1[1].copy(), w2[1].copy()
        if where == "w1":
            u1.reshape(E, 2 * I, -1)[3, 40, 2] = 255
        else:
            u2.reshape(E, H, -1)[3, :, 1] = 255
        got = run_layer(x, logits, (w1[0], u1, w1[2], bytes_dev(u1)), (w2[0], u2, w2[2], bytes_dev(u2)), I, k, True, "bf16")
        reached = ref.route(logits, k, True)[:, 3] > 0
        assert 0 < reached.sum() < T
        np.testing.assert_array_equal(np.isnan(got).all(axis=1), reached)
        np.testing.assert_array_equal(np.isnan(got).any(axis=1), reached)


def test_layer_infinite_and_large_inputs():
    """An infinite input makes its own row not finite and no other; inputs near the
    largest float keep their value through the split."""
    say("layer infinite inputs")
    T, H, I, E, k = 4, 128, 32, 4, 2
    for kind in KINDS:
        x, logits, w1, w2 = layer_case(8, T, H, I, E, kind)
        x[1, 7] = np.inf
        got = run_layer(x, logits, w1, w2, I, k, True, kind)
        assert not np.isfinite(got[1]).any()
        rest = [0, 2, 3]
        check_layer(got[rest], x[rest], logits[rest], w1, w2, I, k, True, kind)


def test_layer_workspaces_streams_and_graph_agree():
    t = torch()
    T, H, I, E, k = 33, 512, 200, 40, 4
    x, logits, w1, w2 = layer_case(6, T, H, I, E, "bf16")
    _, logits2, _, _ = layer_case(7, T, H, I, E, "bf16")
    say("layer workspaces")
    want = [run_layer(x, l, w1, w2, I, k, True, "bf16") for l in (logits, logits2)]
    np.testing.assert_array_equal(run_layer(x, logits, w1, w2, I, k, True, "bf16", workspace="library"), want[0])
    X, L = dev(x, "bf16"), [dev(logits), dev(logits2)]
    streams = [t.cuda.Stream() for _ in range(3)]
    outs = [t.zeros((T, H), dtype=t.bfloat16, device="cuda:0") for _ in range(6)]
    t.cuda.synchronize()
    say("layer streams")
    for i, o in enumerate(outs):
        lib.gemm_mx_moe(T, H, I, E, k, True, L[i % 2], E, X, ref.BF16, H, w1[2], w1[3], w2[2], w2[3], o, H, None, 0, streams[i % 3].cuda_stream)
    t.cuda.synchronize()
    for i, o in enumerate(outs):
        np.testing.assert_array_equal(host(o), want[i % 2])
    say("layer graph")
    need = lib.gemm_mx_moe_workspace_bytes(T, I, k, ref.BF16)
    ws, out, lg = t.empty(need, dtype=t.uint8, device="cuda:0"), outs[0], L[0].clone()
    with pytest.raises(lib.GemmError) as e:
        with t.cuda.graph(t.cuda.CUDAGraph()):
            lib.gemm_mx_moe(T, H, I, E, k, True, lg, E, X, ref.BF16, H, w1[2], w1[3], w2[2], w2[3], out, H, None, 0, stream())
    assert e.value.status == lib.GEMM_ERR_CAPTURING
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        lib.gemm_mx_moe(T, H, I, E, k, True, lg, E, X, ref.BF16, H, w1[2], w1[3], w2[2], w2[3], out, H, ws, need, stream())
    for n in range(4):
        lg.copy_(L[n % 2])
        out.fill_(float("nan"))
        g.replay()
        t.cuda.synchronize()
        np.testing.assert_array_equal(host(out), want[n % 2])


# ---------------------------------------------------------------------------
# Together, as they are used.

@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_linear_layer_forward_and_gradients(kind):
    """Y = X W, dX = dY W^T, dW = X^T dY, each operand quantised along the axis its
    product sums over, against the formulas on the quantised values; and the
    FP32 products of this library on the dequantised operands agree."""
    t = torch()
    M, K, N = 70, 200, 150
    say(f"linear layer {kind}")
    rng = np.random.default_rng(12)
    x, w, dy = (ref.to_type(rng.standard_normal(s), ref.TYPES[kind]) for s in ((M, K), (K, N), (M, N)))
    dx_, dw_, ddy = dev(x, kind), dev(w, kind), dev(dy, kind)

    def quantize(src, trans, rows, k):
        c, s = operand_buffers(rows, k, 0)
        lib.gemm_mx_quantize(trans, rows, k, src, ref.TYPES[kind], rows if trans else k, c, s, stream())
        return c, s

    def product(m, n, k, a, b):
        out = t.full((m, n), float("nan"), device="cuda:0")
        lib.gemm_mx(m, n, k, 1.0, *a, *b, 0.0, out, ref.F32, n, None, 0, stream())
        return host(out)

    def q(v):
        return ref.decode(*ref.quantize(v), v.shape[1])

    xq, wt = quantize(dx_, False, M, K), quantize(dw_, True, N, K)
    got = {"y": product(M, N, K, xq, wt),
           "dx": product(M, K, N, quantize(ddy, False, M, N), quantize(dw_, False, K, N)),
           "dw": product(K, N, M, quantize(dx_, True, K, M), quantize(ddy, True, N, M))}
    pairs = {"y": (q(x), q(w.T)), "dx": (q(dy), q(w)), "dw": (q(x.T), q(dy.T))}
    for name, (a, b) in pairs.items():
        want, S = ref.product(a, b)
        assert (np.abs(got[name] - want) <= (a.shape[1] + 4) * 2.0 ** -23 * S).all(), name
    av, bv = t.empty((M, K), device="cuda:0"), t.empty((K, N), device="cuda:0")
    lib.gemm_mx_dequantize(False, M, K, *xq, av, ref.F32, K, stream())
    lib.gemm_mx_dequantize(True, N, K, *wt, bv, ref.F32, N, stream())
    c32 = t.empty((M, N), device="cuda:0")
    lib.gemm_f32(av, bv, c32, M, N, K, stream())
    want, S = ref.product(*pairs["y"])
    assert (np.abs(host(c32) - want) <= (K + 4) * 2.0 ** -23 * S).all()


def test_linear_layer_gradients_against_differences():
    """On operands that quantisation leaves unchanged the gradients of L = sum(dY * Y)
    are those of the product itself: a step in one element of X or W that stays
    representable changes L by exactly the gradient times the step (all values
    small multiples of powers of two, so every number here is exact)."""
    t = torch()
    M, K, N = 5, 64, 32
    say("linear layer differences")
    rng = np.random.default_rng(2)

    def grid(*shape):   # e2m1 values with a 6 in every block along either axis
        v = rng.choice([0.0, 0.5, 1.0, 1.5, 2.0, -1.0, -0.5], shape)
        v[:, ::32], v[::32, :] = 6.0, 6.0
        return v

    x, w, dy = grid(M, K), grid(K, N), grid(M, N)

    def run(a, b, m, n, k):   # rows of k values each
        ca, cb = operand_buffers(m, k, 0), operand_buffers(n, k, 0)
        lib.gemm_mx_quantize(False, m, k, dev(a), ref.F32, k, *ca, stream())
        lib.gemm_mx_quantize(False, n, k, dev(b), ref.F32, k, *cb, stream())
        out = t.empty((m, n), device="cuda:0")
        lib.gemm_mx(m, n, k, 1.0, *ca, *cb, 0.0, out, ref.F32, n, None, 0, stream())
        return host(out).astype(np.float64)

    dx, dw = run(dy, w, M, K, N), run(x.T, dy.T, K, N, M)
    base = (dy * run(x, w.T, M, N, K)).sum()
    for i, j in ((1, 1), (3, 40), (4, 63)):
        step = x.copy()
        step[i, j] += 0.5 if x[i, j] < 2 else 1.0
        assert (dy * run(step, w.T, M, N, K)).sum() - base == dx[i, j] * (step[i, j] - x[i, j])
    for i, j in ((1, 1), (33, 5), (63, 31)):
        step = w.copy()
        step[i, j] += 0.5 if w[i, j] < 2 else 1.0
        assert (dy * run(x, step.T, M, N, K)).sum() - base == dw[i, j] * (step[i, j] - w[i, j])


def test_decoding_step():
    """A step of a decoder's feed-forward part: the router's logits by gemm_f32, the
    layer on weights quantised here, its output quantised and through a product."""
    t = torch()
    T, H, I, E, k, N = 3, 256, 96, 8, 2, 200
    say("decoding step")
    rng = np.random.default_rng(21)
    x = ref.to_type(rng.standard_normal((T, H)), ref.BF16)
    wr = rng.standard_normal((H, E)).astype(np.float32) / 16
    w1, w2, w3 = (ref.to_type(rng.standard_normal(s) / 16, ref.BF16) for s in ((E * 2 * I, H), (E * H, I), (N, H)))
    q = []
    for w in (w1, w2, w3):
        c, s = operand_buffers(*w.shape, 0)
        lib.gemm_mx_quantize(False, *w.shape, dev(w, "bf16"), ref.BF16, w.shape[1], c, s, stream())
        q.append((*ref.quantize(w), c, s))
    X, logits = dev(x, "bf16"), t.empty((T, E), device="cuda:0")
    lib.gemm_f32(X.float(), dev(wr), logits, T, E, H, stream())
    y = t.empty((T, H), dtype=t.bfloat16, device="cuda:0")
    lib.gemm_mx_moe(T, H, I, E, k, True, logits, E, X, ref.BF16, H, q[0][2], q[0][3], q[1][2], q[1][3], y, H, None, 0, stream())
    yc, ys = operand_buffers(T, H, 0)
    lib.gemm_mx_quantize(False, T, H, y, ref.BF16, H, yc, ys, stream())
    out = t.empty((T, N), dtype=t.bfloat16, device="cuda:0")
    lib.gemm_mx(T, N, H, 1.0, yc, ys, q[2][2], q[2][3], 0.0, out, ref.BF16, N, None, 0, stream())
    check_layer(host(y), x, logits.cpu().numpy(), q[0], q[1], I, k, True, "bf16")
    codes, scales = ref.quantize(host(y))
    check_product(host(out), (codes, scales), q[2], H, "bf16")


# ---------------------------------------------------------------------------
# Sizes and calls at the edge of what is allowed.

def test_product_of_an_operand_with_itself_into_an_unaligned_c():
    t = torch()
    M, K = 150, 700
    say("product X X^T, C one element off")
    rng = np.random.default_rng(31)
    a = operand(rng, M, K, 126, 128)
    for kind in KINDS:
        C = t.full((M * M + 2,), 7.0, dtype=dtype(kind), device="cuda:0")
        lib.gemm_mx(M, M, K, 1.0, a[2], a[3], a[2], a[3], 0.0, C[1:], ref.TYPES[kind], M, None, 0, stream())
        got = host(C)
        assert got[0] == 7 and got[-1] == 7
        check_product(got[1:-1].reshape(M, M), a, a, K, kind)


@pytest.mark.parametrize("M,N", [(1, 40), (20, 24), (300, 260)])
def test_product_of_the_longest_rows(M, N):
    """K = 2^24: rows of 8 MiB of codes, a tile's offsets up to 2^31. Zero but for a
    few blocks at the ends and in the middle, so that sums are exact."""
    t = torch()
    K = lib.GEMM_MX_MAX_K
    say(f"product {M}x{N}x{K}")
    rng = np.random.default_rng(32)
    blocks = [0, 1, 5, K // 64 - 1, K // 64, K // 32 - 3, K // 32 - 1]
    sides = []
    for rows in (M, N):
        c = t.zeros((rows, K // 2), dtype=t.uint8, device="cuda:0")
        s = t.full((rows, K // 32), 127, dtype=t.uint8, device="cuda:0")
        part = rng.integers(0, 256, (rows, len(blocks), 16), dtype=np.uint8)
        for j, b in enumerate(blocks):
            c[:, 16 * b:16 * b + 16] = bytes_dev(part[:, j])
        packed = np.zeros((rows, ref.padded(32 * len(blocks)) // 2), np.uint8)
        packed[:, :16 * len(blocks)] = part.reshape(rows, -1)
        sides.append((c, s, ref.decode(packed, np.full((rows, packed.shape[1] // 16), 127, np.uint8), 32 * len(blocks))))
    out = t.full((M, N), float("nan"), device="cuda:0")
    lib.gemm_mx(M, N, K, 1.0, sides[0][0], sides[0][1], sides[1][0], sides[1][1], 0.0, out, ref.F32, N, None, 0, stream())
    np.testing.assert_array_equal(host(out), (sides[0][2] @ sides[1][2].T).astype(np.float32))


def test_product_with_more_outputs_than_32_bits_count():
    t = torch()
    M, N, K = 66001, 33001, 128
    say(f"product {M}x{N}x{K} bf16")
    rng = np.random.default_rng(33)
    a, b = operand(rng, M, K, 126, 127), operand(rng, N, K, 126, 127)
    C = t.full((M, N), float("nan"), dtype=t.bfloat16, device="cuda:0")
    lib.gemm_mx(M, N, K, 1.0, a[2], a[3], b[2], b[3], 0.0, C, ref.BF16, N, None, 0, stream())
    assert not t.isnan(C).any().item()
    for rows in (slice(0, 40), slice(M // 2, M // 2 + 40), slice(M - 40, M)):
        part = (a[0][rows], a[1][rows])
        check_product(host(C[rows]), part, b, K, "bf16")


def test_layer_at_its_limits():
    """64 tokens on 16 of 512 experts; and weights past 2^32 bytes, the last expert
    chosen."""
    t = torch()
    say("layer at its limits: tokens, experts, top_k")
    for kind in KINDS:
        x, logits, w1, w2 = layer_case(41, 64, 48, 20, 512, kind)
        check_layer(run_layer(x, logits, w1, w2, 20, 16, True, kind), x, logits, w1, w2, 20, 16, True, kind)
    H, I, E = 8192, 8192, 128
    say(f"layer with {lib.gemm_mx_codes_bytes(E * 2 * I, H) >> 20} MiB of codes")
    rng = np.random.default_rng(42)
    one1, one2 = operand(rng, 2 * I, H, 119, 122), operand(rng, H, I, 119, 122)
    full = []
    for rows, one, k in ((2 * I, one1, H), (H, one2, I)):
        c = t.zeros((E, rows, k // 2), dtype=t.uint8, device="cuda:0")
        s = t.full((E, rows, k // 32), 120, dtype=t.uint8, device="cuda:0")
        c[E - 1], s[E - 1] = one[2], one[3]
        full += [c, s]
    x = ref.to_type(rng.standard_normal((2, H)), ref.BF16)
    logits = np.zeros((2, E), np.float32)
    logits[:, E - 1] = 5.0
    y = t.empty((2, H), dtype=t.bfloat16, device="cuda:0")
    lib.gemm_mx_moe(2, H, I, E, 1, True, dev(logits), E, dev(x, "bf16"), ref.BF16, H, *full, y, H, None, 0, stream())
    check_layer(host(y), x, np.zeros((2, 1), np.float32), one1, one2, I, 1, True, "bf16")
