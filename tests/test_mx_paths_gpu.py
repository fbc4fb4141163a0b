"""The gemm_mx* entry points on the GPU: what tests/test_mx_gpu.py leaves open, against
the same reference (tests/mx_reference.py) and by the same rules."""
import numpy as np
import pytest

import mx_reference as ref
from fp32_gemm_07_amd import binding as lib
from gpu_util import say, torch
from test_mx_gpu import KINDS, bytes_dev, run_layer

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
