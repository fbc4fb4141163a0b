"""The gemm_mx* entry points without a GPU: sizes and refusals (every check runs
before any HIP call), and the NumPy reference of the GPU tests against hand-worked
blocks."""
import ctypes

import numpy as np
import pytest

import mx_reference as ref
from fp32_gemm_07_amd import binding as lib

VP = ctypes.c_void_p
BASE = 0x7f0000000000
X, CODES, SCALES, C = (VP(BASE + i * 0x1000000000) for i in range(4))
CODES2, SCALES2, WS = (VP(BASE + i * 0x1000000000) for i in range(4, 7))
f = ctypes.c_float


def at(p, by):
    return VP(p.value + by)


def test_sizes():
    assert lib.gemm_mx_codes_bytes(3, 128) == 3 * 64 and lib.gemm_mx_scales_bytes(3, 128) == 3 * 4
    assert lib.gemm_mx_codes_bytes(3, 129) == 3 * 128 and lib.gemm_mx_scales_bytes(3, 129) == 3 * 8
    assert lib.gemm_mx_codes_bytes(0, 5) == 0 and lib.gemm_mx_codes_bytes(5, 0) == 0
    assert lib.gemm_mx_codes_bytes(-1, 5) == 0 and lib.gemm_mx_scales_bytes(1, -5) == 0
    assert lib.gemm_mx_codes_bytes(1, lib.GEMM_MX_MAX_K + 1) == 0
    assert lib.gemm_mx_codes_bytes(2 ** 31 - 1, 4096) == 0   # more than 2^40 values
    # past 32 bits
    assert lib.gemm_mx_codes_bytes(1 << 20, 8192) == (1 << 20) * 4096
    # hidden activations in 2 or 3 bfloat16 parts, and the list of reached experts
    few = lib.gemm_mx_moe_workspace_bytes(1, 1, 1, lib.GEMM_TYPE_BF16) - 2 * 128 * 2
    assert 0 < few <= 16384
    assert lib.gemm_mx_moe_workspace_bytes(2, 100, 3, lib.GEMM_TYPE_BF16) == 2 * 3 * 128 * 2 * 2 + few
    assert lib.gemm_mx_moe_workspace_bytes(2, 100, 3, lib.GEMM_TYPE_F32) == 3 * 2 * 3 * 128 * 2 + few
    for bad in ((0, 1, 1, 0), (65, 1, 1, 0), (1, 0, 1, 0), (1, 1, 0, 0), (1, 1, 17, 0), (1, 1, 1, 3)):
        assert lib.gemm_mx_moe_workspace_bytes(*bad) == 0


def _workspaces():
    for M, N, K in ((1, 4096, 4096), (512, 512, 131072), (4096, 4096, 4096), (1, 1, 1 << 24), (33, 65, 999999)):
        yield M, N, K, lib.gemm_mx_workspace_bytes(M, N, K)


def test_product_workspace_is_bounded():
    for M, N, K, need in _workspaces():
        assert 0 <= need <= 64 << 20, (M, N, K, need)
    for bad in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (-1, 4, 4), (4, 4, lib.GEMM_MX_MAX_K + 1)):
        assert lib.gemm_mx_workspace_bytes(*bad) == 0


@pytest.mark.parametrize("entry", ["gemm_mx_quantize", "gemm_mx_dequantize"])
def test_conversion_refusals(entry):
    def st(trans=0, rows=8, K=64, x=X, kind=0, ld=64, codes=CODES, scales=SCALES):
        if entry == "gemm_mx_quantize":
            return lib.raw_status(entry, trans, rows, K, x, kind, ld, codes, scales, None)
        return lib.raw_status(entry, trans, rows, K, codes, scales, x, kind, ld, None)

    assert st(rows=-1) == st(K=-1) == lib.GEMM_ERR_INVALID_DIM
    assert st(ld=63) == lib.GEMM_ERR_INVALID_DIM
    assert st(trans=1, ld=7) == lib.GEMM_ERR_INVALID_DIM
    assert st(K=lib.GEMM_MX_MAX_K + 1, ld=lib.GEMM_MX_MAX_K + 1) == lib.GEMM_ERR_INVALID_DIM
    assert st(rows=2 ** 31 - 1, K=4096, ld=4096) == lib.GEMM_ERR_INVALID_DIM
    assert st(rows=2 ** 20, ld=2 ** 30) == lib.GEMM_ERR_INVALID_DIM
    assert st(kind=3) == st(kind=-1) == lib.GEMM_ERR_INVALID_TYPE
    assert st(x=None) == st(codes=None) == st(scales=None) == lib.GEMM_ERR_NULL_PTR
    assert st(x=at(X, 2)) == st(kind=1, x=at(X, 1)) == lib.GEMM_ERR_ALIGNMENT
    assert st(codes=at(CODES, 8)) == st(scales=at(SCALES, 2)) == lib.GEMM_ERR_ALIGNMENT
    assert st(x=CODES) == st(x=SCALES) == lib.GEMM_ERR_ALIAS
    assert st(codes=at(X, 8 * 64 * 4 - 16)) == lib.GEMM_ERR_ALIAS
    if entry == "gemm_mx_quantize":
        assert st(scales=CODES) == lib.GEMM_ERR_ALIAS
    # nothing to do
    assert st(rows=0, x=None, codes=None, scales=None) == lib.GEMM_OK
    assert st(K=0, x=None, codes=None, scales=None) == lib.GEMM_OK


def product(M=8, N=8, K=64, alpha=1.0, ac=CODES, sa=SCALES, bc=CODES2, sb=SCALES2, beta=0.0, c=C, kind=0, ldc=8, ws=None, wb=0):
    return lib.raw_status("gemm_mx", M, N, K, f(alpha), ac, sa, bc, sb, f(beta), c, kind, ldc, ws, wb, None)


def test_product_refusals():
    assert product(M=-1) == product(N=-1) == product(K=-1) == lib.GEMM_ERR_INVALID_DIM
    assert product(K=lib.GEMM_MX_MAX_K + 1) == product(ldc=7) == lib.GEMM_ERR_INVALID_DIM
    assert product(M=2 ** 31 - 1, N=4096, ldc=4096) == lib.GEMM_ERR_INVALID_DIM
    assert product(kind=7) == lib.GEMM_ERR_INVALID_TYPE
    for name in ("ac", "sa", "bc", "sb", "c"):
        assert product(**{name: None}) == lib.GEMM_ERR_NULL_PTR, name
    assert product(ac=at(CODES, 8)) == product(bc=at(CODES2, 4)) == lib.GEMM_ERR_ALIGNMENT
    assert product(sa=at(SCALES, 1)) == product(sb=at(SCALES2, 2)) == lib.GEMM_ERR_ALIGNMENT
    assert product(c=at(C, 2)) == lib.GEMM_ERR_ALIGNMENT
    for p in (CODES, SCALES, CODES2, SCALES2):
        assert product(c=p) == lib.GEMM_ERR_ALIAS
    assert product(M=0, ac=None, sa=None, bc=None, sb=None, c=None) == lib.GEMM_OK
    assert product(N=0, ac=None, sa=None, bc=None, sb=None, c=None) == lib.GEMM_OK
    need = lib.gemm_mx_workspace_bytes(512, 512, 131072)
    if need:
        assert product(M=512, N=512, K=131072, ldc=512, ws=WS, wb=need - 1) == lib.GEMM_ERR_WORKSPACE
        assert product(M=512, N=512, K=131072, ldc=512, ws=at(WS, 8), wb=need) == lib.GEMM_ERR_ALIGNMENT
        assert product(M=512, N=512, K=131072, ldc=512, ws=C, wb=need) == lib.GEMM_ERR_ALIAS
        assert product(M=512, N=512, K=131072, ldc=512, ws=CODES, wb=need) == lib.GEMM_ERR_ALIAS


def layer(tokens=2, hidden=64, inter=32, experts=4, top_k=2, logits=X, ldl=4, x=at(X, 0x10000000), kind=0, ldx=64, w1c=CODES, w1s=SCALES, w2c=CODES2,
          w2s=SCALES2, y=C, ldy=64, ws=WS, wb=1 << 30):
    return lib.raw_status("gemm_mx_moe", tokens, hidden, inter, experts, top_k, 1, logits, ldl, x, kind, ldx, w1c, w1s, w2c, w2s, y, ldy, ws, wb, None)


def test_layer_refusals():
    for bad in ({"tokens": -1}, {"tokens": 65}, {"hidden": 0}, {"inter": 0}, {"experts": 0}, {"experts": 513, "ldl": 513}, {"top_k": 0},
                {"top_k": 5}, {"experts": 32, "ldl": 32, "top_k": 17}, {"ldl": 3}, {"ldx": 63}, {"ldy": 63}, {"hidden": 1 << 25, "ldx": 1 << 25, "ldy": 1 << 25}):
        assert layer(**bad) == lib.GEMM_ERR_INVALID_DIM, bad
    assert layer(kind=5) == lib.GEMM_ERR_INVALID_TYPE
    for name in ("logits", "x", "w1c", "w1s", "w2c", "w2s", "y"):
        assert layer(**{name: None}) == lib.GEMM_ERR_NULL_PTR, name
    assert layer(w1c=at(CODES, 8)) == layer(w2s=at(SCALES2, 2)) == layer(x=at(X, 0x10000002)) == lib.GEMM_ERR_ALIGNMENT
    for p in (X, at(X, 0x10000000), CODES, SCALES, CODES2, SCALES2):
        assert layer(y=p) == lib.GEMM_ERR_ALIAS
    need = lib.gemm_mx_moe_workspace_bytes(2, 32, 2, 0)
    assert layer(wb=need - 1) == lib.GEMM_ERR_WORKSPACE
    assert layer(ws=at(WS, 8)) == lib.GEMM_ERR_ALIGNMENT
    for p in (X, at(X, 0x10000000), CODES, SCALES, CODES2, SCALES2, C):
        assert layer(ws=p, wb=need) == lib.GEMM_ERR_ALIAS
    assert layer(tokens=0, logits=None, x=None, w1c=None, w1s=None, w2c=None, w2s=None, y=None, ws=None, wb=0) == lib.GEMM_OK


def test_new_statuses_have_text():
    texts = {lib.gemm_status_string(s) for s in range(12)}
    assert len(texts) == 12 and "unknown status" not in texts


def test_reference_by_hand():
    # max 7: scale 2^(2 - 2) = 1; ties go to the even code, 7 saturates
    x = np.zeros((1, 32))
    x[0, :12] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5.5, 0.26, -0.1, -0.0]
    codes, scales = ref.quantize(x)
    assert scales[0, 0] == 127 and (scales[0, 1:] == 0).all()
    n = np.stack((codes & 15, codes >> 4), -1).reshape(-1)[:12]
    assert list(n) == [7, 0, 2, 2, 4, 4, 6, 6, 15, 1, 8, 8]
    assert list(ref.decode(codes, scales, 12)[0]) == [6, 0, 1, 1, 2, 2, 4, 4, -6, 0.5, 0, 0]
    x[0, 3] = np.inf
    codes, scales = ref.quantize(x)
    assert scales[0, 0] == 255 and (codes == 0).all() and np.isnan(ref.decode(codes, scales, 32)).all()
    tiny = np.full((1, 32), 2.0 ** -149)
    codes, scales = ref.quantize(tiny)
    assert scales[0, 0] == 0 and (codes == 0).all()
    w = ref.route(np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0, np.nan, 1, 2]]), 2, True)
    assert list(w[0]) == [0, 0.5, 0.5, 0] and list(w[1]) == [0] * 4 and np.isnan(w[2]).all()
