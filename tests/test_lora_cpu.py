"""gemm_lora and gemm_lora_backward without a GPU: sizes and refusals (every check runs
before any HIP call), and the NumPy reference of the GPU tests against hand-worked rows
and differences."""
import ctypes
import os
import re

import numpy as np

import rows_reference as ref
from fp32_gemm_07_amd import binding as lib

VP = ctypes.c_void_p
BASE = 0x7f0000000000
A, B, RANKS, SCALES, IDS, X, C, Y, DY, DX, DA, DB, WS = (BASE + i * 0x1000000000 for i in range(13))


def _vp(p):
    return VP(p) if p else None


def adapters(type=0, n=24, k=16, rank=4, count=3, a=A, b=B, ranks=RANKS, scales=SCALES):
    return lib.gemm_lora_t(type, n, k, rank, count, a, b, ranks, scales)


def forward(rows=8, set=None, null_set=False, ids=IDS, x=X, ldx=16, c=C, ldc=24, y=Y, ldy=24, ws=WS, wb=1 << 30, **more):
    s = set or adapters(**more)
    return lib.raw_status("gemm_lora", rows, None if null_set else ctypes.byref(s), _vp(ids), _vp(x), ldx, _vp(c), ldc, _vp(y), ldy, _vp(ws), wb, None)


def backward(rows=8, null_set=False, ids=IDS, x=X, ldx=16, dy=DY, lddy=24, c=C, ldc=16, dx=DX, lddx=16, da=DA, db=DB, ws=WS, wb=1 << 40, **more):
    s = adapters(**more)
    return lib.raw_status("gemm_lora_backward", rows, None if null_set else ctypes.byref(s), _vp(ids), _vp(x), ldx, _vp(dy), lddy, _vp(c), ldc, _vp(dx), lddx,
                          _vp(da), _vp(db), _vp(ws), wb, None)


SET_DIMS = ({"rows": -1}, {"rows": lib.GEMM_LORA_MAX_ROWS + 1}, {"n": 0}, {"k": 0}, {"rank": 0}, {"rank": lib.GEMM_LORA_MAX_RANK + 1}, {"count": 0},
            {"count": lib.GEMM_LORA_MAX_ADAPTERS + 1}, {"n": lib.GEMM_LORA_MAX_DIM + 1}, {"k": lib.GEMM_LORA_MAX_DIM + 1}, {"n": -5})


def test_forward_refusals():
    for bad in SET_DIMS + ({"ldx": 15}, {"ldc": 23}, {"ldy": 23}):
        assert forward(**bad) == lib.GEMM_ERR_INVALID_DIM, bad
    assert forward(type=3) == forward(type=-1) == lib.GEMM_ERR_INVALID_TYPE
    assert forward(null_set=True) == lib.GEMM_ERR_NULL_PTR
    for name in ("ids", "x", "y", "a", "b"):
        assert forward(**{name: None}) == lib.GEMM_ERR_NULL_PTR, name
    for bad in ({"ids": IDS + 2}, {"x": X + 2}, {"y": Y + 1}, {"c": C + 2}, {"a": A + 2}, {"b": B + 1}, {"ranks": RANKS + 2}, {"scales": SCALES + 3},
                {"type": 1, "x": X + 1}):
        assert forward(**bad) == lib.GEMM_ERR_ALIGNMENT, bad
    # Y on everything else; on C but for the whole of it with the same stride
    last = 4 * (8 * 24 - 1)
    for p in (X, A, B, RANKS, SCALES, IDS, X - last, A + 4 * (3 * 4 * 16 - 1), B + 4 * (3 * 4 * 24 - 1)):
        assert forward(y=p) == lib.GEMM_ERR_ALIAS, hex(p)
    assert forward(y=C + 4) == forward(y=C, ldy=25) == forward(y=C - last) == lib.GEMM_ERR_ALIAS
    assert lib.gemm_lora_workspace_bytes(8, adapters()) == 0   # one kernel
    wide = {"rows": 65, "ldx": 16}
    need = lib.gemm_lora_workspace_bytes(65, adapters())
    assert need >= 65 * 4 * 4
    assert forward(wb=need - 1, **wide) == lib.GEMM_ERR_WORKSPACE
    assert forward(ws=WS + 8, **wide) == lib.GEMM_ERR_ALIGNMENT
    for p in (X, C, Y, IDS, A, B, RANKS, SCALES):
        assert forward(ws=p, wb=need, **wide) == lib.GEMM_ERR_ALIAS
    assert forward(rows=0, ids=None, x=None, c=None, y=None, a=None, b=None, ws=None, wb=0) == lib.GEMM_OK


def test_backward_refusals():
    for bad in SET_DIMS + ({"ldx": 15}, {"lddy": 23}, {"ldc": 15}, {"lddx": 15}):
        assert backward(**bad) == lib.GEMM_ERR_INVALID_DIM, bad
    assert backward(type=9) == lib.GEMM_ERR_INVALID_TYPE
    assert backward(null_set=True) == lib.GEMM_ERR_NULL_PTR
    for name in ("ids", "x", "dy", "a", "b", "da", "db"):   # (one of dA and dB)
        assert backward(**{name: None}) == lib.GEMM_ERR_NULL_PTR, name
    for bad in ({"ids": IDS + 1}, {"x": X + 2}, {"dy": DY + 2}, {"c": C + 1}, {"dx": DX + 2}, {"da": DA + 2}, {"db": DB + 1}):
        assert backward(**bad) == lib.GEMM_ERR_ALIGNMENT, bad
    for p in (X, DY, A, B, RANKS, SCALES, IDS):
        assert backward(dx=p) == backward(da=p) == backward(db=p) == lib.GEMM_ERR_ALIAS, hex(p)
    assert backward(dx=DA) == backward(da=DB) == backward(da=C) == backward(db=C) == backward(dx=C, da=C) == lib.GEMM_ERR_ALIAS
    assert backward(dx=C + 4) == backward(dx=C, lddx=17) == lib.GEMM_ERR_ALIAS
    need = lib.gemm_lora_backward_workspace_bytes(8, adapters())
    assert backward(wb=need - 1) == lib.GEMM_ERR_WORKSPACE
    assert backward(ws=WS + 4) == lib.GEMM_ERR_ALIGNMENT
    for p in (X, C, DY, DX, DA, DB, IDS, A, B, RANKS, SCALES):
        assert backward(ws=p, wb=need) == lib.GEMM_ERR_ALIAS
    assert backward(dx=None, da=None, db=None, ids=None, x=None, dy=None) == lib.GEMM_OK
    assert backward(rows=0, da=None, db=None, ids=None, x=None, dy=None, a=None, b=None) == lib.GEMM_OK


def test_workspace_sizes():
    for bad in ({"n": 0}, {"rank": 129}, {"type": 4}, {"count": 1025}):
        assert lib.gemm_lora_workspace_bytes(8, adapters(**bad)) == lib.gemm_lora_backward_workspace_bytes(8, adapters(**bad)) == 0, bad
    assert lib.gemm_lora_workspace_bytes(0, adapters()) == lib.gemm_lora_workspace_bytes(-1, adapters()) == 0
    # H alone for many rows, whatever the columns: floats, or three bfloat16 parts
    many = {"n": 1 << 18, "k": 1 << 18, "rank": 128}
    assert lib.gemm_lora_workspace_bytes(1 << 20, adapters(**many)) == (1 << 20) * 128 * 4
    assert lib.gemm_lora_workspace_bytes(1 << 20, adapters(type=1, **many)) == (1 << 20) * 128 * 6
    # past 32 bits: B once more
    assert lib.gemm_lora_backward_workspace_bytes(1, adapters(n=1 << 18, rank=128, count=1024)) > (1 << 18) * 128 * 1024 * 4


def test_binding_mirrors_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gemm.h")).read()
    found = re.findall(r"\b(GEMM_LORA_\w+)\s*=\s*(\d+)(?:\s*<<\s*(\d+))?", text)
    assert len(found) == 4
    for name, value, shift in found:
        assert getattr(lib, name) == int(value) << int(shift or 0), name


def test_reference_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a = np.array([[[1.0, 0.0], [9.0, 9.0]], [[0.0, 1.0], [1.0, 1.0]]])
    b = np.array([[[2.0, 9.0]], [[1.0, 10.0]]])
    y, mag = ref.lora(x, np.array([[100.0], [200.0], [300.0]]), a, b, np.array([1, 0, -1]), np.array([1, 2]), np.array([0.5, 2.0]))
    assert y.tolist() == [[100 + 2 * (2 + 30)], [200 + 0.5 * 2 * 3], [300]] and mag.tolist() == y.tolist()


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(7)
    x, c, dy = rng.normal(size=(6, 5)), rng.normal(size=(6, 4)), rng.normal(size=(6, 4))
    a, b = rng.normal(size=(3, 3, 5)), rng.normal(size=(3, 4, 3))
    ids, ranks, scales = np.array([0, 1, 1, -1, 0, 7]), np.array([2, 3, 1]), np.array([0.5, -2.0, 1.0])
    (dx, da, db), _ = ref.lora_backward(x, dy, None, a, b, ids, ranks, scales)

    def loss():
        return (ref.lora(x, c, a, b, ids, ranks, scales)[0] * dy).sum()

    h = 1e-6   # the loss is bilinear in each: differences are exact but for 2^-52 / h
    for array, grad in ((x, dx), (a, da), (b, db)):
        for at in np.ndindex(*array.shape):
            keep = array[at]
            array[at] = keep + h
            up = loss()
            array[at] = keep - h
            down = loss()
            array[at] = keep
            assert abs((up - down) / (2 * h) - grad[at]) < 1e-7, at


def test_backward_does_not_look_at_x_without_the_adapters_gradients():
    """dX needs dY, A and B alone: the call comes as far as its last check, the workspace's, whatever X is."""
    need = lib.gemm_lora_backward_workspace_bytes(8, adapters())
    for x in ({"x": None}, {"x": None, "ldx": 0}, {"x": X + 2}, {"dx": X, "c": None}, {"dx": X, "c": X}):
        assert backward(da=None, db=None, wb=need - 1, **x) == lib.GEMM_ERR_WORKSPACE, x
    for x in ({"x": None}, {"x": X + 2, "da": None}):
        assert backward(wb=need - 1, **x) in (lib.GEMM_ERR_NULL_PTR, lib.GEMM_ERR_ALIGNMENT), x
