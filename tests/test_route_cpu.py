"""gemm_route, gemm_route_backward and gemm_mx_moe_routed without a GPU: refusals (every
check runs before any HIP call), and the NumPy reference of the GPU tests against
hand-worked choices and differences."""
import ctypes
import os
import re

import numpy as np
import pytest

import rows_reference as ref
from fp32_gemm_07_amd import binding as lib

VP = ctypes.c_void_p
BASE = 0x7f0000000000
LOGITS, BIAS, CHOSEN, WEIGHTS, COUNTS, DW, DL = (VP(BASE + i * 0x1000000000) for i in range(7))
X, Y, W1C, W1S, W2C, W2S, WS = (VP(BASE + i * 0x1000000000) for i in range(7, 14))


def at(p, by):
    return VP(p.value + by)


def route(tokens=4, experts=16, top_k=2, score=0, groups=1, top_groups=1, group_top=1, logits=LOGITS, kind=0, ld=16, bias=BIAS, chosen=CHOSEN,
          weights=WEIGHTS, counts=COUNTS, router=True):
    r = lib.gemm_route_t(experts, top_k, score, groups, top_groups, group_top, True, 1.0)
    return lib.raw_status("gemm_route", tokens, ctypes.byref(r) if router else None, logits, kind, ld, bias, chosen, weights, counts, None)


def backward(tokens=4, experts=16, top_k=2, score=0, groups=1, top_groups=1, group_top=1, logits=LOGITS, kind=0, ld=16, chosen=CHOSEN, dw=DW, dl=DL,
             ldd=16, router=True):
    r = lib.gemm_route_t(experts, top_k, score, groups, top_groups, group_top, True, 1.0)
    return lib.raw_status("gemm_route_backward", tokens, ctypes.byref(r) if router else None, logits, kind, ld, chosen, dw, dl, ldd, None)


@pytest.mark.parametrize("call", [route, backward])
def test_router_refusals(call):
    for bad in ({"tokens": -1}, {"experts": 0}, {"experts": 513, "ld": 513}, {"top_k": 0}, {"top_k": 17}, {"experts": 2, "top_k": 3}, {"groups": 0},
                {"groups": 3}, {"groups": 4, "top_groups": 5}, {"groups": 4, "top_groups": 0}, {"group_top": 0}, {"group_top": 3},
                {"experts": 130, "groups": 65, "ld": 130}, {"groups": 16, "top_groups": 1, "top_k": 2}, {"ld": 15}, {"tokens": 2 ** 31 - 1, "ld": 1 << 20}):
        assert call(**bad) == lib.GEMM_ERR_INVALID_DIM, bad
    assert call(kind=3) == call(kind=-1) == call(score=2) == call(score=-1) == lib.GEMM_ERR_INVALID_TYPE
    assert call(router=False) == call(logits=None) == call(chosen=None) == lib.GEMM_ERR_NULL_PTR
    assert call(logits=at(LOGITS, 2)) == call(kind=1, logits=at(LOGITS, 1)) == call(chosen=at(CHOSEN, 2)) == lib.GEMM_ERR_ALIGNMENT


def test_route_refusals():
    assert route(weights=None) == lib.GEMM_ERR_NULL_PTR
    assert route(weights=at(WEIGHTS, 1)) == route(bias=at(BIAS, 2)) == route(counts=at(COUNTS, 3)) == lib.GEMM_ERR_ALIGNMENT
    # outputs on inputs and on each other: 4 x 16 logits, 4 x 2 choices, 16 counts
    for bad in ({"chosen": LOGITS}, {"weights": at(LOGITS, 4 * 63)}, {"counts": at(LOGITS, 4 * 60)}, {"chosen": BIAS}, {"counts": BIAS},
                {"weights": at(CHOSEN, 28)}, {"counts": at(WEIGHTS, 28)}, {"chosen": at(COUNTS, 60)}):
        assert route(**bad) == lib.GEMM_ERR_ALIAS, bad
    assert route(tokens=0, logits=None, chosen=None, weights=None, counts=None, bias=None) == lib.GEMM_OK


def test_backward_refusals():
    assert backward(ldd=15) == lib.GEMM_ERR_INVALID_DIM
    assert backward(dw=None) == backward(dl=None) == lib.GEMM_ERR_NULL_PTR
    assert backward(dw=at(DW, 2)) == backward(dl=at(DL, 2)) == backward(kind=2, dl=at(DL, 1)) == lib.GEMM_ERR_ALIGNMENT
    for p in (LOGITS, CHOSEN, DW, at(LOGITS, 4 * 63), at(DW, 28)):
        assert backward(dl=p) == lib.GEMM_ERR_ALIAS
    assert backward(tokens=0, logits=None, chosen=None, dw=None, dl=None) == lib.GEMM_OK


def layer(tokens=2, hidden=64, inter=32, experts=4, top_k=2, chosen=CHOSEN, weights=WEIGHTS, x=X, kind=0, ldx=64, w1c=W1C, w1s=W1S, w2c=W2C, w2s=W2S,
          y=Y, ldy=64, ws=WS, wb=1 << 30):
    return lib.raw_status("gemm_mx_moe_routed", tokens, hidden, inter, experts, top_k, chosen, weights, x, kind, ldx, w1c, w1s, w2c, w2s, y, ldy, ws, wb,
                          None)


def test_layer_refusals():
    for bad in ({"tokens": -1}, {"tokens": 65}, {"hidden": 0}, {"inter": 0}, {"experts": 0}, {"experts": 513}, {"top_k": 0}, {"top_k": 5},
                {"experts": 32, "top_k": 17}, {"ldx": 63}, {"ldy": 63}):
        assert layer(**bad) == lib.GEMM_ERR_INVALID_DIM, bad
    assert layer(kind=5) == lib.GEMM_ERR_INVALID_TYPE
    for name in ("chosen", "weights", "x", "w1c", "w1s", "w2c", "w2s", "y"):
        assert layer(**{name: None}) == lib.GEMM_ERR_NULL_PTR, name
    assert layer(chosen=at(CHOSEN, 2)) == layer(weights=at(WEIGHTS, 1)) == layer(w1c=at(W1C, 8)) == lib.GEMM_ERR_ALIGNMENT
    for p in (CHOSEN, WEIGHTS, X, W1C, W1S, W2C, W2S):
        assert layer(y=p) == lib.GEMM_ERR_ALIAS
    need = lib.gemm_mx_moe_workspace_bytes(2, 32, 2, 0)
    assert layer(wb=need - 1) == lib.GEMM_ERR_WORKSPACE
    assert layer(ws=at(WS, 8)) == lib.GEMM_ERR_ALIGNMENT
    for p in (CHOSEN, WEIGHTS, X, W1C, W2S, Y):
        assert layer(ws=p, wb=need) == lib.GEMM_ERR_ALIAS
    assert layer(tokens=0, chosen=None, weights=None, x=None, w1c=None, w1s=None, w2c=None, w2s=None, y=None, ws=None, wb=0) == lib.GEMM_OK


def test_binding_mirrors_the_header():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gemm.h")).read()
    found = re.findall(r"\b(GEMM_ROUTE_\w+)\s*=\s*(\d+)", text)
    assert len(found) == 5
    for name, value in found:
        assert getattr(lib, name) == int(value), name


def test_reference_by_hand():
    l = np.array([[1.0, 3.0, 3.0, 0.0], [0.0, -np.inf, 5.0, -np.inf], [0, np.nan, 1, 2], [-np.inf] * 4])
    c, w, n = ref.route(l, None, ref.Router(4, 2, ref.SOFTMAX, renormalize=True, scale=2.0))
    assert c.tolist() == [[1, 2], [2, 0], [-1, -1], [-1, -1]] and n.tolist() == [1, 1, 2, 0]
    assert w[0].tolist() == [1, 1] and np.allclose(w[1], 2 / (1 + np.exp([-5, 5]))) and np.isnan(w[2]).all() and (w[3] == 0).all()
    # a bias moves the choice, not the weight
    c, w, _ = ref.route(np.zeros((1, 4)), np.array([0, 0.1, 0, 0.2]), ref.Router(4, 2, ref.SIGMOID))
    assert c.tolist() == [[3, 1]] and w.tolist() == [[0.5, 0.5]]
    # the best group by its best expert, and by its two best together
    l = np.log(np.array([[8.0, 1, 6, 5, 7, 1]]) / 28)
    c, _, _ = ref.route(l, None, ref.Router(6, 2, ref.SOFTMAX, 3, 1, 1))
    assert c.tolist() == [[0, 1]]
    c, _, _ = ref.route(l, None, ref.Router(6, 2, ref.SOFTMAX, 3, 1, 2))
    assert c.tolist() == [[2, 3]]


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("renormalize", [False, True])
def test_reference_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(5)
    r = ref.Router(9, 3, score, renormalize=renormalize, scale=1.5)
    l = rng.normal(size=(4, 9)) * 2
    chosen, _, _ = ref.route(l, None, r)
    dw = rng.normal(size=(4, 3))
    d, _ = ref.route_backward(l, chosen, dw, r)
    h = 1e-5
    for t in range(4):
        for e in range(9):
            up, down = l[t].copy(), l[t].copy()
            up[e] += h
            down[e] -= h
            slope = (dw[t] * (ref.weights_of(up, chosen[t], r) - ref.weights_of(down, chosen[t], r))).sum() / (2 * h)
            assert abs(slope - d[t, e]) < 1e-8   # h^2 of the third derivative, and 2^-52 / h
