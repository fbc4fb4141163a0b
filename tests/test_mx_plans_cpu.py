"""gemm_mx_plan without a GPU (256 compute units are assumed there)."""
import ctypes

import pytest

from fp32_gemm_07_amd import binding as lib
from mx_plans import IDS, PLANS, is_plan


@pytest.mark.parametrize("M,N,K,tile,split", PLANS, ids=IDS)
def test_plan(M, N, K, tile, split):
    p = lib.gemm_mx_plan(M, N, K)
    assert is_plan(p, tile, split), p
    KP = -(-K // 128) * 128
    assert p.split_k == -(-KP // p.k_chunk) and (p.k_chunk == KP if p.split_k == 1 else p.k_chunk % 256 == 0)
    assert lib.gemm_mx_workspace_bytes(M, N, K) == (4 * p.split_k * M * N if split else 0) <= 64 << 20


def test_every_kernel_is_among_them():
    kernels = {(tile, split) for _, _, _, tile, split in PLANS}
    tiles = [(64, 64, 4), (128, 128, 4), (128, 128, 2), (256, 128, 2), (256, 256, 2)]
    assert kernels == {(t, s) for t in tiles for s in (False, True)} | {((16, 16, 0), False), ((32, 16, 0), False)}
    for tile, split in kernels:
        if tile[0] > 64 and not split:   # even and odd numbers of 128-value stretches
            assert {-(-K // 128) % 2 for _, _, K, t, s in PLANS if (t, s) == (tile, split)} == {0, 1}, tile


def test_plan_refusals():
    p = lib.gemm_mx_plan_t()
    for bad in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (-1, 4, 4), (4, 4, lib.GEMM_MX_MAX_K + 1), (2 ** 31 - 1, 4, 4096)):
        assert lib.raw_status("gemm_mx_plan", *bad, ctypes.byref(p)) == lib.GEMM_ERR_INVALID_DIM
    assert lib.raw_status("gemm_mx_plan", 4, 4, 4, None) == lib.GEMM_ERR_NULL_PTR
