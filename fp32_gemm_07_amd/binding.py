"""ctypes binding of libgemm (the C ABI in include/gemm.h), same names, marshalling only.

Every entry takes device pointers as Python ints (or anything with a
``data_ptr()`` method, such as a torch tensor on the GPU) and a HIP stream
handle as an int (``torch.cuda.current_stream().cuda_stream``; 0 = null
stream). Nonzero statuses raise ``GemmError``; nothing here computes.

The library must have been built (``fp32_gemm_07_amd.build.build()``): a
missing library raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os

from .build import LIB_PATH

GEMM_OK = 0
GEMM_ERR_INVALID_DIM = 1
GEMM_ERR_NULL_PTR = 2
GEMM_ERR_ALIAS = 3
GEMM_ERR_WORKSPACE = 4
GEMM_ERR_INVALID_PLAN = 5
GEMM_ERR_HIP = 6
GEMM_ERR_UNSUPPORTED_DEVICE = 7
GEMM_ERR_CAPTURING = 8
GEMM_ERR_SCRATCH_LIMIT = 9
GEMM_ERR_INVALID_TYPE = 10
GEMM_ERR_ALIGNMENT = 11

GEMM_TYPE_F32 = 0
GEMM_TYPE_BF16 = 1
GEMM_TYPE_F16 = 2

GEMM_MX_MAX_K = 1 << 24
GEMM_MX_MOE_MAX_TOKENS = 64
GEMM_MX_MOE_MAX_EXPERTS = 512
GEMM_MX_MOE_MAX_TOP_K = 16

GEMM_ROUTE_SOFTMAX = 0
GEMM_ROUTE_SIGMOID = 1
GEMM_ROUTE_MAX_EXPERTS = 512
GEMM_ROUTE_MAX_TOP_K = 16
GEMM_ROUTE_MAX_GROUPS = 64

GEMM_LORA_MAX_ROWS = 1 << 20
GEMM_LORA_MAX_DIM = 1 << 18
GEMM_LORA_MAX_RANK = 128
GEMM_LORA_MAX_ADAPTERS = 1024

GEMM_KERNEL_AUTO = 0
GEMM_KERNEL_MFMA_256x256 = 1
GEMM_KERNEL_MFMA_256x128 = 2
GEMM_KERNEL_MFMA_128x128 = 3
GEMM_KERNEL_MFMA_64x64 = 4
GEMM_KERNEL_MFMA_256x256_W8 = 5
GEMM_KERNEL_VALU_64x64 = 10
GEMM_KERNEL_MFMA16_256x128 = 13
GEMM_KERNEL_MFMA16_128x128 = 14
GEMM_KERNEL_MFMA16_64x64 = 15
GEMM_KERNEL_MFMA16_128x128_K16 = 17
GEMM_KERNEL_MFMA16_256x128_K16 = 18
GEMM_KERNEL_MFMA_128x128_W1 = 19
GEMM_KERNEL_MFMA_64x64_W1 = 21
GEMM_KERNEL_DMA32_256x256_W8 = 30
GEMM_KERNEL_DMA32_128x128_W4 = 33
GEMM_KERNEL_DMA16_128x128_W4 = 34
GEMM_KERNEL_DMA32_256x256_W8_S3 = 35
GEMM_KERNEL_DMA16_64x64 = 36
GEMM_KERNEL_DMA32_64x64 = 37
GEMM_KERNEL_DMA16_128x64 = 38
GEMM_KERNEL_DMA32_128x128_W8 = 39
GEMM_KERNEL_DMA32_64x64_S3 = 45
GEMM_KERNEL_DMA32_128x128_W8_S3 = 46
GEMM_KERNEL_DMA16_96x96_S3 = 47
GEMM_KERNEL_LADDER_V0 = 40
GEMM_KERNEL_LADDER_V1 = 41
GEMM_KERNEL_LADDER_V2 = 42
GEMM_KERNEL_LADDER_V3 = 43

KERNELS = {
    "mfma32_256x256": GEMM_KERNEL_MFMA_256x256,
    "mfma32_256x256_w8": GEMM_KERNEL_MFMA_256x256_W8,
    "mfma32_256x128": GEMM_KERNEL_MFMA_256x128,
    "mfma32_128x128": GEMM_KERNEL_MFMA_128x128,
    "mfma32_64x64": GEMM_KERNEL_MFMA_64x64,
    "mfma16_256x128": GEMM_KERNEL_MFMA16_256x128,
    "mfma16_128x128": GEMM_KERNEL_MFMA16_128x128,
    "mfma16_64x64": GEMM_KERNEL_MFMA16_64x64,
    "mfma16_128x128_k16": GEMM_KERNEL_MFMA16_128x128_K16,
    "mfma16_256x128_k16": GEMM_KERNEL_MFMA16_256x128_K16,
    "mfma32_128x128_w1": GEMM_KERNEL_MFMA_128x128_W1,
    "mfma32_64x64_w1": GEMM_KERNEL_MFMA_64x64_W1,
    "dma32_256x256_w8": GEMM_KERNEL_DMA32_256x256_W8,
    "dma32_128x128_w4": GEMM_KERNEL_DMA32_128x128_W4,
    "dma16_128x128_w4": GEMM_KERNEL_DMA16_128x128_W4,
    "dma32_256x256_w8_s3": GEMM_KERNEL_DMA32_256x256_W8_S3,
    "dma16_64x64": GEMM_KERNEL_DMA16_64x64,
    "dma32_64x64": GEMM_KERNEL_DMA32_64x64,
    "dma16_128x64": GEMM_KERNEL_DMA16_128x64,
    "dma32_128x128_w8": GEMM_KERNEL_DMA32_128x128_W8,
    "dma32_64x64_s3": GEMM_KERNEL_DMA32_64x64_S3,
    "dma32_128x128_w8_s3": GEMM_KERNEL_DMA32_128x128_W8_S3,
    "dma16_96x96_s3": GEMM_KERNEL_DMA16_96x96_S3,
    "valu_64x64": GEMM_KERNEL_VALU_64x64,
    "ladder_v0": GEMM_KERNEL_LADDER_V0,
    "ladder_v1": GEMM_KERNEL_LADDER_V1,
    "ladder_v2": GEMM_KERNEL_LADDER_V2,
    "ladder_v3": GEMM_KERNEL_LADDER_V3,
}

# Every symbol include/gemm.h declares.
EXPORTS = (
    "gemm_f32", "gemm_f32_noalloc", "gemm_f32_noalloc_scratch_bytes", "gemm_f32_workspace_bytes",
    "gemm_f32_ex", "gemm_f32_plan", "gemm_f32_plan_cus",
    "gemm_f32_plan_workspace_bytes", "gemm_f32_with_plan", "gemm_f32_general",
    "gemm_f32_general_workspace_bytes", "gemm_mx_codes_bytes", "gemm_mx_scales_bytes",
    "gemm_mx_quantize", "gemm_mx_dequantize", "gemm_mx", "gemm_mx_workspace_bytes", "gemm_mx_plan",
    "gemm_mx_moe", "gemm_mx_moe_workspace_bytes", "gemm_mx_moe_routed", "gemm_route",
    "gemm_route_backward", "gemm_lora", "gemm_lora_workspace_bytes", "gemm_lora_backward",
    "gemm_lora_backward_workspace_bytes", "gemm_kernel_name", "gemm_status_string",
    "gemm_last_hip_error",
)


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        text = gemm_status_string(status)
        if status == GEMM_ERR_HIP:
            text += f" (hipError_t {gemm_last_hip_error()})"
        super().__init__(f"{where}: {text} [status {status}]")


class gemm_plan_t(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("split_k", ctypes.c_int),
                ("k_chunk", ctypes.c_int), ("split_tail", ctypes.c_int)]

    def __repr__(self):
        return (f"gemm_plan_t(kernel={gemm_kernel_name(self.kernel)}, split_k={self.split_k}, "
                f"k_chunk={self.k_chunk}, split_tail={self.split_tail})")


class gemm_mx_plan_t(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int), ("stages", ctypes.c_int),
                ("split_k", ctypes.c_int), ("k_chunk", ctypes.c_int)]

    def __repr__(self):
        return (f"gemm_mx_plan_t(tile_m={self.tile_m}, tile_n={self.tile_n}, stages={self.stages}, "
                f"split_k={self.split_k}, k_chunk={self.k_chunk})")


class gemm_route_t(ctypes.Structure):
    """A router: how many experts, how many of them a token chooses, and how."""
    _fields_ = [("experts", ctypes.c_int), ("top_k", ctypes.c_int), ("score", ctypes.c_int),
                ("groups", ctypes.c_int), ("top_groups", ctypes.c_int), ("group_top", ctypes.c_int),
                ("renormalize", ctypes.c_int), ("scale", ctypes.c_float)]

    def __init__(self, experts: int, top_k: int, score: int = GEMM_ROUTE_SOFTMAX, groups: int = 1,
                 top_groups: int = 1, group_top: int = 1, renormalize: bool = False,
                 scale: float = 1.0):
        super().__init__(experts, top_k, score, groups, top_groups, group_top,
                         int(bool(renormalize)), scale)

    def __repr__(self):
        return (f"gemm_route_t(experts={self.experts}, top_k={self.top_k}, score={self.score}, "
                f"groups={self.groups}, top_groups={self.top_groups}, group_top={self.group_top}, "
                f"renormalize={self.renormalize}, scale={self.scale})")


class gemm_lora_t(ctypes.Structure):
    """A set of low-rank adapters. Device pointers as everywhere (tensors or ints); the set
    keeps no tensor alive."""
    _fields_ = [("type", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("rank", ctypes.c_int), ("adapters", ctypes.c_int), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p)]

    def __init__(self, type: int, N: int, K: int, rank: int, adapters: int, A, B, ranks=None,
                 scales=None):
        super().__init__(type, N, K, rank, adapters, _addr(A) or None, _addr(B) or None,
                         _addr(ranks) or None, _addr(scales) or None)

    def __repr__(self):
        return (f"gemm_lora_t(type={self.type}, N={self.N}, K={self.K}, rank={self.rank}, "
                f"adapters={self.adapters})")


_lib = None


def _share_hip_runtime() -> None:
    """Make libgemm use the HIP runtime the caller's memory and streams come from.

    PyTorch-ROCm wheels bundle their own libamdhip64 (and HSA runtime) under
    the soname libamdhip64.so.7. A process that ends up with two HIP runtimes
    cannot use the GPU from the second one (device enumeration fails), and
    pointers and streams of one are meaningless to the other. libgemm names
    its runtime only by soname, and the dynamic linker resolves a soname to a
    library already loaded under it, so loading torch first makes libgemm
    bind to torch's runtime. Without torch installed, the system ROCm runtime
    is used.
    """
    try:
        import torch  # noqa: F401
    except ImportError:
        pass


def library_path() -> str:
    return LIB_PATH


def load():
    """Load libgemm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libgemm is not built ({LIB_PATH} missing); run "
                               "fp32_gemm_07_amd.build.build() first")
        _share_hip_runtime()
        lib = ctypes.CDLL(LIB_PATH)
        vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        plan_p = ctypes.POINTER(gemm_plan_t)
        lib.gemm_f32.argtypes = [vp, vp, vp, i, i, i, vp]
        lib.gemm_f32.restype = i
        lib.gemm_f32_noalloc.argtypes = [vp, vp, vp, i, i, i, vp]
        lib.gemm_f32_noalloc.restype = i
        lib.gemm_f32_noalloc_scratch_bytes.argtypes = []
        lib.gemm_f32_noalloc_scratch_bytes.restype = sz
        lib.gemm_f32_workspace_bytes.argtypes = [i, i, i]
        lib.gemm_f32_workspace_bytes.restype = sz
        lib.gemm_f32_ex.argtypes = [vp, vp, vp, i, i, i, vp, sz, vp]
        lib.gemm_f32_ex.restype = i
        lib.gemm_f32_plan.argtypes = [i, i, i, plan_p]
        lib.gemm_f32_plan.restype = i
        lib.gemm_f32_plan_cus.argtypes = [i, i, i, i, plan_p]
        lib.gemm_f32_plan_cus.restype = i
        lib.gemm_f32_plan_workspace_bytes.argtypes = [i, i, i, plan_p]
        lib.gemm_f32_plan_workspace_bytes.restype = sz
        lib.gemm_f32_with_plan.argtypes = [vp, vp, vp, i, i, i, plan_p, vp, sz, vp]
        lib.gemm_f32_with_plan.restype = i
        f = ctypes.c_float
        lib.gemm_f32_general.argtypes = [i, i, i, i, i, f, vp, i, vp, i, f, vp, i, vp, sz, vp]
        lib.gemm_f32_general.restype = i
        lib.gemm_f32_general_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
        lib.gemm_f32_general_workspace_bytes.restype = sz
        lib.gemm_mx_codes_bytes.argtypes = [i, i]
        lib.gemm_mx_codes_bytes.restype = sz
        lib.gemm_mx_scales_bytes.argtypes = [i, i]
        lib.gemm_mx_scales_bytes.restype = sz
        lib.gemm_mx_quantize.argtypes = [i, i, i, vp, i, i, vp, vp, vp]
        lib.gemm_mx_quantize.restype = i
        lib.gemm_mx_dequantize.argtypes = [i, i, i, vp, vp, vp, i, i, vp]
        lib.gemm_mx_dequantize.restype = i
        lib.gemm_mx.argtypes = [i, i, i, f, vp, vp, vp, vp, f, vp, i, i, vp, sz, vp]
        lib.gemm_mx.restype = i
        lib.gemm_mx_workspace_bytes.argtypes = [i, i, i]
        lib.gemm_mx_workspace_bytes.restype = sz
        lib.gemm_mx_plan.argtypes = [i, i, i, ctypes.POINTER(gemm_mx_plan_t)]
        lib.gemm_mx_plan.restype = i
        lib.gemm_mx_moe.argtypes = [i, i, i, i, i, i, vp, i, vp, i, i, vp, vp, vp, vp, vp, i, vp,
                                    sz, vp]
        lib.gemm_mx_moe.restype = i
        lib.gemm_mx_moe_workspace_bytes.argtypes = [i, i, i, i]
        lib.gemm_mx_moe_workspace_bytes.restype = sz
        lib.gemm_mx_moe_routed.argtypes = [i, i, i, i, i, vp, vp, vp, i, i, vp, vp, vp, vp, vp, i,
                                           vp, sz, vp]
        lib.gemm_mx_moe_routed.restype = i
        route_p = ctypes.POINTER(gemm_route_t)
        lib.gemm_route.argtypes = [i, route_p, vp, i, i, vp, vp, vp, vp, vp]
        lib.gemm_route.restype = i
        lib.gemm_route_backward.argtypes = [i, route_p, vp, i, i, vp, vp, vp, i, vp]
        lib.gemm_route_backward.restype = i
        lora_p = ctypes.POINTER(gemm_lora_t)
        lib.gemm_lora.argtypes = [i, lora_p, vp, vp, i, vp, i, vp, i, vp, sz, vp]
        lib.gemm_lora.restype = i
        lib.gemm_lora_workspace_bytes.argtypes = [i, lora_p]
        lib.gemm_lora_workspace_bytes.restype = sz
        lib.gemm_lora_backward.argtypes = [i, lora_p, vp, vp, i, vp, i, vp, i, vp, i, vp, vp, vp, sz,
                                           vp]
        lib.gemm_lora_backward.restype = i
        lib.gemm_lora_backward_workspace_bytes.argtypes = [i, lora_p]
        lib.gemm_lora_backward_workspace_bytes.restype = sz
        lib.gemm_kernel_name.argtypes = [i]
        lib.gemm_kernel_name.restype = ctypes.c_char_p
        lib.gemm_status_string.argtypes = [i]
        lib.gemm_status_string.restype = ctypes.c_char_p
        lib.gemm_last_hip_error.argtypes = []
        lib.gemm_last_hip_error.restype = i
        _lib = lib
    return _lib


def _addr(p) -> int:
    if p is None:
        return 0
    if hasattr(p, "data_ptr"):
        return int(p.data_ptr())
    return int(p)


def _check(status: int, where: str) -> int:
    if status != GEMM_OK:
        raise GemmError(status, where)
    return status


def gemm_f32(A, B, C, M: int, N: int, K: int, stream: int = 0) -> None:
    _check(load().gemm_f32(_addr(A), _addr(B), _addr(C), M, N, K, stream or None), "gemm_f32")


def gemm_f32_noalloc(A, B, C, M: int, N: int, K: int, stream: int = 0) -> None:
    _check(load().gemm_f32_noalloc(_addr(A), _addr(B), _addr(C), M, N, K, stream or None),
           "gemm_f32_noalloc")


def gemm_f32_noalloc_scratch_bytes() -> int:
    return int(load().gemm_f32_noalloc_scratch_bytes())


def gemm_f32_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().gemm_f32_workspace_bytes(M, N, K))


def gemm_f32_ex(A, B, C, M: int, N: int, K: int, workspace, workspace_bytes: int,
                stream: int = 0) -> None:
    _check(load().gemm_f32_ex(_addr(A), _addr(B), _addr(C), M, N, K, _addr(workspace) or None,
                              workspace_bytes, stream or None), "gemm_f32_ex")


def gemm_f32_plan(M: int, N: int, K: int) -> gemm_plan_t:
    p = gemm_plan_t()
    _check(load().gemm_f32_plan(M, N, K, ctypes.byref(p)), "gemm_f32_plan")
    return p


def gemm_f32_plan_cus(M: int, N: int, K: int, num_cus: int) -> gemm_plan_t:
    p = gemm_plan_t()
    _check(load().gemm_f32_plan_cus(M, N, K, num_cus, ctypes.byref(p)), "gemm_f32_plan_cus")
    return p


def make_plan(kernel: int, split_k: int = 1, split_tail: bool = False) -> gemm_plan_t:
    """An explicit plan; split_tail splits only the tiles of the last, partial
    round of one tile per CU (copy-fed kernels only)."""
    return gemm_plan_t(kernel, split_k, 0, int(split_tail))


def gemm_f32_plan_workspace_bytes(M: int, N: int, K: int, plan: gemm_plan_t) -> int:
    return int(load().gemm_f32_plan_workspace_bytes(M, N, K, ctypes.byref(plan)))


def gemm_f32_with_plan(A, B, C, M: int, N: int, K: int, plan: gemm_plan_t, workspace=None,
                       workspace_bytes: int = 0, stream: int = 0) -> None:
    _check(load().gemm_f32_with_plan(_addr(A), _addr(B), _addr(C), M, N, K, ctypes.byref(plan),
                                     _addr(workspace) or None, workspace_bytes, stream or None),
           "gemm_f32_with_plan")


def gemm_f32_general(trans_a: bool, trans_b: bool, M: int, N: int, K: int, alpha: float, A,
                     lda: int, B, ldb: int, beta: float, C, ldc: int, workspace=None,
                     workspace_bytes: int = 0, stream: int = 0) -> None:
    _check(load().gemm_f32_general(int(bool(trans_a)), int(bool(trans_b)), M, N, K, alpha,
                                   _addr(A) or None, lda, _addr(B) or None, ldb, beta,
                                   _addr(C) or None, ldc, _addr(workspace) or None,
                                   workspace_bytes, stream or None), "gemm_f32_general")


def gemm_f32_general_workspace_bytes(trans_a: bool, trans_b: bool, M: int, N: int, K: int,
                                     lda: int, ldb: int) -> int:
    return int(load().gemm_f32_general_workspace_bytes(int(bool(trans_a)), int(bool(trans_b)),
                                                       M, N, K, lda, ldb))


def gemm_mx_codes_bytes(rows: int, K: int) -> int:
    return int(load().gemm_mx_codes_bytes(rows, K))


def gemm_mx_scales_bytes(rows: int, K: int) -> int:
    return int(load().gemm_mx_scales_bytes(rows, K))


def gemm_mx_quantize(trans: bool, rows: int, K: int, X, x_type: int, ldx: int, codes, scales,
                     stream: int = 0) -> None:
    _check(load().gemm_mx_quantize(int(bool(trans)), rows, K, _addr(X) or None, x_type, ldx,
                                   _addr(codes) or None, _addr(scales) or None, stream or None),
           "gemm_mx_quantize")


def gemm_mx_dequantize(trans: bool, rows: int, K: int, codes, scales, Y, y_type: int, ldy: int,
                       stream: int = 0) -> None:
    _check(load().gemm_mx_dequantize(int(bool(trans)), rows, K, _addr(codes) or None,
                                     _addr(scales) or None, _addr(Y) or None, y_type, ldy,
                                     stream or None), "gemm_mx_dequantize")


def gemm_mx(M: int, N: int, K: int, alpha: float, A_codes, A_scales, B_codes, B_scales,
            beta: float, C, c_type: int, ldc: int, workspace=None, workspace_bytes: int = 0,
            stream: int = 0) -> None:
    _check(load().gemm_mx(M, N, K, alpha, _addr(A_codes) or None, _addr(A_scales) or None,
                          _addr(B_codes) or None, _addr(B_scales) or None, beta, _addr(C) or None,
                          c_type, ldc, _addr(workspace) or None, workspace_bytes, stream or None),
           "gemm_mx")


def gemm_mx_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().gemm_mx_workspace_bytes(M, N, K))


def gemm_mx_plan(M: int, N: int, K: int) -> gemm_mx_plan_t:
    p = gemm_mx_plan_t()
    _check(load().gemm_mx_plan(M, N, K, ctypes.byref(p)), "gemm_mx_plan")
    return p


def gemm_mx_moe(tokens: int, hidden: int, inter: int, experts: int, top_k: int, renormalize: bool,
                logits, ld_logits: int, X, x_type: int, ldx: int, W1_codes, W1_scales, W2_codes,
                W2_scales, Y, ldy: int, workspace=None, workspace_bytes: int = 0,
                stream: int = 0) -> None:
    _check(load().gemm_mx_moe(tokens, hidden, inter, experts, top_k, int(bool(renormalize)),
                              _addr(logits) or None, ld_logits, _addr(X) or None, x_type, ldx,
                              _addr(W1_codes) or None, _addr(W1_scales) or None,
                              _addr(W2_codes) or None, _addr(W2_scales) or None, _addr(Y) or None,
                              ldy, _addr(workspace) or None, workspace_bytes, stream or None),
           "gemm_mx_moe")


def gemm_mx_moe_workspace_bytes(tokens: int, inter: int, top_k: int, x_type: int) -> int:
    return int(load().gemm_mx_moe_workspace_bytes(tokens, inter, top_k, x_type))


def gemm_mx_moe_routed(tokens: int, hidden: int, inter: int, experts: int, top_k: int, chosen,
                       weights, X, x_type: int, ldx: int, W1_codes, W1_scales, W2_codes, W2_scales,
                       Y, ldy: int, workspace=None, workspace_bytes: int = 0,
                       stream: int = 0) -> None:
    _check(load().gemm_mx_moe_routed(tokens, hidden, inter, experts, top_k, _addr(chosen) or None,
                                     _addr(weights) or None, _addr(X) or None, x_type, ldx,
                                     _addr(W1_codes) or None, _addr(W1_scales) or None,
                                     _addr(W2_codes) or None, _addr(W2_scales) or None,
                                     _addr(Y) or None, ldy, _addr(workspace) or None,
                                     workspace_bytes, stream or None), "gemm_mx_moe_routed")


def gemm_route(tokens: int, router: gemm_route_t, logits, logits_type: int, ld_logits: int, bias,
               chosen, weights, counts=None, stream: int = 0) -> None:
    _check(load().gemm_route(tokens, ctypes.byref(router), _addr(logits) or None, logits_type,
                             ld_logits, _addr(bias) or None, _addr(chosen) or None,
                             _addr(weights) or None, _addr(counts) or None, stream or None),
           "gemm_route")


def gemm_route_backward(tokens: int, router: gemm_route_t, logits, logits_type: int,
                        ld_logits: int, chosen, dweights, dlogits, ld_dlogits: int,
                        stream: int = 0) -> None:
    _check(load().gemm_route_backward(tokens, ctypes.byref(router), _addr(logits) or None,
                                      logits_type, ld_logits, _addr(chosen) or None,
                                      _addr(dweights) or None, _addr(dlogits) or None, ld_dlogits,
                                      stream or None), "gemm_route_backward")


def gemm_lora(rows: int, set: gemm_lora_t, ids, X, ldx: int, C, ldc: int, Y, ldy: int,
              workspace=None, workspace_bytes: int = 0, stream: int = 0) -> None:
    _check(load().gemm_lora(rows, ctypes.byref(set), _addr(ids) or None, _addr(X) or None, ldx,
                            _addr(C) or None, ldc, _addr(Y) or None, ldy, _addr(workspace) or None,
                            workspace_bytes, stream or None), "gemm_lora")


def gemm_lora_workspace_bytes(rows: int, set: gemm_lora_t) -> int:
    return int(load().gemm_lora_workspace_bytes(rows, ctypes.byref(set)))


def gemm_lora_backward(rows: int, set: gemm_lora_t, ids, X, ldx: int, dY, lddy: int, C, ldc: int,
                       dX, lddx: int, dA, dB, workspace=None, workspace_bytes: int = 0,
                       stream: int = 0) -> None:
    _check(load().gemm_lora_backward(rows, ctypes.byref(set), _addr(ids) or None, _addr(X) or None,
                                     ldx, _addr(dY) or None, lddy, _addr(C) or None, ldc,
                                     _addr(dX) or None, lddx, _addr(dA) or None, _addr(dB) or None,
                                     _addr(workspace) or None, workspace_bytes, stream or None),
           "gemm_lora_backward")


def gemm_lora_backward_workspace_bytes(rows: int, set: gemm_lora_t) -> int:
    return int(load().gemm_lora_backward_workspace_bytes(rows, ctypes.byref(set)))


def gemm_kernel_name(kernel: int) -> str:
    return load().gemm_kernel_name(kernel).decode()


def gemm_status_string(status: int) -> str:
    return load().gemm_status_string(status).decode()


def gemm_last_hip_error() -> int:
    return int(load().gemm_last_hip_error())


def raw_status(fn: str, *args) -> int:
    """Call an entry point and return its raw status (for tests of the error paths)."""
    return int(getattr(load(), fn)(*args))
