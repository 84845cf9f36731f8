"""Binding of libmosaic: ctypes for include/mosaic.h, and a small extension module for the
operators of include/mosaic_ops.h (csrc/marshal.cpp: their calls are short enough for the
host's side of a call to show).

Argument marshalling only: every step of the path runs in the CUDA library. PyTorch
provides device memory and the current stream. There is no CPU fallback: a missing
library or a non-CUDA tensor raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import build

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmosaic.so")
_lib = None

MQ_OK = 0
MQ_GEMM_AUTO = 0
MQ_GEMM_DECODE = 1
MQ_GEMM_PREFILL = 2
MQ_GEMM_BASE_ONLY = 4
MQ_GEMM_RESIDUAL_ONLY = 8
MQ_LAYER_PREPARED = 16
MQ_GEMM_WEIGHTS_READY = 32

EXPORTED = (
    "mq_sf_swz_bytes", "mq_budget_blocks", "mq_quantize_weight_workspace_bytes", "mq_delta_topk_workspace_bytes",
    "mq_gemm_workspace_bytes", "mq_quantize_weight", "mq_hessian_diag", "mq_delta_score_topk", "mq_pack_residual",
    "mq_quantize_act", "mq_gemm", "mq_run_layer", "mq_get_error", "mq_status_string", "mq_launch_count",
    "mq_gemm_noalloc", "mq_gemm_noalloc_scratch_limit", "mq_quantize_weight_delta", "mq_topk_blocks",
    "mq_pack_residual_weight", "mq_gemm_act", "mq_weight_bytes", "mq_fp4_mma_loop", "mq_fp4_mma_loop_flops",
    "mq_test_arm_wait_fault", "mq_smooth_scales", "mq_smooth_apply", "mq_timeline_read",
    "mq_kv_cache_bytes", "mq_gemv", "mq_gemv_workspace_bytes", "mq_qk_norm_rope", "mq_kv_append", "mq_qkv_append", "mq_kv_read",
    "mq_kv_attention_workspace_bytes", "mq_kv_attention",
)

MQ_BF16 = 0
MQ_F16 = 1
GEMV_MAX_TOKENS = 16


class MosaicError(RuntimeError):
    pass


class NVFP4Mat(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("codes", ctypes.c_void_p), ("sf", ctypes.c_void_p),
                ("sf_swz", ctypes.c_void_p), ("gscale", ctypes.c_void_p)]


class ResidualPacked(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("K", ctypes.c_int), ("nblk", ctypes.c_int), ("blk_codes", ctypes.c_void_p),
                ("blk_sf", ctypes.c_void_p), ("blk_kt", ctypes.c_void_p), ("tile_ptr", ctypes.c_void_p),
                ("bitmap", ctypes.c_void_p)]


class LayerBuffers(ctypes.Structure):
    _fields_ = [("base", NVFP4Mat), ("resid_full", NVFP4Mat), ("xq", NVFP4Mat), ("H", ctypes.c_void_p),
                ("delta", ctypes.c_void_p), ("rank", ctypes.c_void_p), ("sel", ctypes.c_void_p),
                ("packed", ResidualPacked), ("ws_quant", ctypes.c_void_p), ("ws_quant_bytes", ctypes.c_size_t),
                ("ws_gemm", ctypes.c_void_p), ("ws_gemm_bytes", ctypes.c_size_t), ("W_dev", ctypes.c_void_p),
                ("X_dev", ctypes.c_void_p), ("Xcal_dev", ctypes.c_void_p), ("Y_dev", ctypes.c_void_p)]


class KVCacheStruct(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("D", ctypes.c_int), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


def lib():
    """Load libmosaic.so (built by ``__graft_entry__.build()`` or ``build.py``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise MosaicError(f"libmosaic.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    P = ctypes.POINTER
    L.mq_sf_swz_bytes.argtypes = [i32, i32]
    L.mq_sf_swz_bytes.restype = sz
    L.mq_weight_bytes.argtypes = [i32, i32]
    L.mq_weight_bytes.restype = sz
    L.mq_fp4_mma_loop.argtypes = [i32, i32, vp]
    L.mq_fp4_mma_loop.restype = i32
    L.mq_fp4_mma_loop_flops.argtypes = [i32, i32]
    L.mq_fp4_mma_loop_flops.restype = ctypes.c_double
    L.mq_timeline_read.argtypes = [vp, ctypes.c_size_t]
    L.mq_timeline_read.restype = i32
    L.mq_test_arm_wait_fault.argtypes = [i32, ctypes.c_double]
    L.mq_test_arm_wait_fault.restype = i32
    L.mq_smooth_scales.argtypes = [vp, i32, vp, i32, i32, vp, vp]
    L.mq_smooth_scales.restype = i32
    L.mq_smooth_apply.argtypes = [vp, i32, i32, vp, i32, vp, vp]
    L.mq_smooth_apply.restype = i32
    L.mq_budget_blocks.argtypes = [i32, i32, ctypes.c_double]
    L.mq_budget_blocks.restype = i32
    L.mq_quantize_weight_workspace_bytes.argtypes = [i32, i32]
    L.mq_quantize_weight_workspace_bytes.restype = sz
    L.mq_delta_topk_workspace_bytes.argtypes = [i32, i32, i32]
    L.mq_delta_topk_workspace_bytes.restype = sz
    L.mq_gemm_workspace_bytes.argtypes = [i32, i32, i32, ctypes.c_uint]
    L.mq_gemm_workspace_bytes.restype = sz
    L.mq_quantize_weight.argtypes = [vp, i32, i32, P(NVFP4Mat), P(NVFP4Mat), vp, sz, vp]
    L.mq_hessian_diag.argtypes = [vp, i32, i32, vp, vp]
    L.mq_delta_score_topk.argtypes = [vp, vp, P(NVFP4Mat), P(NVFP4Mat), i32, vp, vp, vp, vp, sz, vp]
    L.mq_pack_residual.argtypes = [P(NVFP4Mat), vp, i32, P(ResidualPacked), vp]
    L.mq_quantize_act.argtypes = [vp, i32, i32, P(NVFP4Mat), vp]
    L.mq_gemm.argtypes = [P(NVFP4Mat), P(NVFP4Mat), P(ResidualPacked), vp, i32, i32, i32, ctypes.c_uint, vp, sz, vp]
    for f in ("mq_quantize_weight", "mq_hessian_diag", "mq_delta_score_topk", "mq_pack_residual", "mq_quantize_act",
              "mq_gemm", "mq_get_error"):
        getattr(L, f).restype = i32
    L.mq_run_layer.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, ctypes.c_uint, i32, P(LayerBuffers), vp]
    L.mq_run_layer.restype = i32
    L.mq_gemm_noalloc.argtypes = [P(NVFP4Mat), P(NVFP4Mat), P(ResidualPacked), vp, i32, i32, i32, ctypes.c_uint, vp]
    L.mq_gemm_noalloc.restype = i32
    L.mq_gemm_noalloc_scratch_limit.argtypes = []
    L.mq_gemm_noalloc_scratch_limit.restype = sz
    L.mq_quantize_weight_delta.argtypes = [vp, i32, i32, vp, P(NVFP4Mat), P(NVFP4Mat), vp, vp, sz, vp]
    L.mq_quantize_weight_delta.restype = i32
    L.mq_topk_blocks.argtypes = [vp, i32, i32, vp, vp, vp]
    L.mq_topk_blocks.restype = i32
    L.mq_pack_residual_weight.argtypes = [vp, P(NVFP4Mat), vp, i32, P(ResidualPacked), vp]
    L.mq_pack_residual_weight.restype = i32
    L.mq_gemm_act.argtypes = [vp, P(NVFP4Mat), P(ResidualPacked), vp, i32, i32, i32, ctypes.c_uint, vp, sz, vp, vp]
    L.mq_gemm_act.restype = i32
    L.mq_get_error.argtypes = [vp]
    L.mq_status_string.argtypes = [i32]
    L.mq_status_string.restype = ctypes.c_char_p
    L.mq_launch_count.argtypes = []
    L.mq_launch_count.restype = ctypes.c_uint64
    i64, u32, f32 = ctypes.c_int64, ctypes.c_uint, ctypes.c_float
    L.mq_kv_cache_bytes.argtypes = [i32] * 4
    L.mq_kv_cache_bytes.restype = sz
    L.mq_kv_attention_workspace_bytes.argtypes = [i32] * 4
    L.mq_kv_attention_workspace_bytes.restype = sz
    L.mq_gemv.argtypes = [vp, i32, i64, vp, vp, vp, i64, i32, i32, i32, u32, vp, sz, vp]
    L.mq_gemv_workspace_bytes.argtypes = [i32, i32]
    L.mq_gemv_workspace_bytes.restype = sz
    L.mq_qk_norm_rope.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, f32, vp, vp, i32, i32, vp]
    L.mq_kv_append.argtypes = [vp, vp, i32, i32, vp, vp, vp]
    L.mq_qkv_append.argtypes = [vp, vp, vp, vp, vp, i32, i32, vp, vp, f32, vp, vp, i32, i32, vp, vp, vp]
    L.mq_kv_read.argtypes = [vp, vp, i32, vp, vp, i32, vp]
    L.mq_kv_attention.argtypes = [vp, vp, vp, i32, i32, vp, vp, i64, i32, i32, vp, i32, vp, f32, i32, vp, sz, vp]
    for f in ("mq_gemv", "mq_qk_norm_rope", "mq_kv_append", "mq_qkv_append", "mq_kv_read", "mq_kv_attention"):
        getattr(L, f).restype = i32
    _lib = L
    return L


def _check(status: int, what: str):
    if status != MQ_OK:
        raise MosaicError(f"{what}: {lib().mq_status_string(status).decode()} (status {status})")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise MosaicError("libmosaic takes CUDA tensors only")
    return t.data_ptr()


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _u8(*shape, device):
    return torch.empty(shape, dtype=torch.uint8, device=device)


def mat(d: dict) -> NVFP4Mat:
    return NVFP4Mat(d["rows"], d["cols"], _ptr(d.get("codes")), _ptr(d.get("sf")), _ptr(d.get("sf_swz")),
                    _ptr(d.get("gscale")))


def packed_struct(p: dict | None) -> ResidualPacked | None:
    if p is None:
        return None
    return ResidualPacked(p["N"], p["K"], p["nblk"], _ptr(p.get("blk_codes")), _ptr(p.get("blk_sf")),
                          _ptr(p.get("blk_kt")), _ptr(p.get("tile_ptr")), _ptr(p.get("bitmap")))


# ------------------------------------------------------------------ allocation helpers
def alloc_weight(N: int, K: int, device, with_sf: bool = True) -> tuple[dict, dict]:
    """Base (GEMM-ready NVFP4 weight) and full-residual buffers of an N x K weight.

    The base's codes, tiled scales and tensor scale are views of ONE allocation of
    mq_weight_bytes(N, K) bytes at the offsets include/mosaic.h states; its optional
    linear scales and the residual are separate tensors."""
    L = lib()
    nbytes = L.mq_weight_bytes(N, K)
    if nbytes == 0:
        raise MosaicError(f"bad weight shape {N} x {K}")
    blob = _u8(nbytes, device=device)
    nc, ns = N * (K // 2), L.mq_sf_swz_bytes(N, K)
    base = {"rows": N, "cols": K, "codes": blob[:nc].view(N, K // 2),
            "sf": _u8(N, K // 16, device=device) if with_sf else None,
            "sf_swz": blob[nc:nc + ns],
            "gscale": blob[nc + ns:nc + ns + 4].view(torch.float32), "blob": blob}
    resid = {"rows": N, "cols": K, "codes": _u8(N, K // 2, device=device), "sf": _u8(N, K // 16, device=device),
             "sf_swz": None, "gscale": None}
    return base, resid


def alloc_act(M: int, K: int, device, with_sf: bool = False) -> dict:
    L = lib()
    return {"rows": M, "cols": K, "codes": _u8(M, K // 2, device=device),
            "sf": _u8(M, K // 16, device=device) if with_sf else None,
            "sf_swz": _u8(L.mq_sf_swz_bytes(M, K), device=device),
            "gscale": torch.empty(M, dtype=torch.float32, device=device)}


def alloc_packed(N: int, K: int, budget: int, device) -> dict:
    KB = K // 64
    KW = (KB + 31) // 32
    nb = max(budget, 1)
    return {"N": N, "K": K, "nblk": budget, "blk_codes": _u8(nb, 2048, device=device),
            "blk_sf": _u8(nb, 512, device=device), "blk_kt": torch.empty(nb, dtype=torch.int32, device=device),
            "tile_ptr": torch.empty(N // 64 + 1, dtype=torch.int32, device=device),
            "bitmap": torch.empty((N // 64, KW), dtype=torch.int32, device=device)}


# ------------------------------------------------------------------ the path (C names)
def mq_smooth_scales(Xcal: torch.Tensor, W: torch.Tensor, s: torch.Tensor, stream=None):
    T, K = Xcal.shape
    N = W.shape[0]
    _check(lib().mq_smooth_scales(_ptr(Xcal), T, _ptr(W), N, K, _ptr(s), _stream(stream)), "mq_smooth_scales")


def mq_smooth_apply(A: torch.Tensor, s: torch.Tensor, invert: bool, out: torch.Tensor, stream=None):
    rows, K = A.shape
    _check(lib().mq_smooth_apply(_ptr(A), rows, K, _ptr(s), 1 if invert else 0, _ptr(out), _stream(stream)),
           "mq_smooth_apply")


def mq_quantize_weight(W: torch.Tensor, base: dict, resid: dict, ws: torch.Tensor, stream=None):
    N, K = W.shape
    _check(lib().mq_quantize_weight(_ptr(W), N, K, ctypes.byref(mat(base)), ctypes.byref(mat(resid)), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)), "mq_quantize_weight")


def mq_quantize_weight_delta(W: torch.Tensor, H: torch.Tensor, base: dict, resid: dict | None, delta: torch.Tensor,
                             ws: torch.Tensor, stream=None):
    """resid None: the full residual is not stored (see mq_pack_residual_weight)."""
    N, K = W.shape
    r = None if resid is None else ctypes.byref(mat(resid))
    _check(lib().mq_quantize_weight_delta(_ptr(W), N, K, _ptr(H), ctypes.byref(mat(base)), r,
                                          _ptr(delta), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "mq_quantize_weight_delta")


def mq_topk_blocks(delta: torch.Tensor, budget: int, rank, sel, stream=None):
    _check(lib().mq_topk_blocks(_ptr(delta), delta.numel(), budget, _ptr(rank), _ptr(sel), _stream(stream)),
           "mq_topk_blocks")


def mq_hessian_diag(Xcal: torch.Tensor, H: torch.Tensor, stream=None):
    T, K = Xcal.shape
    _check(lib().mq_hessian_diag(_ptr(Xcal), T, K, _ptr(H), _stream(stream)), "mq_hessian_diag")


def mq_delta_score_topk(W, H, base: dict, resid: dict | None, budget: int, delta, rank, sel, ws=None, stream=None):
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    rs = None if resid is None else ctypes.byref(mat(resid))
    _check(lib().mq_delta_score_topk(_ptr(W), _ptr(H), ctypes.byref(mat(base)), rs, budget, _ptr(delta), _ptr(rank),
                                     _ptr(sel), _ptr(ws), wsb, _stream(stream)), "mq_delta_score_topk")


def mq_pack_residual(resid: dict, sel, budget: int, packed: dict, stream=None):
    _check(lib().mq_pack_residual(ctypes.byref(mat(resid)), _ptr(sel), budget, ctypes.byref(packed_struct(packed)),
                                  _stream(stream)), "mq_pack_residual")


def mq_pack_residual_weight(W: torch.Tensor, base: dict, sel, budget: int, packed: dict, stream=None):
    _check(lib().mq_pack_residual_weight(_ptr(W), ctypes.byref(mat(base)), _ptr(sel), budget,
                                         ctypes.byref(packed_struct(packed)), _stream(stream)),
           "mq_pack_residual_weight")


def mq_quantize_act(X: torch.Tensor, xq: dict, stream=None):
    M, K = X.shape
    _check(lib().mq_quantize_act(_ptr(X), M, K, ctypes.byref(mat(xq)), _stream(stream)), "mq_quantize_act")


def mq_gemm(xq: dict, wq: dict, packed: dict | None, Y: torch.Tensor, M: int, N: int, K: int, flags: int = 0,
            ws: torch.Tensor | None = None, stream=None):
    ps = packed_struct(packed)
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().mq_gemm(ctypes.byref(mat(xq)), ctypes.byref(mat(wq)), None if ps is None else ctypes.byref(ps),
                         _ptr(Y), M, N, K, flags, _ptr(ws), wsb, _stream(stream)), "mq_gemm")


def mq_run_layer(W, X, Xcal, Y, M: int, N: int, K: int, T: int, budget: int, flags: int, host: bool,
                 buf: LayerBuffers, stream=None):
    """Whole path in one call. With host=True, W/X/Xcal/Y are pinned CPU tensors."""
    def p(t):
        if t is None:
            return None
        if host:
            if t.is_cuda:
                raise MosaicError("host=True expects CPU tensors")
            return t.data_ptr()
        return _ptr(t)
    _check(lib().mq_run_layer(p(W), p(X), p(Xcal), p(Y), M, N, K, T, budget, flags, 1 if host else 0,
                              ctypes.byref(buf), _stream(stream)), "mq_run_layer")


def mq_gemm_act(X: torch.Tensor, wq: dict, packed: dict | None, Y: torch.Tensor, M: int, N: int, K: int,
                flags: int = 0, ws: torch.Tensor | None = None, gx: torch.Tensor | None = None, stream=None):
    """Decode-kernel GEMM that quantizes the bf16 activations itself (gx receives g_x)."""
    ps = packed_struct(packed)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().mq_gemm_act(_ptr(X), ctypes.byref(mat(wq)), None if ps is None else ctypes.byref(ps), _ptr(Y), M, N,
                             K, flags, _ptr(ws), nbytes, _ptr(gx), _stream(stream)), "mq_gemm_act")


def mq_gemm_noalloc(xq: dict, wq: dict, packed: dict | None, Y: torch.Tensor, M: int, N: int, K: int,
                    flags: int = 0, stream=None):
    """mq_gemm for callers that cannot allocate device memory: no workspace argument,
    the split-K scratch is a static buffer inside the library (see include/mosaic.h)."""
    ps = packed_struct(packed)
    _check(lib().mq_gemm_noalloc(ctypes.byref(mat(xq)), ctypes.byref(mat(wq)), None if ps is None else ctypes.byref(ps),
                                 _ptr(Y), M, N, K, flags, _stream(stream)), "mq_gemm_noalloc")


def mq_fp4_mma_loop(ctas: int, iters: int, stream=None) -> float:
    """Launch the FP4 MMA-loop probe (include/mosaic_probe.h); returns its flop count."""
    _check(lib().mq_fp4_mma_loop(ctas, iters, _stream(stream)), "mq_fp4_mma_loop")
    return float(lib().mq_fp4_mma_loop_flops(ctas, iters))


def mq_get_error(stream=None) -> int:
    return lib().mq_get_error(_stream(stream))


def mq_launch_count() -> int:
    return int(lib().mq_launch_count())


def gemm_workspace(M: int, N: int, K: int, flags: int, device) -> torch.Tensor | None:
    """Zero-initialised workspace for mq_gemm (the tile counters must start at zero)."""
    n = lib().mq_gemm_workspace_bytes(M, N, K, flags)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device) if n else None


# ------------------------------------------------------------------ mosaic_ops.h
_marshal = None


def _ops():
    """The extension module that checks these operators' operands and calls the library (csrc/marshal.cpp)."""
    global _marshal
    if _marshal is None:
        L = lib()
        path = build.marshal_path()
        if not os.path.exists(path):
            raise MosaicError(f"{path} is not built; run __graft_entry__.build()")
        spec = importlib.util.spec_from_file_location(__package__ + "._marshal", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.bind(MosaicError, *(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
            "mq_gemv", "mq_qk_norm_rope", "mq_kv_append", "mq_qkv_append", "mq_kv_read", "mq_kv_attention",
            "mq_status_string", "mq_gemv_workspace_bytes")))
        _marshal = m
    return _marshal


def _raw(stream):
    return None if stream is None else stream.cuda_stream


class Weight:
    """A packed weight (base, and optionally its residual blocks) with the C structs that
    the calls take, built once. Keeps the tensors alive."""

    def __init__(self, base: dict, packed: dict | None = None):
        self.N, self.K = base["rows"], base["cols"]
        self.base, self.packed, self.dev = base, packed, base["codes"].get_device()
        self._mat, self._res = mat(base), packed_struct(packed)
        self.base_ptr = ctypes.addressof(self._mat)
        self.packed_ptr = None if self._res is None else ctypes.addressof(self._res)


class KVCache:
    """A paged NVFP4 key/value cache (include/mosaic_ops.h, mq_kv_cache) over a byte tensor
    [pages][heads][page_size / 16][18 D]; k_scale, v_scale: fp32 [heads] or None (1.0)."""

    def __init__(self, pages: torch.Tensor, k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None):
        if pages.dtype != torch.uint8 or pages.dim() != 4 or not pages.is_contiguous() or pages.shape[3] not in (1152, 2304):
            raise MosaicError("pages: a contiguous uint8 tensor [pages][heads][page_size / 16][18 D], D = 64 or 128")
        self.pages, self.k_scale, self.v_scale = pages, k_scale, v_scale
        self.num_pages, self.heads, self.D = pages.shape[0], pages.shape[1], pages.shape[3] // 18
        self.page_size, self.dev = 16 * pages.shape[2], pages.get_device()
        for s in (k_scale, v_scale):
            if s is not None:
                if s.dtype != torch.float32 or s.device != pages.device or s.numel() < self.heads or not s.is_contiguous():
                    raise MosaicError(f"tensor scales: {self.heads} contiguous fp32 values on {pages.device} are wanted")
        self._struct = KVCacheStruct(_ptr(pages), self.num_pages, self.page_size, self.heads, self.D, _ptr(k_scale),
                                     _ptr(v_scale))
        self.ptr = ctypes.addressof(self._struct)

    @classmethod
    def alloc(cls, num_pages: int, page_size: int, heads: int, D: int, device="cuda", k_scale=None, v_scale=None):
        if lib().mq_kv_cache_bytes(num_pages, page_size, heads, D) == 0:
            raise MosaicError(f"bad cache shape: {num_pages} pages of {page_size}, {heads} heads, D = {D}")
        return cls(torch.zeros((num_pages, heads, page_size // 16, 18 * D), dtype=torch.uint8, device=device), k_scale,
                   v_scale)


def mq_gemv(X: torch.Tensor, w: Weight, Y: torch.Tensor, flags: int = 0, stream=None, ws=None):
    """Y [M][N] = X [M][K] times the packed weight, X in 16 bits (not quantized), M <= 16. ws:
    mq_gemv_workspace_bytes(M, K) bytes, or None: a block of PyTorch's caching allocator."""
    (_marshal or _ops()).gemv(X, Y, w.N, w.K, w.dev, w.base_ptr, w.packed_ptr, flags, _raw(stream), ws)


def mq_qk_norm_rope(q, k, q_out, k_out, pos=None, freq=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                    interleaved: bool = False, stream=None):
    """Head norms and the rotation of q [T][heads][D] and k (either may be None); the
    outputs may be the inputs. freq: fp64 [rot / 2] radians a position."""
    (_marshal or _ops()).qk_norm_rope(q, k, q_out, k_out, pos, freq, q_weight, k_weight, eps, interleaved, _raw(stream))


def mq_kv_append(k, v, slots, cache: KVCache, stream=None):
    """Rows k, v [T][heads][D] into the cache at slots (int64 [T], negative: skipped)."""
    (_marshal or _ops()).kv_append(k, v, slots, cache.ptr, cache.dev, _raw(stream))


def mq_qkv_append(q, k, v, q_out, slots, cache: KVCache, pos=None, freq=None, q_weight=None, k_weight=None,
                  eps: float = 1e-6, interleaved: bool = False, k_out=None, stream=None):
    """mq_qk_norm_rope and mq_kv_append in one launch (the turned keys go to the cache, and
    to k_out if given)."""
    (_marshal or _ops()).qkv_append(q, k, v, q_out, k_out, pos, freq, q_weight, k_weight, eps, interleaved, slots,
                                    cache.ptr, cache.dev, _raw(stream))


def mq_kv_read(cache: KVCache, slots, k, v, stream=None):
    """The cached rows of slots (int64 [T]) as 16-bit k, v [T][heads][D]."""
    (_marshal or _ops()).kv_read(cache.ptr, cache.dev, slots, k, v, _raw(stream))


def kv_attention_workspace(q: torch.Tensor, cache: KVCache, max_q: int = 1) -> torch.Tensor | None:
    """Zeroed workspace for mq_kv_attention with q's heads (see include/mosaic_ops.h)."""
    with torch.cuda.device(q.device):
        n = lib().mq_kv_attention_workspace_bytes(q.shape[1], cache.heads, cache.D, max_q)
    return torch.zeros(n, dtype=torch.uint8, device=q.device) if n else None


def mq_kv_attention(q, cache: KVCache, block_table, kv_len, out, scale: float, cu_q=None, max_q: int = 1,
                    window: int = 0, lse=None, ws=None, stream=None):
    """out [T][heads][D] = attention of q over the cached tokens. block_table: int32 [B][pages],
    kv_len: int32 [B], cu_q: int32 [B + 1] or None (one query token a sequence), lse: fp32
    [T][heads] or None, ws: kv_attention_workspace(q, cache, max_q)."""
    (_marshal or _ops()).kv_attention(q, cache.ptr, cache.dev, block_table, kv_len, out, scale, cu_q, max_q, window, lse, ws,
                                      _raw(stream))


# ------------------------------------------------------------------ convenience
class Layer:
    """One linear layer through the whole path: quantize W, H from calibration tokens,
    Delta + top-K, pack, then per call quantize X and run the fused GEMM. Buffers are
    allocated once (torch) and reused."""

    def __init__(self, N: int, K: int, budget: int, device="cuda", with_sf: bool = True):
        self.N, self.K, self.budget, self.device = N, K, budget, device
        self.base, self.resid = alloc_weight(N, K, device, with_sf)
        self.qws = torch.empty(lib().mq_quantize_weight_workspace_bytes(N, K), dtype=torch.uint8, device=device)
        self.H = torch.empty(K, dtype=torch.float32, device=device)
        self.delta = torch.empty((N // 64) * (K // 64), dtype=torch.float64, device=device)
        self.rank = torch.empty(max(budget, 1), dtype=torch.int32, device=device)
        self.sel = torch.empty(max(budget, 1), dtype=torch.int32, device=device)
        self.packed = alloc_packed(N, K, budget, device)
        self._act = {}
        self._ws = {}  # of forward_fresh: stream -> ((M, flags) of the last call, workspace)

    def prepare(self, W: torch.Tensor, Xcal: torch.Tensor, stream=None):
        """A1..A5 through the separate calls (quantize, H, Delta + top-K, pack)."""
        mq_quantize_weight(W, self.base, self.resid, self.qws, stream)
        mq_hessian_diag(Xcal, self.H, stream)
        mq_delta_score_topk(W, self.H, self.base, None, self.budget, self.delta, self.rank, self.sel, None, stream)
        mq_pack_residual(self.resid, self.sel, self.budget, self.packed, stream)

    def prepare_fused(self, W: torch.Tensor, Xcal: torch.Tensor, stream=None):
        """A1..A5 with quantization and Delta in one pass over W; the full residual is stored
        and the selected blocks packed from it."""
        mq_hessian_diag(Xcal, self.H, stream)
        mq_quantize_weight_delta(W, self.H, self.base, self.resid, self.delta, self.qws, stream)
        mq_topk_blocks(self.delta, self.budget, self.rank, self.sel, stream)
        mq_pack_residual(self.resid, self.sel, self.budget, self.packed, stream)

    def prepare_path(self, W: torch.Tensor, Xcal: torch.Tensor, stream=None):
        """A1..A5 as mq_run_layer: the full residual is not stored; the selected blocks are
        recomputed from W when packed."""
        mq_hessian_diag(Xcal, self.H, stream)
        mq_quantize_weight_delta(W, self.H, self.base, None, self.delta, self.qws, stream)
        mq_topk_blocks(self.delta, self.budget, self.rank, self.sel, stream)
        mq_pack_residual_weight(W, self.base, self.sel, self.budget, self.packed, stream)

    def _kept(self, key, make):
        """The tensors that make() gives, kept for the next call with this key. What a captured call
        makes lies in its graph's memory, and is zeroed by a replay alone: the call keeps it to itself."""
        if key in self._act:
            return self._act[key]
        made = make()
        if not torch.cuda.is_current_stream_capturing():
            self._act[key] = made
        return made

    def act_buffers(self, M: int, flags: int = 0, slot: int = 0):
        """Quantized X, Y and the GEMM workspace for M tokens (cached per M, flags and slot:
        calls in flight together on different streams take different slots)."""
        return self._kept((M, flags, slot), lambda: (
            alloc_act(M, self.K, self.device), torch.empty((M, self.N), dtype=torch.bfloat16, device=self.device),
            gemm_workspace(M, self.N, self.K, flags, self.device)))

    def buffers(self, M: int, T: int, flags: int = 0, staging: bool = False, slot: int = 0) -> LayerBuffers:
        """The ctypes struct mq_run_layer takes (staging buffers for host inputs). Every slot
        has its own activation and staging buffers; the layer's weights are shared."""
        xq, Y, ws = self.act_buffers(M, flags, slot)
        b = LayerBuffers()
        b.act = xq, Y, ws  # alive as long as the pointers
        b.base, b.resid_full, b.xq = mat(self.base), mat(self.resid), mat(xq)
        b.H, b.delta, b.rank, b.sel = _ptr(self.H), _ptr(self.delta), _ptr(self.rank), _ptr(self.sel)
        b.packed = packed_struct(self.packed)
        b.ws_quant, b.ws_quant_bytes = _ptr(self.qws), self.qws.numel()
        b.ws_gemm, b.ws_gemm_bytes = (_ptr(ws), ws.numel()) if ws is not None else (None, 0)
        if staging:
            bf = torch.bfloat16
            w, x, xc = self._kept(("staging", M, T, slot), lambda: (
                torch.empty((self.N, self.K), dtype=bf, device=self.device),
                torch.empty((M, self.K), dtype=bf, device=self.device),
                torch.empty((T, self.K), dtype=bf, device=self.device)))
            b.staging = w, x, xc  # alive as long as the pointers
            b.W_dev, b.X_dev, b.Xcal_dev, b.Y_dev = _ptr(w), _ptr(x), _ptr(xc), _ptr(Y)
        return b

    def forward(self, X: torch.Tensor, flags: int = 0, stream=None) -> torch.Tensor:
        """A6 + A7/A8 on bf16 X [M][K] (device). Returns the layer's output buffer for this M
        and flags: the next call with the same M and flags writes into the same tensor."""
        M = X.shape[0]
        xq, Y, ws = self.act_buffers(M, flags)
        mq_quantize_act(X, xq, stream)
        mq_gemm(xq, self.base, self.packed, Y, M, self.N, self.K, flags, ws, stream)
        return Y

    def _gemm_workspace(self, M: int, flags: int, stream: int):
        """mq_gemm's workspace for M tokens on the current stream: one a stream, as large as any
        call needed. Where its counters lie goes by M, and a call leaves its own at zero: they are
        cleared when M changes. A captured call has its own, cleared at every replay."""
        n = lib().mq_gemm_workspace_bytes(M, self.N, self.K, flags)
        if n == 0:
            return None
        captured = torch.cuda.is_current_stream_capturing()
        last, ws = (None, None) if captured else self._ws.get(stream, (None, None))
        if last != (M, flags):
            if ws is None or ws.numel() < n:
                ws = _u8(n, device=self.device)
            # the last bytes of the n: a counter for 16 x 64 outputs, or for more of them
            ws[max(0, n - 4 * -(-M // 16) * (self.N // 64)):n].zero_()
            if not captured:
                self._ws[stream] = (M, flags), ws
        return ws

    def forward_fresh(self, X: torch.Tensor, flags: int = 0) -> torch.Tensor:
        """forward, of strided X too, on the current stream with buffers of this call alone (the workspace: of the
        stream's calls): the result is a new tensor, nothing is kept for this number of tokens,
        and calls on several streams or in captured graphs share no buffer."""
        if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != self.K:
            raise MosaicError(f"X [M][{self.K}] in bf16 is wanted, got {tuple(X.shape)} of {X.dtype}")
        X = X.contiguous()
        L, (M, K), s = lib(), X.shape, _stream()
        codes = M * K // 2
        sf = codes + -(-M // 128) * 8 * K  # rows in tiles of 128, a byte for 16 columns
        buf = torch.empty(sf + 4 * M, dtype=torch.uint8, device=X.device)
        p = buf.data_ptr()
        xq = NVFP4Mat(M, K, p, None, p + codes, p + sf)
        ws = self._gemm_workspace(M, flags, s.value)
        w = self.weight
        Y = torch.empty((M, self.N), dtype=torch.bfloat16, device=X.device)
        _check(L.mq_quantize_act(_ptr(X), M, K, ctypes.byref(xq), s), "mq_quantize_act")
        _check(L.mq_gemm(ctypes.byref(xq), ctypes.byref(w._mat), None if w._res is None else ctypes.byref(w._res), Y.data_ptr(),
                         M, self.N, K, flags, *((None, 0) if ws is None else (ws.data_ptr(), ws.numel())), s), "mq_gemm")
        return Y

    @property
    def weight(self) -> Weight:
        """The packed weight as mq_gemv takes it (built once; it reads the same buffers)."""
        if not hasattr(self, "_weight"):
            self._weight = Weight(self.base, self.packed)
        return self._weight

    def forward_16bit(self, X: torch.Tensor, out: torch.Tensor | None = None, flags: int = 0, stream=None):
        """X [M][K] in bf16 or fp16, M <= 16, times the packed weight without quantizing X
        (mq_gemv): a new tensor (of stream's memory pool), or out."""
        if out is None:
            with torch.cuda.stream(stream):
                out = torch.empty((X.shape[0], self.N), dtype=X.dtype, device=X.device)
        mq_gemv(X, self.weight, out, flags, stream)
        return out


class AttentionLayer:
    """The attention half of a decoder layer on quantized weights and a 4-bit cache:
    qkv projection, head norms + rotation + cache append, attention, out projection.

    qkv: a Layer of (q_heads + 2 kv_heads) * D rows (queries, keys, values); out: a Layer of
    q_heads * D columns; freq: fp64 [rot / 2]; q_norm, k_norm: [D] weights or None."""

    def __init__(self, qkv: Layer, out: Layer, q_heads: int, cache: KVCache, freq, q_norm=None, k_norm=None,
                 eps: float = 1e-6, interleaved: bool = False, scale: float | None = None, window: int = 0):
        D, H = cache.D, cache.heads
        if qkv.N != (q_heads + 2 * H) * D or out.K != q_heads * D:
            raise MosaicError(f"qkv must have {(q_heads + 2 * H) * D} rows and out {q_heads * D} columns")
        self.qkv, self.out, self.q_heads, self.cache = qkv, out, q_heads, cache
        self.freq, self.q_norm, self.k_norm, self.eps, self.interleaved = freq, q_norm, k_norm, eps, interleaved
        self.scale = D ** -0.5 if scale is None else scale
        self.window = window
        self._ws = {}

    def _project(self, layer: Layer, X):
        # up to 16 tokens the weight's bytes bound the product: X stays in 16 bits
        if X.shape[0] <= GEMV_MAX_TOKENS:
            return layer.forward_16bit(X)
        if X.dtype != torch.bfloat16:
            raise MosaicError("more than 16 tokens are taken in bf16")
        return layer.forward_fresh(X)

    def _workspace(self, q, max_q):
        # A captured call gets its own, zeroed at every replay: one kept here would be shared by
        # graphs that may run together, and be zeroed by the first one only.
        if torch.cuda.is_current_stream_capturing():
            return kv_attention_workspace(q, self.cache, max_q)
        # One for each stream, large enough for every max_q met on it (the size does not fall as
        # max_q grows): calls of all shapes may take turns on a workspace.
        key = torch.cuda.current_stream(q.device)
        served, ws = self._ws.get(key, (0, None))
        if max_q > served:
            more = kv_attention_workspace(q, self.cache, max_q)
            if ws is None or more is None or more.numel() > ws.numel():
                ws = more
            self._ws[key] = max_q, ws
        return ws

    def step(self, X, pos, slots, block_table, kv_len, cu_q=None, max_q: int = 1, stream=None, ws=None):
        """One pass of the T new tokens X [T][hidden] (bf16; fp16 up to 16 tokens): their keys
        and values are appended at slots, then they attend to their sequences. kv_len counts
        them. Tokens of one sequence are adjacent (cu_q). Returns a new tensor. Every stream and
        every captured call has its own buffers (ws: kv_attention_workspace(q, cache, max_q) of the
        caller's), so calls may overlap on different streams, as far as the cache's pages and the
        caller's ws allow it."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.step(X, pos, slots, block_table, kv_len, cu_q, max_q, None, ws)
        if not X.is_cuda:
            raise MosaicError("libmosaic takes CUDA tensors only")
        if X.get_device() != torch.cuda.current_device():
            with torch.cuda.device(X.get_device()):
                return self.step(X, pos, slots, block_table, kv_len, cu_q, max_q, None, ws)
        T, D, H, Hq = X.shape[0], self.cache.D, self.cache.heads, self.q_heads
        if T == 0:
            return X.new_empty((0, self.out.N))
        y = self._project(self.qkv, X).view(T, Hq + 2 * H, D)
        q, k, v = y[:, :Hq], y[:, Hq:Hq + H], y[:, Hq + H:]
        mq_qkv_append(q, k, v, q, slots, self.cache, pos, self.freq, self.q_norm, self.k_norm, self.eps,
                      self.interleaved)
        o = torch.empty((T, Hq, D), dtype=X.dtype, device=X.device)
        mq_kv_attention(q, self.cache, block_table, kv_len, o, self.scale, cu_q, max_q, self.window, None,
                        self._workspace(q, max_q) if ws is None else ws)
        return self._project(self.out, o.view(T, Hq * D))
