"""Python binding of libattn.so — argument marshalling only.

Every step of the attention path runs in the library's CUDA kernels; this
module converts torch tensors to pointers and sizes, passes the current CUDA
stream, and raises on a non-zero status.  There is no CPU fallback: if the
library is missing or the device is not sm_100, calls raise.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn.so")

ATTN_BF16, ATTN_FP16 = 0, 1
_DTYPES = {torch.bfloat16: ATTN_BF16, torch.float16: ATTN_FP16}

STATUS = {
    0: "ATTN_OK", -1: "ATTN_ERR_NULL", -2: "ATTN_ERR_SHAPE", -3: "ATTN_ERR_HEADDIM",
    -4: "ATTN_ERR_ALIGN", -5: "ATTN_ERR_DTYPE", -6: "ATTN_ERR_DEVICE", -7: "ATTN_ERR_LAUNCH",
    -8: "ATTN_ERR_TIMEOUT", -9: "ATTN_ERR_ARG", -10: "ATTN_ERR_SCRATCH", -11: "ATTN_ERR_PAGE",
}

# Kernel launches one attn_bwd call makes: the preprocess, then the main
# backward (d = 64), or the main backward and the dQ conversion (d = 128).
def bwd_launches(d: int) -> int:
    return 2 if d == 64 else 3

# Every symbol include/attn.h declares.
EXPORTS = ("attn_fwd", "attn_bwd", "attn_bwd_prep", "attn_bwd_main", "attn_bwd_workspace_bytes",
           "attn_bwd_noalloc", "attn_sdpa_host", "attn_sdpa_host_scratch_bytes",
           "attn_fwd_blocksparse", "attn_bwd_blocksparse", "attn_fp8_quantize", "attn_fwd_fp8",
           "attn_fwd_dropout", "attn_bwd_dropout", "attn_linear_fwd", "attn_linear_workspace_bytes",
           "attn_cache_append", "attn_cache_attend", "attn_cache_attend_workspace_bytes",
           "attn_decay_fwd", "attn_decay_bwd", "attn_decay_step", "attn_decay_workspace_bytes",
           "attn_last_device_status", "attn_selftest_wait_timeout",
           "attn_last_cuda_error_string", "attn_strerror", "attn_version")

# Size of the built-in scratch attn_bwd_noalloc uses (bytes, per device).
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        extra = ""
        if status in (-6, -7):
            extra = f"; CUDA: {lib().attn_last_cuda_error_string().decode()}"
        super().__init__(f"{where}: {STATUS.get(status, status)} ({strerror(status)}{extra})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libattn.so from the package directory (never from elsewhere)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m io_aware_exact_30_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, ci, cf, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.attn_fwd.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, vp]
        L.attn_fwd.restype = ci
        L.attn_bwd.argtypes = [vp] * 10 + [ci, ci, ci, ci, ci, cf, ci, vp]
        L.attn_bwd.restype = ci
        L.attn_bwd_prep.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, ci, vp]
        L.attn_bwd_prep.restype = ci
        L.attn_bwd_main.argtypes = [vp] * 8 + [ci, ci, ci, ci, ci, cf, ci, vp]
        L.attn_bwd_main.restype = ci
        L.attn_bwd_noalloc.argtypes = [vp] * 9 + [ci, ci, ci, ci, ci, cf, ci, vp]
        L.attn_bwd_noalloc.restype = ci
        L.attn_fwd_blocksparse.argtypes = [vp] * 6 + [ci, ci, ci, ci, ci, cf, ci, vp]
        L.attn_fwd_blocksparse.restype = ci
        L.attn_bwd_blocksparse.argtypes = [vp] * 11 + [ci, ci, ci, ci, ci, cf, ci, vp]
        L.attn_bwd_blocksparse.restype = ci
        L.attn_linear_workspace_bytes.argtypes = [ci, ci, ci, ci]
        L.attn_linear_workspace_bytes.restype = sz
        L.attn_linear_fwd.argtypes = [vp] * 5 + [ci, ci, ci, ci, cf, ci, vp]
        L.attn_linear_fwd.restype = ci
        L.attn_cache_append.argtypes = [vp] * 9 + [ci] * 8 + [vp]
        L.attn_cache_append.restype = ci
        L.attn_cache_attend_workspace_bytes.argtypes = [ci] * 6
        L.attn_cache_attend_workspace_bytes.restype = sz
        L.attn_cache_attend.argtypes = [vp] * 11 + [ci] * 10 + [cf, ci, vp]
        L.attn_cache_attend.restype = ci
        L.attn_decay_workspace_bytes.argtypes = [ci] * 5
        L.attn_decay_workspace_bytes.restype = sz
        L.attn_decay_fwd.argtypes = [vp] * 9 + [ci] * 5 + [cf, ci, vp]
        L.attn_decay_fwd.restype = ci
        L.attn_decay_bwd.argtypes = [vp] * 13 + [ci] * 5 + [cf, ci, vp]
        L.attn_decay_bwd.restype = ci
        L.attn_decay_step.argtypes = [vp] * 7 + [ci] * 3 + [cf, ci, vp]
        L.attn_decay_step.restype = ci
        u64 = ctypes.c_ulonglong
        L.attn_fwd_dropout.argtypes = [vp] * 5 + [ci, ci, ci, ci, ci, cf, cf, u64, ci, vp]
        L.attn_fwd_dropout.restype = ci
        L.attn_bwd_dropout.argtypes = [vp] * 10 + [ci, ci, ci, ci, ci, cf, cf, u64, ci, vp]
        L.attn_bwd_dropout.restype = ci
        L.attn_fp8_quantize.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, vp]
        L.attn_fp8_quantize.restype = ci
        L.attn_fwd_fp8.argtypes = [vp] * 7 + [ci, ci, ci, ci, ci, cf, ci, ci, vp]
        L.attn_fwd_fp8.restype = ci
        L.attn_sdpa_host_scratch_bytes.argtypes = [ci, ci, ci, ci, ci, ci]
        L.attn_sdpa_host_scratch_bytes.restype = sz
        L.attn_sdpa_host.argtypes = [vp] * 10 + [sz, ci, ci, ci, ci, ci, cf, ci, ci, vp]
        L.attn_sdpa_host.restype = ci
        L.attn_bwd_workspace_bytes.argtypes = [ci, ci, ci, ci]
        L.attn_bwd_workspace_bytes.restype = sz
        L.attn_last_device_status.argtypes = [vp]
        L.attn_last_device_status.restype = ci
        L.attn_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
        L.attn_selftest_wait_timeout.restype = ci
        L.attn_strerror.argtypes = [ci]
        L.attn_strerror.restype = ctypes.c_char_p
        L.attn_last_cuda_error_string.argtypes = []
        L.attn_last_cuda_error_string.restype = ctypes.c_char_p
        L.attn_version.argtypes = []
        L.attn_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().attn_strerror(int(status)).decode()


def version() -> str:
    return lib().attn_version().decode()


def _stream(device, stream):
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.current_stream(device).cuda_stream


def _check(rc: int, where: str):
    if rc != 0:
        raise AttnError(rc, where)


def _shape(q):
    if q.dim() != 4:
        raise ValueError("q must be (B, H, N, d)")
    return q.shape


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _dtype(q):
    if q.dtype not in _DTYPES:
        raise TypeError(f"dtype must be bfloat16 or float16, got {q.dtype}")
    return _DTYPES[q.dtype]


def _same(ref, *ts, names):
    for t, n in zip(ts, names):
        if t.dtype != ref.dtype or t.shape != ref.shape or not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous with the shape and dtype of q")


def attn_fwd(q, k, v, o, lse, causal: bool, scale: float | None = None, stream=None) -> None:
    """O, LSE <- attention(q, k, v); all tensors caller-allocated, (B, H, N, d) / (B, H, N)."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, names=("k", "v", "o"))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, int(bool(causal)),
                        scale, _dtype(q), ctypes.c_void_p(_stream(q.device, stream)))
    _check(rc, "attn_fwd")


def attn_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib().attn_bwd_workspace_bytes(B, H, N, d))


def attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, causal: bool,
             scale: float | None = None, stream=None) -> None:
    """dQ, dK, dV <- gradients of sum(O * dout), recomputing P from lse."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, dout, dq, dk, dv, names=("k", "v", "o", "dout", "dq", "dk", "dv"))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    need = attn_bwd_workspace_bytes(B, H, N, d)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace needs {need} bytes")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                        _ptr(dv), _ptr(workspace), B, H, N, d, int(bool(causal)), scale, _dtype(q),
                        ctypes.c_void_p(_stream(q.device, stream)))
    _check(rc, "attn_bwd")


def attn_bwd_prep(o, dout, lse, workspace, stream=None) -> None:
    """Stage D = rowdot(dout, o) and lse * log2(e) in the workspace; clear the dQ accumulator."""
    B, H, N, d = _shape(o)
    _same(o, dout, names=("dout",))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    need = attn_bwd_workspace_bytes(B, H, N, d)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace needs {need} bytes")
    rc = lib().attn_bwd_prep(_ptr(o), _ptr(dout), _ptr(lse), _ptr(workspace), B, H, N, d, _dtype(o),
                             ctypes.c_void_p(_stream(o.device, stream)))
    _check(rc, "attn_bwd_prep")


def attn_bwd_main(q, k, v, dout, dq, dk, dv, workspace, causal: bool,
                  scale: float | None = None, stream=None) -> None:
    """Recompute backward on a workspace prepared by attn_bwd_prep."""
    B, H, N, d = _shape(q)
    _same(q, k, v, dout, dq, dk, dv, names=("k", "v", "dout", "dq", "dk", "dv"))
    need = attn_bwd_workspace_bytes(B, H, N, d)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace needs {need} bytes")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_bwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                             _ptr(workspace), B, H, N, d, int(bool(causal)), scale, _dtype(q),
                             ctypes.c_void_p(_stream(q.device, stream)))
    _check(rc, "attn_bwd_main")


def attn_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, causal: bool,
                     scale: float | None = None, stream=None) -> None:
    """attn_bwd without a workspace argument: the library uses its own fixed
    device array (``NOALLOC_SCRATCH_BYTES`` per device) and allocates nothing.
    For callers that have their inputs and outputs but no way to obtain
    scratch memory.  Calls that overlap on the GPU share that array and race."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, dout, dq, dk, dv, names=("k", "v", "o", "dout", "dq", "dk", "dv"))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                                _ptr(dk), _ptr(dv), B, H, N, d, int(bool(causal)), scale, _dtype(q),
                                ctypes.c_void_p(_stream(q.device, stream)))
    _check(rc, "attn_bwd_noalloc")


# Block size of attn_fwd_blocksparse / attn_bwd_blocksparse masks (rows and keys).
BLOCK = 128


def _check_mask(mask, N, device):
    nb = (N + BLOCK - 1) // BLOCK
    if (mask.dtype not in (torch.uint8, torch.bool) or tuple(mask.shape) != (nb, nb)
            or not mask.is_contiguous() or mask.device != device):
        raise ValueError(f"block mask must be a contiguous ({nb}, {nb}) uint8/bool tensor on {device}")


def attn_fwd_blocksparse(q, k, v, o, lse, block_mask, causal: bool, scale: float | None = None,
                         stream=None) -> None:
    """attn_fwd over the 128 x 128 blocks ``block_mask`` marks (one mask for all heads)."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, names=("k", "v", "o"))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    _check_mask(block_mask, N, q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_fwd_blocksparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(block_mask),
                                    B, H, N, d, int(bool(causal)), scale, _dtype(q),
                                    ctypes.c_void_p(_stream(q.device, stream)))
    _check(rc, "attn_fwd_blocksparse")


def attn_bwd_blocksparse(q, k, v, o, lse, dout, dq, dk, dv, workspace, block_mask, causal: bool,
                         scale: float | None = None, stream=None) -> None:
    """attn_bwd over the 128 x 128 blocks ``block_mask`` marks."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, dout, dq, dk, dv, names=("k", "v", "o", "dout", "dq", "dk", "dv"))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    _check_mask(block_mask, N, q.device)
    need = attn_bwd_workspace_bytes(B, H, N, d)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace needs {need} bytes")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_bwd_blocksparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                    _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                                    _ptr(block_mask), B, H, N, d, int(bool(causal)), scale,
                                    _dtype(q), ctypes.c_void_p(_stream(q.device, stream)))
    _check(rc, "attn_bwd_blocksparse")


def attn_fp8_quantize(x, x8, scales, signs=None, rotate: bool = True, stream=None) -> None:
    """x8 <- e4m3 codes of x's rows (times ``signs``, Hadamard-rotated when
    ``rotate``), one scale per 128-row block of each head into ``scales``."""
    B, H, N, d = _shape(x)
    nb = (N + 127) // 128
    if x8.dtype != torch.uint8 or tuple(x8.shape) != (B, H, N, d) or not x8.is_contiguous():
        raise ValueError("x8 must be a contiguous uint8 (B, H, N, d) tensor")
    if scales.dtype != torch.float32 or tuple(scales.shape) != (B, H, nb) or not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous float32 (B, H, {nb}) tensor")
    if signs is not None and (signs.dtype != torch.int8 or tuple(signs.shape) != (d,)):
        raise ValueError("signs must be an int8 tensor of d entries")
    rc = lib().attn_fp8_quantize(_ptr(x), _ptr(x8), _ptr(scales), _ptr(signs), int(bool(rotate)),
                                 B, H, N, d, _dtype(x), ctypes.c_void_p(_stream(x.device, stream)))
    _check(rc, "attn_fp8_quantize")


def attn_fwd_fp8(q8, k8, q_scale, k_scale, v, o, lse, causal: bool, scale: float | None = None,
                 rotated: bool = True, stream=None) -> None:
    """Forward with e4m3 scores (codes and scales from attn_fp8_quantize)."""
    B, H, N, d = _shape(v)
    _same(v, o, names=("o",))
    for t, n in ((q8, "q8"), (k8, "k8")):
        if t.dtype != torch.uint8 or tuple(t.shape) != (B, H, N, d) or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous uint8 (B, H, N, d) tensor")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(q_scale), _ptr(k_scale), _ptr(v), _ptr(o),
                            _ptr(lse), B, H, N, d, int(bool(causal)), scale, int(bool(rotated)),
                            _dtype(v), ctypes.c_void_p(_stream(v.device, stream)))
    _check(rc, "attn_fwd_fp8")


def attn_fwd_dropout(q, k, v, o, lse, causal: bool, dropout_p: float, seed: int,
                     scale: float | None = None, stream=None) -> None:
    """attn_fwd with dropout on P (Philox4x32-10 mask from ``seed``)."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, names=("k", "v", "o"))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_fwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                                int(bool(causal)), scale, float(dropout_p),
                                int(seed) & 0xFFFFFFFFFFFFFFFF, _dtype(q),
                                ctypes.c_void_p(_stream(q.device, stream)))
    _check(rc, "attn_fwd_dropout")


def attn_bwd_dropout(q, k, v, o, lse, dout, dq, dk, dv, workspace, causal: bool,
                     dropout_p: float, seed: int, scale: float | None = None, stream=None) -> None:
    """attn_bwd for attn_fwd_dropout (the same dropout_p and seed)."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, dout, dq, dk, dv, names=("k", "v", "o", "dout", "dq", "dk", "dv"))
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 (B, H, N) tensor")
    need = attn_bwd_workspace_bytes(B, H, N, d)
    if workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace needs {need} bytes")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_bwd_dropout(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), B, H, N, d,
                                int(bool(causal)), scale, float(dropout_p),
                                int(seed) & 0xFFFFFFFFFFFFFFFF, _dtype(q),
                                ctypes.c_void_p(_stream(q.device, stream)))
    _check(rc, "attn_bwd_dropout")


def attn_linear_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib().attn_linear_workspace_bytes(B, H, N, d))


def attn_linear_fwd(q, k, v, o, workspace, scale: float | None = None, stream=None) -> None:
    """Causal linear attention O_i = scale sum_{j<=i} (q_i . k_j) v_j (d = 128)."""
    B, H, N, d = _shape(q)
    _same(q, k, v, o, names=("k", "v", "o"))
    need = attn_linear_workspace_bytes(B, H, N, d)
    if need == 0 or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace needs {need} bytes (d must be 128)")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_linear_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(workspace), B, H, N, d,
                               scale, _dtype(q), ctypes.c_void_p(_stream(q.device, stream)))
    _check(rc, "attn_linear_fwd")


# Page sizes (tokens) of the 8-bit cache.
PAGE_SIZES = (16, 32, 64, 128)
_CODES = (torch.float8_e4m3fn, torch.uint8)
_F32, _I32 = torch.float32, torch.int32


class Cache8(NamedTuple):
    """A paged key/value cache in e4m3: codes (num_pages, Hkv, page, d)
    float8_e4m3fn (or the same bytes as uint8), and one power-of-two fp32 scale for
    each page and head, (num_pages, Hkv); value = code * scale."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def cache_alloc(num_pages: int, Hkv: int, page: int, d: int, device="cuda") -> Cache8:
    """An empty cache.  Pages need no clearing when they are used again."""
    if page not in PAGE_SIZES:
        raise ValueError(f"page must be one of {PAGE_SIZES}")
    codes = [torch.zeros((num_pages, Hkv, page, d), dtype=torch.uint8,
                         device=device).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros((num_pages, Hkv), dtype=torch.float32, device=device) for _ in range(2)]
    return Cache8(*codes, *scales)


# The token-by-token calls run for a few microseconds on the device, so their
# marshalling counts: tensors are checked without building intermediate objects,
# addresses are passed as integers, and the current stream is read as a handle.

def _at(t):
    return None if t is None else t.data_ptr()


def _handle(t, stream):
    """Handle of `stream`, or of the current stream of t's device."""
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if not t.is_cuda:
        raise ValueError("tensors must be device memory")
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _alike(shape, dtype, ts, names):
    for t, n in zip(ts, names):
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous with shape {tuple(shape)} and dtype {dtype}")


def _optional(t, shape, dtype, name):
    if t is not None and (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} {tuple(shape)} tensor")


def _cache_shape(k, v, ks, vs, d, page_table, lens, B):
    """(num_pages, Hkv, page, max_pages) of a cache whose arrays fit together."""
    shape, code = k.shape, k.dtype
    if len(shape) != 4 or shape[3] != d or shape[2] not in PAGE_SIZES:
        raise ValueError(f"cache codes must be (num_pages, Hkv, page, {d}), page one of {PAGE_SIZES}")
    P, H, page, _ = shape
    if code not in _CODES:
        raise ValueError("cache codes must be float8_e4m3fn or uint8")
    if v.dtype is not code or v.shape != shape or not k.is_contiguous() or not v.is_contiguous():
        raise ValueError(f"cache k and v must be contiguous with shape {tuple(shape)} and one dtype")
    if ks.dtype is not _F32 or vs.dtype is not _F32 or ks.shape != (P, H) or vs.shape != (P, H) \
            or not ks.is_contiguous() or not vs.is_contiguous():
        raise ValueError(f"cache k_scale and v_scale must be contiguous float32 ({P}, {H}) tensors")
    table = page_table.shape
    if page_table.dtype is not _I32 or len(table) != 2 or table[0] != B or not page_table.is_contiguous():
        raise ValueError(f"page_table must be a contiguous int32 ({B}, max_pages) tensor")
    if lens.dtype is not _I32 or lens.shape != (B,) or not lens.is_contiguous():
        raise ValueError(f"lens must be a contiguous int32 ({B},) tensor")
    return P, H, page, table[1]


def _check_workspace(workspace, need):
    if need and (workspace is None or not workspace.is_contiguous()
                 or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace needs {need} contiguous bytes")


def attn_cache_append(k, v, cache: Cache8, page_table, lens, n_new=None, stream=None) -> None:
    """Stores the first n_new[b] (None: all T) new tokens of k, v (B, Hkv, T, d)
    behind the lens[b] tokens that sequence b holds; lens is not updated."""
    shape = _shape(k)
    B, H, T, d = shape
    code = _dtype(k)
    _alike(shape, k.dtype, (k, v), ("k", "v"))
    k8, v8, ks, vs = cache
    P, Hkv, page, width = _cache_shape(k8, v8, ks, vs, d, page_table, lens, B)
    if H != Hkv:
        raise ValueError(f"k and v have {H} heads, the cache {Hkv}")
    _optional(n_new, (B,), torch.int32, "n_new")
    rc = lib().attn_cache_append(k.data_ptr(), v.data_ptr(), k8.data_ptr(), v8.data_ptr(), ks.data_ptr(),
                                 vs.data_ptr(), page_table.data_ptr(), lens.data_ptr(), _at(n_new), B, H,
                                 T, d, P, page, width, code, _handle(k, stream))
    _check(rc, "attn_cache_append")


@functools.lru_cache(maxsize=256)
def attn_cache_attend_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, d: int, max_len: int) -> int:
    return int(lib().attn_cache_attend_workspace_bytes(B, Hq, Hkv, T, d, max_len))


def attn_cache_attend(q, cache: Cache8, page_table, lens, o, lse, workspace=None, causal: bool = True,
                      scale: float | None = None, q_lens=None, max_len: int | None = None,
                      stream=None) -> None:
    """O, LSE <- attention of the last q_lens[b] (None: T) queries of each sequence
    over its lens[b] tokens in the cache; rows past q_lens[b] are left as they
    were.  max_len: an upper bound of lens (None: the table's capacity)."""
    shape = _shape(q)
    _alike(shape, q.dtype, (q, o), ("q", "o"))
    _alike(shape[:3], torch.float32, (lse,), ("lse",))
    _attend(q, shape, cache, page_table, lens, o, lse, workspace, causal, scale, q_lens, max_len, stream)


def _attend(q, shape, cache, page_table, lens, o, lse, workspace, causal, scale, q_lens, max_len, stream):
    """attn_cache_attend with o and lse known to fit; workspace False: allocate it."""
    B, Hq, T, d = shape
    code = _dtype(q)
    k8, v8, ks, vs = cache
    P, Hkv, page, width = _cache_shape(k8, v8, ks, vs, d, page_table, lens, B)
    _optional(q_lens, (B,), torch.int32, "q_lens")
    max_len = width * page if max_len is None else int(max_len)
    need = attn_cache_attend_workspace_bytes(B, Hq, Hkv, T, d, max_len)
    if workspace is False:
        workspace = q.new_empty(need, dtype=torch.uint8) if need else None
    else:
        _check_workspace(workspace, need)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_cache_attend(q.data_ptr(), k8.data_ptr(), v8.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                                 page_table.data_ptr(), lens.data_ptr(), _at(q_lens), o.data_ptr(),
                                 lse.data_ptr(), _at(workspace), B, Hq, Hkv, T, d, P, page, width, max_len,
                                 1 if causal else 0, scale, code, _handle(q, stream))
    _check(rc, "attn_cache_attend")


@functools.lru_cache(maxsize=256)
def attn_decay_workspace_bytes(B: int, H: int, N: int, d: int, backward: bool = False) -> int:
    return int(lib().attn_decay_workspace_bytes(B, H, N, d, int(bool(backward))))


def attn_decay_fwd(q, k, v, log_decay, o, state_in=None, state_out=None, lens=None, workspace=None,
                   scale: float | None = None, stream=None, zero_past: bool = False) -> None:
    """O, state_out <- linear attention with a decay for each head, from state_in
    (None: zeros); rows of o past lens[b] are written as zeros or left as they were."""
    shape = _shape(q)
    B, H, N, d = shape
    code = _dtype(q)
    _alike(shape, q.dtype, (q, k, v, o), ("q", "k", "v", "o"))
    _alike((H,), torch.float32, (log_decay,), ("log_decay",))
    _optional(state_in, (B, H, d, d), torch.float32, "state_in")
    _optional(state_out, (B, H, d, d), torch.float32, "state_out")
    _optional(lens, (B,), torch.int32, "lens")
    _check_workspace(workspace, attn_decay_workspace_bytes(B, H, N, d))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_decay_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _at(state_in),
                              _at(lens), o.data_ptr(), _at(state_out), _at(workspace), B, H, N, d,
                              1 if zero_past else 0, scale, code, _handle(q, stream))
    _check(rc, "attn_decay_fwd")


def attn_decay_bwd(q, k, v, log_decay, dout, dq, dk, dv, state_in=None, dstate_out=None,
                   dstate_in=None, lens=None, workspace=None, scale: float | None = None,
                   stream=None, zero_past: bool = False) -> None:
    """dQ, dK, dV, dstate_in <- gradients of sum(O * dout) + sum(state_out *
    dstate_out); rows past lens[b] are written as zeros or left as they were."""
    shape = _shape(q)
    B, H, N, d = shape
    code = _dtype(q)
    _alike(shape, q.dtype, (q, k, v, dout, dq, dk, dv), ("q", "k", "v", "dout", "dq", "dk", "dv"))
    _alike((H,), torch.float32, (log_decay,), ("log_decay",))
    _optional(state_in, (B, H, d, d), torch.float32, "state_in")
    _optional(dstate_out, (B, H, d, d), torch.float32, "dstate_out")
    _optional(dstate_in, (B, H, d, d), torch.float32, "dstate_in")
    _optional(lens, (B,), torch.int32, "lens")
    _check_workspace(workspace, attn_decay_workspace_bytes(B, H, N, d, True))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_decay_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                              dout.data_ptr(), _at(state_in), _at(dstate_out), _at(lens), dq.data_ptr(),
                              dk.data_ptr(), dv.data_ptr(), _at(dstate_in), _at(workspace), B, H, N, d,
                              1 if zero_past else 0, scale, code, _handle(q, stream))
    _check(rc, "attn_decay_bwd")


def attn_decay_step(q, k, v, log_decay, state_in, o, state_out, scale: float | None = None,
                    stream=None) -> None:
    """O, state_out <- one token, q, k, v, o (B, H, 1, d); state_out may be state_in."""
    shape = _shape(q)
    B, H, N, d = shape
    if N != 1:
        raise ValueError("a step takes one token: q must be (B, H, 1, d)")
    code = _dtype(q)
    _alike(shape, q.dtype, (q, k, v, o), ("q", "k", "v", "o"))
    _alike((H,), torch.float32, (log_decay,), ("log_decay",))
    _alike((B, H, d, d), torch.float32, (state_in,) if state_in is state_out else (state_in, state_out),
           ("state_in", "state_out"))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_decay_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                               state_in.data_ptr(), o.data_ptr(), state_out.data_ptr(), B, H, d, scale,
                               code, _handle(q, stream))
    _check(rc, "attn_decay_step")


def attn_sdpa_host_scratch_bytes(B: int, H: int, N: int, d: int, with_backward: bool,
                                 heads_per_chunk: int = 0) -> int:
    return int(lib().attn_sdpa_host_scratch_bytes(B, H, N, d, int(bool(with_backward)),
                                                  int(heads_per_chunk)))


def attn_sdpa_host(q, k, v, dout, o, lse, dq, dk, dv, scratch, causal: bool,
                   scale: float | None = None, heads_per_chunk: int = 0, stream=None) -> None:
    """Attention from host buffers: q, k, v, dout and the outputs are CPU
    tensors (pinned, for the copies to overlap); ``dout=None`` runs the forward
    alone (o and lse required).  ``scratch`` is a CUDA uint8 tensor of
    attn_sdpa_host_scratch_bytes() bytes."""
    B, H, N, d = _shape(q)
    host = [t for t in (q, k, v, dout, o, lse, dq, dk, dv) if t is not None]
    if any(t.device.type != "cpu" or not t.is_contiguous() for t in host):
        raise ValueError("host tensors must be contiguous CPU tensors")
    if scratch.device.type != "cuda":
        raise ValueError("scratch must be device memory")
    sc = 1.0 / math.sqrt(d) if scale is None else float(scale)
    rc = lib().attn_sdpa_host(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(o), _ptr(lse),
                              _ptr(dq), _ptr(dk), _ptr(dv), _ptr(scratch),
                              scratch.numel() * scratch.element_size(), B, H, N, d,
                              int(bool(causal)), sc, _dtype(q), int(heads_per_chunk),
                              ctypes.c_void_p(_stream(scratch.device, stream)))
    _check(rc, "attn_sdpa_host")


def attn_last_device_status(stream=None, device=None) -> int:
    st = _stream(device or torch.cuda.current_device(), stream)
    return int(lib().attn_last_device_status(ctypes.c_void_p(st)))


def attn_selftest_wait_timeout(timeout_us: int, stream=None) -> None:
    st = _stream(torch.cuda.current_device(), stream)
    _check(lib().attn_selftest_wait_timeout(int(timeout_us), ctypes.c_void_p(st)),
           "attn_selftest_wait_timeout")


# ------------------------------------------------------------ conveniences --
def forward(q, k, v, causal: bool = False, scale: float | None = None):
    """Allocates O and LSE with torch and runs attn_fwd; returns (o, lse)."""
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    attn_fwd(q, k, v, o, lse, causal, scale)
    return o, lse


def backward(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None,
             workspace=None):
    """Allocates dQ, dK, dV (and the workspace if not given); returns (dq, dk, dv)."""
    B, H, N, d = _shape(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = torch.empty(attn_bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8,
                                device=q.device)
    attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, causal, scale)
    return dq, dk, dv


def forward_blocksparse(q, k, v, block_mask, causal: bool = False, scale: float | None = None):
    """Allocates O and LSE and runs attn_fwd_blocksparse; returns (o, lse)."""
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    attn_fwd_blocksparse(q, k, v, o, lse, block_mask, causal, scale)
    return o, lse


def backward_blocksparse(q, k, v, o, lse, dout, block_mask, causal: bool = False,
                         scale: float | None = None):
    """Allocates dQ, dK, dV and the workspace; returns (dq, dk, dv)."""
    B, H, N, d = _shape(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(attn_bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8, device=q.device)
    attn_bwd_blocksparse(q, k, v, o, lse, dout, dq, dk, dv, ws, block_mask, causal, scale)
    return dq, dk, dv


def forward_fp8(q, k, v, causal: bool = False, scale: float | None = None, signs=None,
                rotate: bool = True):
    """Quantises q and k (rotated unless ``rotate`` is False) and runs
    attn_fwd_fp8; returns (o, lse).  ``signs``: int8 (d,) device tensor."""
    B, H, N, d = _shape(q)
    nb = (N + 127) // 128
    q8 = torch.empty((B, H, N, d), dtype=torch.uint8, device=q.device)
    k8 = torch.empty_like(q8)
    qs = torch.empty((B, H, nb), dtype=torch.float32, device=q.device)
    ks = torch.empty_like(qs)
    attn_fp8_quantize(q, q8, qs, signs, rotate)
    attn_fp8_quantize(k, k8, ks, signs, rotate)
    o = torch.empty_like(v)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    attn_fwd_fp8(q8, k8, qs, ks, v, o, lse, causal, scale, rotate)
    return o, lse


def forward_dropout(q, k, v, dropout_p: float, seed: int, causal: bool = False,
                    scale: float | None = None):
    """Allocates O and LSE and runs attn_fwd_dropout; returns (o, lse)."""
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    attn_fwd_dropout(q, k, v, o, lse, causal, dropout_p, seed, scale)
    return o, lse


def backward_dropout(q, k, v, o, lse, dout, dropout_p: float, seed: int, causal: bool = False,
                     scale: float | None = None):
    """Allocates dQ, dK, dV and the workspace; runs attn_bwd_dropout."""
    B, H, N, d = _shape(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(attn_bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8, device=q.device)
    attn_bwd_dropout(q, k, v, o, lse, dout, dq, dk, dv, ws, causal, dropout_p, seed, scale)
    return dq, dk, dv


def linear_forward(q, k, v, scale: float | None = None):
    """Allocates O and the workspace and runs attn_linear_fwd; returns o."""
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    ws = torch.empty(max(1, attn_linear_workspace_bytes(B, H, N, d)), dtype=torch.uint8,
                     device=q.device)
    attn_linear_fwd(q, k, v, o, ws, scale)
    return o


def cache_append(k, v, cache: Cache8, page_table, lens, n_new=None) -> None:
    """Stores new tokens in the cache: attn_cache_append."""
    attn_cache_append(k, v, cache, page_table, lens, n_new)


def cache_attend(q, cache: Cache8, page_table, lens, causal: bool = True, scale: float | None = None,
                 q_lens=None, max_len: int | None = None):
    """Allocates O, LSE and the workspace and runs attn_cache_attend; returns
    (o, lse).  Rows past q_lens[b] are 0 and -inf."""
    shape = _shape(q)
    _alike(shape, q.dtype, (q,), ("q",))
    o = torch.empty_like(q) if q_lens is None else torch.zeros_like(q)
    B, Hq, T, _ = shape
    lse = q.new_empty((B, Hq, T), dtype=torch.float32)
    if q_lens is not None:
        lse.fill_(-math.inf)
    _attend(q, shape, cache, page_table, lens, o, lse, False, causal, scale, q_lens, max_len, None)
    return o, lse


def decay_forward(q, k, v, log_decay, scale: float | None = None, state=None, lens=None):
    """Allocates O, the state and the workspace and runs attn_decay_fwd; returns
    (o, state after the last token).  Rows past lens[b] are 0."""
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    out = q.new_empty((B, H, d, d), dtype=torch.float32)
    need = attn_decay_workspace_bytes(B, H, N, d)
    ws = q.new_empty(need, dtype=torch.uint8) if need else None
    attn_decay_fwd(q, k, v, log_decay, o, state, out, lens, ws, scale, zero_past=True)
    return o, out


def decay_backward(q, k, v, log_decay, dout, scale: float | None = None, state=None, dstate=None,
                   lens=None):
    """Allocates the gradients and the workspace and runs attn_decay_bwd; returns
    (dq, dk, dv, gradient of the state before the first token).  Rows past
    lens[b] are 0."""
    B, H, N, d = _shape(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ds = q.new_empty((B, H, d, d), dtype=torch.float32)
    need = attn_decay_workspace_bytes(B, H, N, d, True)
    ws = q.new_empty(need, dtype=torch.uint8) if need else None
    attn_decay_bwd(q, k, v, log_decay, dout, dq, dk, dv, state, dstate, ds, lens, ws, scale, zero_past=True)
    return dq, dk, dv, ds


def decay_step(q, k, v, log_decay, state, scale: float | None = None, state_out=None):
    """One token: returns (o, state_out); state_out defaults to a new tensor and
    may be ``state`` itself."""
    o = torch.empty_like(q)
    out = torch.empty_like(state) if state_out is None else state_out
    attn_decay_step(q, k, v, log_decay, state, o, out, scale)
    return o, out


# ------------------------------------------------------------ several GPUs --
# Every (batch, head) pair is independent in both passes, so one problem's heads
# split across the ranks of a process group (one GPU each) with no exchange:
# each rank runs the single-GPU calls above on a contiguous range of the
# flattened B*H heads (views of the inputs; an LSE slice that would not be
# 16-byte aligned is copied).  The one collective is an optional all-gather of the
# outputs, for callers that want the whole tensors on every rank.  (Dropout is
# not offered here: its random bytes are keyed by the head index within the
# call, so a rank's slice would draw other bytes than the whole call.)

def head_shard(BH: int, rank: int, world: int) -> tuple[int, int]:
    """(first head, number of heads) of rank `rank` among `world` for B*H = BH
    flattened heads: contiguous ranges, the first BH % world ranks one head more."""
    if world < 1 or not 0 <= rank < world or BH < 0:
        raise ValueError("need 0 <= rank < world and BH >= 0")
    base, extra = divmod(BH, world)
    return rank * base + min(rank, extra), base + (1 if rank < extra else 0)


def _heads(x, s, n):
    """Heads [s, s + n) of a (B, H, ...) tensor as a contiguous (1, n, ...) tensor:
    a view, or a copy where the view would not start on the 16-byte boundary the
    ABI requires (an fp32 LSE slice when s * N is not a multiple of 4)."""
    B, H = x.shape[0], x.shape[1]
    view = x.reshape(B * H, *x.shape[2:])[s:s + n].unsqueeze(0)
    return view if view.data_ptr() % 16 == 0 else view.clone()


def _gather_heads(parts, shape, s_n, group):
    """All-gather every rank's (1, n_r, ...) slice into one (B, H, ...) tensor;
    uneven counts are padded to the largest for the collective."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    m = max(n for _, n in s_n)
    outs = []
    for part in parts:
        pad = part.new_zeros((1, m) + tuple(part.shape[2:]))
        pad[:, :part.shape[1]] = part
        bufs = [torch.empty_like(pad) for _ in range(world)]
        dist.all_gather(bufs, pad, group=group)
        full = torch.cat([b[0, :n] for b, (_, n) in zip(bufs, s_n)], dim=0)
        outs.append(full.reshape(shape[:2] + tuple(part.shape[2:])))
    return outs


def forward_sharded(q, k, v, causal: bool = False, scale: float | None = None, group=None,
                    gather: bool = True):
    """The forward of (B, H, N, d) q, k, v (the same on every rank of `group`)
    split by heads: this rank computes its head_shard() range with attn_fwd.
    gather=True returns the whole (o, lse) on every rank (one all-gather each);
    gather=False returns this rank's (o, lse) of shape (1, n, N, d) and (1, n, N)
    and its (first head, count)."""
    import torch.distributed as dist
    B, H, N, d = _shape(q)
    world, rank = dist.get_world_size(group), dist.get_rank(group)
    s_n = [head_shard(B * H, r, world) for r in range(world)]
    s, n = s_n[rank]
    if n > 0:
        o, lse = forward(_heads(q, s, n), _heads(k, s, n), _heads(v, s, n), causal, scale)
    else:
        o = q.new_empty((1, 0, N, d))
        lse = torch.empty((1, 0, N), dtype=torch.float32, device=q.device)
    if not gather:
        return o, lse, (s, n)
    o, lse = _gather_heads([o, lse], (B, H), s_n, group)
    return o, lse


def backward_sharded(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None,
                     group=None, gather: bool = True):
    """The backward split by heads as forward_sharded: this rank runs attn_bwd on
    its head range; gather=True returns the whole (dq, dk, dv) on every rank,
    gather=False this rank's slices and its (first head, count)."""
    import torch.distributed as dist
    B, H, N, d = _shape(q)
    world, rank = dist.get_world_size(group), dist.get_rank(group)
    s_n = [head_shard(B * H, r, world) for r in range(world)]
    s, n = s_n[rank]
    if n > 0:
        grads = backward(*(_heads(x, s, n) for x in (q, k, v, o, lse, dout)), causal, scale)
    else:
        grads = tuple(x.new_empty((1, 0, N, d)) for x in (q, k, v))
    if not gather:
        return (*grads, (s, n))
    return tuple(_gather_heads(list(grads), (B, H), s_n, group))
