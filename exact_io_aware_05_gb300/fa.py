"""Binding of libfa.so (include/fa.h): argument marshalling only.

Every function here checks tensor dtypes, shapes, devices and contiguity,
reads the current CUDA stream, and calls the C entry point of the same name
with raw device pointers, through ctypes.  The rotary and cache calls, which
take a few microseconds on the device, are checked and made by the CPython
module _fa_py (csrc/fa_py.c); where a check of its does not pass, the checks
here say why, and where it was not built for the running interpreter, they and
ctypes make the call, 3 to 4 us slower.  No attention arithmetic happens in Python and
there is no fallback: importing this module fails if libfa.so is missing, and
every nonzero status raises ``FAError``.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run exact_io_aware_05_gb300.build.build() "
                      "(or __graft_entry__.build()) first")

try:
    from . import _fa_py
except ImportError:
    _fa_py = None

_lib = ctypes.CDLL(LIB_PATH)
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_lib.fa_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp]
_lib.fa_fwd.restype = _i
_lib.fa_fwd_f32.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp]
_lib.fa_fwd_f32.restype = _i
_lib.fa_fwd_masked.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _i, _f, _vp]
_lib.fa_fwd_masked.restype = _i
_lib.fa_bwd_masked.argtypes = [_vp] * 9 + [_i] * 7 + [_vp, _i, _i, _f, _vp, _sz, _vp]
_lib.fa_bwd_masked.restype = _i
_lib.fa_fp8_vt_stride.argtypes = [_i]
_lib.fa_fp8_vt_stride.restype = _sz
_lib.fa_fp8_quantize.argtypes = [_vp] * 4 + [_i] * 5 + [_vp] * 6 + [_vp]
_lib.fa_fp8_quantize.restype = _i
_lib.fa_fwd_fp8.argtypes = [_vp] * 8 + [_i] * 6 + [_f, _vp]
_lib.fa_fwd_fp8.restype = _i
_lib.fa_decode.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]
_lib.fa_decode.restype = _i
_lib.fa_decode_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
_lib.fa_decode_workspace_bytes.restype = _sz
_lib.fa_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
_lib.fa_bwd_workspace_bytes.restype = _sz
_lib.fa_bwd.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _vp, _sz, _vp]
_lib.fa_bwd.restype = _i
_lib.fa_bwd_deterministic.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _vp, _sz, _vp]
_lib.fa_bwd_deterministic.restype = _i
_lib.fa_bwd_stage.argtypes = [_i] + [_vp] * 9 + [_i] * 6 + [_f, _vp, _sz, _vp]
_lib.fa_bwd_stage.restype = _i
_lib.fa_bwd_noalloc.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _vp]
_lib.fa_bwd_noalloc.restype = _i
_lib.fa_sync_status.argtypes = [_vp]
_lib.fa_sync_status.restype = _i
_lib.fa_status_string.argtypes = [_i]
_lib.fa_status_string.restype = ctypes.c_char_p


# one and two fa_heads (data, three strides, H), packed in one go: a step of a serving loop is a few
# microseconds on the device, and a ctypes structure costs one to build
_HEADS = struct.Struct("PqqqiI")
_HEADS2 = struct.Struct("PqqqiIPqqqiI")


class _RopeSpec(ctypes.Structure):
    _fields_ = [("d", _i), ("rot", _i), ("n_axes", _i), ("interleaved", _i),
                ("turns", ctypes.c_ulonglong * 128), ("axis", ctypes.c_ubyte * 128)]


class _KVCache(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("k", "v", "k_scale", "v_scale", "block_table", "lens", "seen", "weight", "order")] + \
               [(n, _i) for n in ("B", "Hkv", "d", "page_size", "num_pages", "max_pages", "dtype")]


_lib.fa_rope_spec_init.argtypes = [_vp, _i, _i, _i, _vp, _vp, _i]
_lib.fa_rope_spec_init.restype = _i
_lib.fa_rope.argtypes = [_vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _vp]
_lib.fa_rope.restype = _i
_lib.fa_cache_append.argtypes = [_vp] * 8 + [_i, _vp]
_lib.fa_cache_append.restype = _i
_lib.fa_decode_paged_workspace_bytes.argtypes = [_i] * 8
_lib.fa_decode_paged_workspace_bytes.restype = _sz
_lib.fa_decode_paged.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _f, _i, _vp, _sz, _vp]
_lib.fa_decode_paged.restype = _i
_lib.fa_cache_evict.argtypes = [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]
_lib.fa_cache_evict.restype = _i

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT, FA_ERR_BAD_INDEX = range(6)
FA_BF16, FA_F32, FA_E4M3 = range(3)


class FAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {_lib.fa_status_string(status).decode()} (status {status})")


def lib() -> ctypes.CDLL:
    return _lib


def _check(fn: str, st: int) -> None:
    if st != FA_OK:
        raise FAError(fn, st)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: torch.device) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _shapes(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k must be [B, H, T, d]")
    B, H, Tq, d = q.shape
    Tk = k.shape[2]
    return B, H, Tq, Tk, d


def fa_fwd(q, k, v, o, lse, causal: bool, scale: float, stream=None) -> None:
    """O and lse for bf16 q [B,H,Tq,d], k/v [B,H,Tk,d]; o bf16 like q, lse f32 [B,H,Tq]."""
    B, H, Tq, Tk, d = _shapes(q, k)
    dev = q.device
    _need(q, "q", torch.bfloat16, (B, H, Tq, d), dev)
    _need(k, "k", torch.bfloat16, (B, H, Tk, d), dev)
    _need(v, "v", torch.bfloat16, (B, H, Tk, d), dev)
    _need(o, "o", torch.bfloat16, (B, H, Tq, d), dev)
    _need(lse, "lse", torch.float32, (B, H, Tq), dev)
    _check("fa_fwd", _lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Tq, Tk, d,
                                 int(bool(causal)), float(scale), _stream(stream)))


def _block_mask(block_mask, B, H, Tq, Tk, dev):
    """(pointer, per_head) of a block mask: a uint8/bool tensor on `dev` shaped
    [ceil(Tq/128), ceil(Tk/128)] (all heads) or [B, H, ceil(Tq/128), ceil(Tk/128)]."""
    if block_mask is None:
        return None, 0
    nq, nk = -(-Tq // 128), -(-Tk // 128)
    if block_mask.device != dev or block_mask.dtype not in (torch.uint8, torch.bool) or \
            not block_mask.is_contiguous():
        raise ValueError("block_mask: contiguous uint8 or bool tensor on the inputs' device")
    if tuple(block_mask.shape) == (nq, nk):
        return block_mask.data_ptr(), 0
    if tuple(block_mask.shape) == (B, H, nq, nk):
        return block_mask.data_ptr(), 1
    raise ValueError(f"block_mask: shape ({nq}, {nk}) or ({B}, {H}, {nq}, {nk}), got {tuple(block_mask.shape)}")


def fa_fwd_masked(q, k, v, o, lse, window=(-1, -1), block_mask=None, scale: float = 1.0, stream=None) -> None:
    """fa_fwd under a window (left, right) around the bottom-right diagonal (-1 = unbounded
    side; (-1, 0) is causal) and an optional 128 x 128 block mask."""
    B, H, Tq, Tk, d = _shapes(q, k)
    dev = q.device
    _need(q, "q", torch.bfloat16, (B, H, Tq, d), dev)
    _need(k, "k", torch.bfloat16, (B, H, Tk, d), dev)
    _need(v, "v", torch.bfloat16, (B, H, Tk, d), dev)
    _need(o, "o", torch.bfloat16, (B, H, Tq, d), dev)
    _need(lse, "lse", torch.float32, (B, H, Tq), dev)
    bm, per_head = _block_mask(block_mask, B, H, Tq, Tk, dev)
    _check("fa_fwd_masked", _lib.fa_fwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Tq, Tk, d,
                                               int(window[0]), int(window[1]), bm, per_head, float(scale),
                                               _stream(stream)))


def fa_decode_workspace_bytes(B: int, H: int, Tq: int, Tk: int, d: int) -> int:
    return int(_lib.fa_decode_workspace_bytes(B, H, Tq, Tk, d))


def fa_decode(q, k, v, o, lse, causal: bool, scale: float, workspace: torch.Tensor, stream=None) -> None:
    """Split-KV O and lse (as fa_fwd) for Tq <= 16 (d = 64, 128) or 8 (d = 256) query rows."""
    B, H, Tq, Tk, d = _shapes(q, k)
    dev = q.device
    _need(q, "q", torch.bfloat16, (B, H, Tq, d), dev)
    _need(k, "k", torch.bfloat16, (B, H, Tk, d), dev)
    _need(v, "v", torch.bfloat16, (B, H, Tk, d), dev)
    _need(o, "o", torch.bfloat16, (B, H, Tq, d), dev)
    _need(lse, "lse", torch.float32, (B, H, Tq), dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous tensor on the same device")
    nbytes = workspace.numel() * workspace.element_size()
    _check("fa_decode", _lib.fa_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Tq, Tk, d,
                                       int(bool(causal)), float(scale), _ptr(workspace), nbytes,
                                       _stream(stream)))


def attention_decode(q, k, v, causal: bool, scale: float, workspace=None, stream=None):
    """Allocates O, lse (and the workspace if not given) and runs fa_decode."""
    B, H, Tq, Tk, d = _shapes(q, k)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Tq), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = fa_decode_workspace_bytes(B, H, Tq, Tk, d)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    fa_decode(q, k, v, o, lse, causal, scale, workspace, stream)
    return o, lse


def fa_fwd_f32(q, k, v, o, lse, causal: bool, scale: float, stream=None) -> None:
    """fp32 SIMT forward (precision reference path); all tensors float32."""
    B, H, Tq, Tk, d = _shapes(q, k)
    dev = q.device
    _need(q, "q", torch.float32, (B, H, Tq, d), dev)
    _need(k, "k", torch.float32, (B, H, Tk, d), dev)
    _need(v, "v", torch.float32, (B, H, Tk, d), dev)
    _need(o, "o", torch.float32, (B, H, Tq, d), dev)
    _need(lse, "lse", torch.float32, (B, H, Tq), dev)
    _check("fa_fwd_f32", _lib.fa_fwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Tq, Tk,
                                         d, int(bool(causal)), float(scale), _stream(stream)))


def fa_bwd_workspace_bytes(B: int, H: int, Tq: int, Tk: int, d: int) -> int:
    return int(_lib.fa_bwd_workspace_bytes(B, H, Tq, Tk, d))


def fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, causal: bool, scale: float, workspace: torch.Tensor,
           stream=None) -> None:
    """dQ, dK, dV (bf16) from bf16 q, k, v, o, dO and the f32 lse of fa_fwd."""
    _bwd_call("fa_bwd", q, k, v, o, lse, dO, dq, dk, dv, causal, scale, workspace, stream)


def fa_bwd_deterministic(q, k, v, o, lse, dO, dq, dk, dv, causal: bool, scale: float,
                         workspace: torch.Tensor, stream=None) -> None:
    """fa_bwd with the dQ additions in a fixed order: dq is bitwise reproducible."""
    _bwd_call("fa_bwd_deterministic", q, k, v, o, lse, dO, dq, dk, dv, causal, scale, workspace, stream)


def _bwd_call(entry, q, k, v, o, lse, dO, dq, dk, dv, causal, scale, workspace, stream):
    B, H, Tq, Tk, d = _shapes(q, k)
    dev = q.device
    for name, t, shp in (("q", q, (B, H, Tq, d)), ("k", k, (B, H, Tk, d)), ("v", v, (B, H, Tk, d)),
                         ("o", o, (B, H, Tq, d)), ("dO", dO, (B, H, Tq, d)), ("dq", dq, (B, H, Tq, d)),
                         ("dk", dk, (B, H, Tk, d)), ("dv", dv, (B, H, Tk, d))):
        _need(t, name, torch.bfloat16, shp, dev)
    _need(lse, "lse", torch.float32, (B, H, Tq), dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous tensor on the same device")
    nbytes = workspace.numel() * workspace.element_size()
    _check(entry, getattr(_lib, entry)(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                       _ptr(dk), _ptr(dv), B, H, Tq, Tk, d, int(bool(causal)), float(scale),
                                       _ptr(workspace), nbytes, _stream(stream)))


def fa_bwd_stage(stage: int, q, k, v, o, lse, dO, dq, dk, dv, causal: bool, scale: float,
                 workspace: torch.Tensor, stream=None) -> None:
    """Stage 1, 2 or 3 of fa_bwd (preprocess, tile loop, dQ finish); same arguments."""
    B, H, Tq, Tk, d = _shapes(q, k)
    nbytes = workspace.numel() * workspace.element_size()
    _check("fa_bwd_stage", _lib.fa_bwd_stage(int(stage), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                             _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), B, H, Tq, Tk, d,
                                             int(bool(causal)), float(scale), _ptr(workspace), nbytes,
                                             _stream(stream)))


def fa_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, causal: bool, scale: float, stream=None) -> None:
    """fa_bwd without a workspace argument, for callers that cannot allocate device memory:
    the scratch is a fixed array inside the library (see include/fa.h for its size limit
    and for why overlapping calls on one device must not be issued)."""
    B, H, Tq, Tk, d = _shapes(q, k)
    _check("fa_bwd_noalloc", _lib.fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO),
                                                 _ptr(dq), _ptr(dk), _ptr(dv), B, H, Tq, Tk, d,
                                                 int(bool(causal)), float(scale), _stream(stream)))


def fa_sync_status(stream=None) -> int:
    return int(_lib.fa_sync_status(_stream(stream)))


def fa_status_string(status: int) -> str:
    return _lib.fa_status_string(status).decode()


# ---------------------------------------------------------------- conveniences
def attention_forward(q, k, v, causal: bool, scale: float, stream=None, window=None, block_mask=None):
    """Allocates O and lse with torch and runs fa_fwd (bf16) or fa_fwd_f32 (float32); with a
    window (which replaces `causal`) or a block mask, fa_fwd_masked."""
    B, H, Tq, Tk, d = _shapes(q, k)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Tq), dtype=torch.float32, device=q.device)
    if window is not None or block_mask is not None:
        if window is None:
            window = (-1, 0 if causal else -1)
        elif causal:
            raise ValueError("give either causal or a window")
        fa_fwd_masked(q, k, v, o, lse, window, block_mask, scale, stream)
    else:
        (fa_fwd_f32 if q.dtype == torch.float32 else fa_fwd)(q, k, v, o, lse, causal, scale, stream)
    return o, lse


def fa_fp8_vt_stride(Tk: int) -> int:
    return int(_lib.fa_fp8_vt_stride(Tk))


class FP8Operands(dict):
    """Output of fa_fp8_quantize: q8, k8 [B,H,T,d] and vt8 [B,H,d,ld] e4m3 codes (uint8),
    q_descale [B,H,ceil(Tq/128)], k_descale [B,H,ceil(Tk/128)], v_descale [B,H,d] (f32)."""


def alloc_fp8(B, H, Tq, Tk, d, device) -> FP8Operands:
    u8, f32 = torch.uint8, torch.float32
    return FP8Operands(
        q8=torch.empty((B, H, Tq, d), dtype=u8, device=device),
        k8=torch.empty((B, H, Tk, d), dtype=u8, device=device),
        vt8=torch.empty((B, H, d, fa_fp8_vt_stride(Tk)), dtype=u8, device=device),
        q_descale=torch.empty((B, H, -(-Tq // 128)), dtype=f32, device=device),
        k_descale=torch.empty((B, H, -(-Tk // 128)), dtype=f32, device=device),
        v_descale=torch.empty((B, H, d), dtype=f32, device=device))


def _need_fp8(x: FP8Operands, B, H, Tq, Tk, d, dev):
    _need(x["q8"], "q8", torch.uint8, (B, H, Tq, d), dev)
    _need(x["k8"], "k8", torch.uint8, (B, H, Tk, d), dev)
    _need(x["vt8"], "vt8", torch.uint8, (B, H, d, fa_fp8_vt_stride(Tk)), dev)
    _need(x["q_descale"], "q_descale", torch.float32, (B, H, -(-Tq // 128)), dev)
    _need(x["k_descale"], "k_descale", torch.float32, (B, H, -(-Tk // 128)), dev)
    _need(x["v_descale"], "v_descale", torch.float32, (B, H, d), dev)


def fa_fp8_quantize(q, k, v, signs=None, out: FP8Operands = None, stream=None) -> FP8Operands:
    """e4m3 codes and dequantization factors of bf16 q, k, v (rotated by `signs`, a
    float32 [d] tensor of +-1 on the device, when given)."""
    B, H, Tq, Tk, d = _shapes(q, k)
    dev = q.device
    _need(q, "q", torch.bfloat16, (B, H, Tq, d), dev)
    _need(k, "k", torch.bfloat16, (B, H, Tk, d), dev)
    _need(v, "v", torch.bfloat16, (B, H, Tk, d), dev)
    if signs is not None:
        _need(signs, "signs", torch.float32, (d,), dev)
    x = alloc_fp8(B, H, Tq, Tk, d, dev) if out is None else out
    _need_fp8(x, B, H, Tq, Tk, d, dev)
    _check("fa_fp8_quantize", _lib.fa_fp8_quantize(
        _ptr(q), _ptr(k), _ptr(v), _ptr(signs), B, H, Tq, Tk, d, _ptr(x["q8"]), _ptr(x["k8"]), _ptr(x["vt8"]),
        _ptr(x["q_descale"]), _ptr(x["k_descale"]), _ptr(x["v_descale"]), _stream(stream)))
    return x


def fa_fwd_fp8(x: FP8Operands, o, lse, causal: bool, scale: float, stream=None) -> None:
    """O (bf16) and lse (f32) of attention over the dequantized FP8 operands."""
    B, H, Tq, d = x["q8"].shape
    Tk = x["k8"].shape[2]
    dev = x["q8"].device
    _need_fp8(x, B, H, Tq, Tk, d, dev)
    _need(o, "o", torch.bfloat16, (B, H, Tq, d), dev)
    _need(lse, "lse", torch.float32, (B, H, Tq), dev)
    _check("fa_fwd_fp8", _lib.fa_fwd_fp8(
        _ptr(x["q8"]), _ptr(x["k8"]), _ptr(x["vt8"]), _ptr(x["q_descale"]), _ptr(x["k_descale"]),
        _ptr(x["v_descale"]), _ptr(o), _ptr(lse), B, H, Tq, Tk, d, int(bool(causal)), float(scale),
        _stream(stream)))


def attention_forward_fp8(q, k, v, causal: bool, scale: float, signs=None, stream=None):
    """fa_fp8_quantize then fa_fwd_fp8; returns (o, lse, the FP8 operands)."""
    x = fa_fp8_quantize(q, k, v, signs, stream=stream)
    B, H, Tq, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Tq), dtype=torch.float32, device=q.device)
    fa_fwd_fp8(x, o, lse, causal, scale, stream)
    return o, lse, x


def alloc_workspace(B, H, Tq, Tk, d, device) -> torch.Tensor:
    n = fa_bwd_workspace_bytes(B, H, Tq, Tk, d)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def fa_bwd_masked(q, k, v, o, lse, dO, dq, dk, dv, window=(-1, -1), block_mask=None, deterministic=False,
                  scale: float = 1.0, workspace: torch.Tensor = None, stream=None) -> None:
    """Backward of fa_fwd_masked under the same window and block mask."""
    B, H, Tq, Tk, d = _shapes(q, k)
    dev = q.device
    for name, t, shp in (("q", q, (B, H, Tq, d)), ("k", k, (B, H, Tk, d)), ("v", v, (B, H, Tk, d)),
                         ("o", o, (B, H, Tq, d)), ("dO", dO, (B, H, Tq, d)), ("dq", dq, (B, H, Tq, d)),
                         ("dk", dk, (B, H, Tk, d)), ("dv", dv, (B, H, Tk, d))):
        _need(t, name, torch.bfloat16, shp, dev)
    _need(lse, "lse", torch.float32, (B, H, Tq), dev)
    if workspace is None or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on the same device")
    bm, per_head = _block_mask(block_mask, B, H, Tq, Tk, dev)
    nbytes = workspace.numel() * workspace.element_size()
    _check("fa_bwd_masked", _lib.fa_bwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                               _ptr(dk), _ptr(dv), B, H, Tq, Tk, d, int(window[0]), int(window[1]),
                                               bm, per_head, int(bool(deterministic)), float(scale),
                                               _ptr(workspace), nbytes, _stream(stream)))


def attention_backward(q, k, v, o, lse, dO, causal: bool, scale: float, workspace=None, stream=None,
                       deterministic: bool = False, window=None, block_mask=None):
    """Allocates dQ, dK, dV (and the workspace if not given) and runs fa_bwd
    (fa_bwd_deterministic when `deterministic`; fa_bwd_masked with a window, which
    replaces `causal`, or a block mask)."""
    B, H, Tq, Tk, d = _shapes(q, k)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = alloc_workspace(B, H, Tq, Tk, d, q.device) if workspace is None else workspace
    if window is not None or block_mask is not None:
        if window is None:
            window = (-1, 0 if causal else -1)
        elif causal:
            raise ValueError("give either causal or a window")
        fa_bwd_masked(q, k, v, o, lse, dO, dq, dk, dv, window, block_mask, deterministic, scale, ws, stream)
    else:
        (fa_bwd_deterministic if deterministic else fa_bwd)(q, k, v, o, lse, dO, dq, dk, dv, causal, scale, ws,
                                                            stream)
    return dq, dk, dv


# ---------------------------------------------------------------- rotary positions
class RopeSpec:
    """Rotary positions of head width d: `freqs` gives the frequency of each of the rot / 2
    pairs in radians per position, `axis` the axis of each pair (default: all on axis 0).
    Pair i is features i and i + rot / 2, or, interleaved, 2i and 2i + 1; the d - rot features
    behind the pairs pass through.  Host data only; keep it for all calls."""

    def __init__(self, d: int, freqs, axis=None, interleaved: bool = False):
        freqs = [float(f) for f in freqs]
        axis = [0] * len(freqs) if axis is None else [int(a) for a in axis]
        if len(axis) != len(freqs):
            raise ValueError(f"axis: expected {len(freqs)} entries, got {len(axis)}")
        if not freqs or len(freqs) > 128 or min(axis) < 0 or max(axis) > 255:
            raise ValueError("freqs, axis: 8 to 128 pairs with axes from 0")
        self.d, self.rot, self.n_axes, self.interleaved = int(d), 2 * len(freqs), max(axis) + 1, bool(interleaved)
        self._c = _RopeSpec()
        _check("fa_rope_spec_init", _lib.fa_rope_spec_init(
            ctypes.byref(self._c), self.d, self.rot, self.n_axes, (ctypes.c_double * len(freqs))(*freqs),
            (ctypes.c_ubyte * len(axis))(*axis), int(self.interleaved)))
        self._ref = ctypes.addressof(self._c)

    def __setstate__(self, state):   # of a copy or a pickle: the address is of its own structure
        self.__dict__.update(state)
        self._ref = ctypes.addressof(self._c)


def rope_spec(d: int, sections=None, base: float = 10000.0, rot: int | None = None,
              interleaved: bool = False) -> RopeSpec:
    """The usual frequencies base^(-2i / rot); `sections` splits the rot / 2 pairs into runs,
    one per axis (for instance (16, 24, 24) for time, height and width at rot = 128)."""
    rot = d if rot is None else rot
    sections = (rot // 2,) if sections is None else tuple(sections)
    if sum(sections) != rot // 2:
        raise ValueError(f"sections: {sections} do not add up to {rot // 2} pairs")
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    return RopeSpec(d, [base ** (-2.0 * i / rot) for i in range(rot // 2)], axis, interleaved)


_current_stream = torch._C._cuda_getCurrentRawStream    # of a device index; torch.cuda's builds an object
_current_device = torch._C._cuda_getDevice


class _Without:
    """Stands for _fa_py where it is missing: no call passes its checks."""
    rope = append = decode = evict = staticmethod(lambda *args: None)


if _fa_py is None:
    _fast = _Without
else:
    _fast = _fa_py
    _fa_py.setup(torch.bfloat16, torch.float32, torch.int32, _current_stream, _current_device,
                 *(ctypes.cast(f, _vp).value for f in (_lib.fa_rope, _lib.fa_cache_append, _lib.fa_decode_paged,
                                                       _lib.fa_cache_evict)))


def _launch(fn: str, entry, index: int, stream, *args) -> None:
    """Calls `entry` with the tensors' device current and a stream of that device: the given one, or
    its current stream."""
    if index < 0:
        raise ValueError(f"{fn}: expected CUDA tensors")
    stream = _current_stream(index) if stream is None else _stream(stream)
    had = _current_device()
    if had == index:
        st = entry(*args, stream)
    else:
        torch.cuda.set_device(index)
        try:
            st = entry(*args, stream)
        finally:
            torch.cuda.set_device(had)
    if st != FA_OK:
        raise FAError(fn, st)


def _again(status, fn: str, call, *args) -> None:
    """After _fa_py: its nonzero status as an error, or, for None, the call with the checks here."""
    if status is not None:
        raise FAError(fn, status)
    call(*args)


def _empties(stream, device, *specs) -> list:
    """torch.empty of each (shape, dtype), for a call on `stream`.  They are of that stream's memory: a
    block that was freed on the current stream may still be in use there.  The caller goes on with them
    on the current stream, so that one is recorded."""
    if stream is None or device.type != "cuda":
        return [torch.empty(shape, dtype=dtype, device=device) for shape, dtype in specs]
    if not isinstance(stream, torch.cuda.Stream):
        raw = _stream(stream)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        out = [torch.empty(shape, dtype=dtype, device=device) for shape, dtype in specs]
    here = torch.cuda.current_stream(device)
    for t in out:
        t.record_stream(here)
    return out


def _heads(t: torch.Tensor, name: str, dtype, shape, index: int) -> tuple:
    """The fields of fa_heads of a [B, H, T, d] tensor; only its last dimension has to be contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name}: expected a tensor on the others' device, got {t.device}")
    sb, sh, st, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # the stride of a dimension of one entry is never used: torch leaves any value there
    B, H, T, _ = shape
    return t.data_ptr(), sb if B > 1 else 0, sh if H > 1 else 0, st if T > 1 else 0, H, 0


def _rope(fn, q, q_out, positions, spec, k, k_out, inverse, stream):
    shape = q.shape
    if len(shape) != 4 or (k is None) != (k_out is None):
        raise ValueError("q, k must be [B, H, T, d], with an output for each")
    B, _, T, d = shape
    if d != spec.d:
        raise ValueError(f"q: expected head width {spec.d}, got {d}")
    dt, index = q.dtype, q.get_device()
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError(f"q: expected torch.bfloat16 or torch.float32, got {dt}")
    if positions.dtype is not torch.int32 or positions.shape != (spec.n_axes, B, T) or \
            positions.get_device() != index or not positions.is_contiguous():
        _need(positions, "positions", torch.int32, (spec.n_axes, B, T), q.device)
    x, y = _heads(q, "q", dt, shape, index), _heads(q_out, "q_out", dt, shape, index)
    if k is None:
        n, x, y = 1, _HEADS.pack(*x), _HEADS.pack(*y)
    else:
        if k.dim() != 4:
            raise ValueError("q, k must be [B, H, T, d], with an output for each")
        shape = (B, k.shape[1], T, d)
        n = 2
        x = _HEADS2.pack(*x, *_heads(k, "k", dt, shape, index))
        y = _HEADS2.pack(*y, *_heads(k_out, "k_out", dt, shape, index))
    _launch(fn, _lib.fa_rope, index, stream, x, y, n, positions.data_ptr(), spec._ref, B, T,
            FA_BF16 if dt is torch.bfloat16 else FA_F32, inverse)


def fa_rope(q, q_out, positions, spec: RopeSpec, k=None, k_out=None, stream=None) -> None:
    """q_out = q [B, Hq, T, d] (and k_out = k [B, Hk, T, d]) with their pairs turned by the
    positions, int32 [n_axes, B, T].  bf16 or float32; strided views with contiguous rows are
    taken as they are; an output may be its input."""
    st = _fast.rope(spec._ref, q, q_out, k, k_out, positions, 0, stream)
    if st != FA_OK:
        _again(st, "fa_rope", _rope, "fa_rope", q, q_out, positions, spec, k, k_out, 0, stream)


def fa_rope_bwd(dq_out, dq, positions, spec: RopeSpec, k=None, k_out=None, stream=None) -> None:
    """Backward of fa_rope: dq, the gradient of q, from dq_out, the gradient of q_out (and
    k_out from k, the gradients of k and of the rotated k)."""
    st = _fast.rope(spec._ref, dq_out, dq, k, k_out, positions, 1, stream)
    if st != FA_OK:
        _again(st, "fa_rope_bwd", _rope, "fa_rope_bwd", dq_out, dq, positions, spec, k, k_out, 1, stream)


def rope_forward(q, k, positions, spec: RopeSpec, stream=None):
    """Allocates contiguous outputs and runs fa_rope on q and k: what fa_fwd takes."""
    q_out, k_out = _empties(stream, q.device, (q.shape, q.dtype), (k.shape, k.dtype))
    fa_rope(q, q_out, positions, spec, k, k_out, stream)
    return q_out, k_out


def rope_backward(dq_out, dk_out, positions, spec: RopeSpec, stream=None):
    """Allocates and returns the gradients of q and k from those of rope_forward's outputs."""
    dq, dk = _empties(stream, dq_out.device, (dq_out.shape, dq_out.dtype), (dk_out.shape, dk_out.dtype))
    fa_rope_bwd(dq_out, dq, positions, spec, dk_out, dk, stream)
    return dq, dk


# ---------------------------------------------------------------- paged key/value cache
class KVCache:
    """Handle of a paged cache (fa_kv_cache in include/fa.h): checks its tensors once and keeps
    them.  k, v: [num_pages, Hkv, page_size, d] bf16, or uint8 e4m3 codes with k_scale and
    v_scale [Hkv] float32; block_table [B, max_pages] int32; lens [B] int32 (entries of each
    sequence, updated by the caller and by fa_cache_evict); seen [B] int32 (tokens ever
    appended; default: lens); weight float32 and order int32 [B, Hkv, max_pages * page_size],
    both optional.  The contents are read at each call.  A tensor assigned to one of these names is
    checked and takes the place of the one before, for calls from then on (a captured graph keeps the
    one that it was captured with); sizes stay as they are."""

    _TENSORS = ("k", "v", "block_table", "lens", "k_scale", "v_scale", "seen", "weight", "order")
    _FIXED = ("B", "Hkv", "d", "page_size", "num_pages", "max_pages", "device")

    def __init__(self, k, v, block_table, lens, k_scale=None, v_scale=None, weight=None, order=None, seen=None):
        if k.dim() != 4 or block_table.dim() != 2:
            raise ValueError("k must be [num_pages, Hkv, page_size, d] and block_table [B, max_pages]")
        if k.dtype not in (torch.bfloat16, torch.uint8):
            raise TypeError(f"k: expected torch.bfloat16 or torch.uint8 (e4m3 codes), got {k.dtype}")
        num_pages, Hkv, ps, d = k.shape
        B, max_pages = block_table.shape
        codes = k.dtype == torch.uint8
        f32, i32, pool, slots = torch.float32, torch.int32, (k.dtype, (num_pages, Hkv, ps, d)), (B, Hkv, max_pages * ps)
        self.__dict__.update(
            B=B, Hkv=Hkv, d=d, page_size=ps, num_pages=num_pages, max_pages=max_pages, device=k.device, _index=k.get_device(),
            _c=_KVCache(B=B, Hkv=Hkv, d=d, page_size=ps, num_pages=num_pages, max_pages=max_pages,
                        dtype=FA_E4M3 if codes else FA_BF16),
            # type and shape of each tensor, and whether it is there: always, never or as the caller likes (None)
            _want=dict(k=(*pool, True), v=(*pool, True), block_table=(i32, (B, max_pages), True), lens=(i32, (B,), True),
                       k_scale=(f32, (Hkv,), codes), v_scale=(f32, (Hkv,), codes), seen=(i32, (B,), None),
                       weight=(f32, slots, None), order=(i32, slots, None)))
        self.__dict__["_ref"] = ctypes.addressof(self._c)
        for name, t in zip(self._TENSORS, (k, v, block_table, lens, k_scale, v_scale, seen, weight, order)):
            setattr(self, name, t)

    def __setattr__(self, name, t):
        if name in self._FIXED:
            raise AttributeError(f"{name} of a KVCache is fixed: its tensors' sizes and the structure say so")
        if name in self._TENSORS:
            dtype, shape, there = self._want[name]
            if there is not None and (t is not None) != there:
                raise ValueError(f"{name}: needed" if there and "scale" not in name else
                                 f"{name}: needed with e4m3 codes and only with them")
            if t is not None:
                if not isinstance(t, torch.Tensor):
                    raise TypeError(f"{name}: expected a tensor, got {type(t).__name__}")
                _need(t, name, dtype, shape, self.device)
            setattr(self._c, name, _ptr(t))   # what the calls read
        self.__dict__[name] = t

    def __delattr__(self, name):
        if name in self._FIXED or name in self._TENSORS:
            raise AttributeError(f"{name} of a KVCache cannot be deleted")
        object.__delattr__(self, name)

    def __reduce__(self):   # copies and pickles are handles of their own, with a structure of their own
        return type(self), (self.k, self.v, self.block_table, self.lens, self.k_scale, self.v_scale, self.weight, self.order,
                            self.seen)


def alloc_kv_cache(B: int, Hkv: int, d: int, max_len: int, page_size: int = 16, k_scale=None, v_scale=None,
                   weight: bool = False, device="cuda") -> KVCache:
    """An empty cache with pages of its own for every sequence, up to max_len entries each: bf16,
    or e4m3 when the scales are given; with `weight` the accumulated weights, arrival numbers
    and token counts that eviction needs."""
    pages = -(-max_len // page_size)
    i32 = dict(dtype=torch.int32, device=device)
    dt = torch.bfloat16 if k_scale is None else torch.uint8
    k, v = (torch.zeros((B * pages, Hkv, page_size, d), dtype=dt, device=device) for _ in range(2))
    table = torch.arange(B * pages, **i32).view(B, pages)
    slots = (B, Hkv, pages * page_size)
    return KVCache(k, v, table, torch.zeros(B, **i32), k_scale, v_scale,
                   torch.zeros(slots, dtype=torch.float32, device=device) if weight else None,
                   torch.zeros(slots, **i32) if weight else None, torch.zeros(B, **i32) if weight else None)


def fa_cache_append(cache: KVCache, k, v, positions=None, spec: RopeSpec | None = None, q=None, q_out=None,
                    new_lens=None, stream=None) -> None:
    """Writes the first new_lens[b] (default: all) of the T rows of k and v [B, Hkv, T, d] as the
    last entries of sequence b; cache.lens (and seen) count them already.  With a spec, k is
    rotated by positions [n_axes, B, T] on the way, and q [B, Hq, T, d] into q_out."""
    st = _fast.append(cache._ref, cache._index, k, v, positions, None if spec is None else spec._ref, q, q_out, new_lens,
                       stream)
    if st != FA_OK:
        _again(st, "fa_cache_append", _append, cache, k, v, positions, spec, q, q_out, new_lens, stream)


def _append(cache, k, v, positions, spec, q, q_out, new_lens, stream) -> None:
    index, B, d = cache._index, cache.B, cache.d
    if k.dim() != 4 or (q is not None and q.dim() != 4):
        raise ValueError("k, v, q must be [B, H, T, d]")
    if (positions is None) != (spec is None):
        raise ValueError("positions and spec come together")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out come together")
    if q is not None and spec is None:
        raise ValueError("q is rotated: it needs a spec and positions")
    T = k.shape[2]
    shape = (B, cache.Hkv, T, d)
    bf16 = torch.bfloat16
    kh, vh = _HEADS.pack(*_heads(k, "k", bf16, shape, index)), _HEADS.pack(*_heads(v, "v", bf16, shape, index))
    pos = ref = qh = oh = new = None
    if spec is not None:
        if positions.dtype is not torch.int32 or positions.shape != (spec.n_axes, B, T) or \
                positions.get_device() != index or not positions.is_contiguous():
            _need(positions, "positions", torch.int32, (spec.n_axes, B, T), cache.device)
        pos, ref = positions.data_ptr(), spec._ref
    if q is not None:
        shape = (B, q.shape[1], T, d)
        qh = _HEADS.pack(*_heads(q, "q", bf16, shape, index))
        oh = _HEADS.pack(*_heads(q_out, "q_out", bf16, shape, index))
    if new_lens is not None:
        _need(new_lens, "new_lens", torch.int32, (B,), cache.device)
        new = new_lens.data_ptr()
    _launch("fa_cache_append", _lib.fa_cache_append, index, stream, cache._ref, kh, vh, qh, oh, pos, ref, new, T)


def fa_decode_paged_workspace_bytes(cache: KVCache, Hq: int, Tq: int = 1, accumulate: bool = False) -> int:
    """Workspace of fa_decode_paged for these sizes, 0 for sizes that it refuses."""
    return int(_lib.fa_decode_paged_workspace_bytes(cache.B, Hq, cache.Hkv, Tq, cache.max_pages, cache.page_size,
                                                    cache.d, int(bool(accumulate))))


def fa_decode_paged(cache: KVCache, q, o, lse, scale: float, workspace: torch.Tensor, causal: bool = True,
                    accumulate: bool = False, stream=None) -> None:
    """O and lse of q [B, Hq, Tq, d] (the last Tq tokens of every sequence) over the cache; with
    `accumulate`, cache.weight grows by each entry's attention probabilities."""
    st = _fast.decode(cache._ref, cache._index, q, o, lse, scale, workspace, causal, accumulate, stream)
    if st != FA_OK:
        _again(st, "fa_decode_paged", _decode, cache, q, o, lse, scale, workspace, causal, accumulate, stream)


def _decode(cache, q, o, lse, scale, workspace, causal, accumulate, stream) -> None:
    dev, index, shape = cache.device, cache._index, q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B, Hq, Tq, d]")
    _, Hq, Tq, _ = shape
    bf16 = torch.bfloat16
    if not (shape[0] == cache.B and shape[3] == cache.d and o.shape == shape and lse.shape == shape[:3] and
            q.dtype is bf16 and o.dtype is bf16 and lse.dtype is torch.float32 and
            q.get_device() == index and o.get_device() == index and lse.get_device() == index and
            q.is_contiguous() and o.is_contiguous() and lse.is_contiguous()):
        shape = (cache.B, Hq, Tq, cache.d)
        _need(q, "q", bf16, shape, dev)
        _need(o, "o", bf16, shape, dev)
        _need(lse, "lse", torch.float32, shape[:3], dev)
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous tensor on the same device")
    _launch("fa_decode_paged", _lib.fa_decode_paged, index, stream, cache._ref, q.data_ptr(), o.data_ptr(),
            lse.data_ptr(), Hq, Tq, int(bool(causal)), scale, int(bool(accumulate)), workspace.data_ptr(),
            workspace.nbytes)


def attention_decode_paged(cache: KVCache, q, scale: float, causal: bool = True, accumulate: bool = False,
                           workspace=None, stream=None):
    """Allocates O, lse (and the workspace if not given) and runs fa_decode_paged."""
    if q.dim() != 4:
        raise ValueError("q must be [B, Hq, Tq, d]")
    specs = [(q.shape, q.dtype), (q.shape[:3], torch.float32)]
    if workspace is None:
        n = fa_decode_paged_workspace_bytes(cache, q.shape[1], q.shape[2], accumulate)
        specs.append(((max(n, 256),), torch.uint8))
    o, lse, *own = _empties(stream, q.device, *specs)
    fa_decode_paged(cache, q, o, lse, scale, own[0] if own else workspace, causal, accumulate, stream)
    return o, lse


def fa_cache_evict(cache: KVCache, budget: int, weight_out=None, order_out=None, lens_out=None, kept=None,
                   n_first: int = 0, n_recent: int = 0, stream=None) -> torch.Tensor:
    """Keeps min(lens, budget) entries of each sequence and KV head: the first n_first and last
    n_recent tokens, then those of the largest cache.weight.  K and V rows move in place; weight,
    order and lens are updated in place unless outputs are given.  Returns kept, int32
    [B, Hkv, budget]: the old slot of each entry, -1 behind the new length."""
    if cache.weight is None:
        raise ValueError("the cache has no weight")
    weight_out = cache.weight if weight_out is None else weight_out
    order_out = cache.order if order_out is None else order_out
    lens_out = cache.lens if lens_out is None else lens_out
    if kept is None:
        kept, = _empties(stream, cache.device, ((cache.B, cache.Hkv, max(int(budget), 0)), torch.int32))
    st = _fast.evict(cache._ref, cache._index, budget, weight_out, order_out, lens_out, kept, n_first, n_recent, stream)
    if st != FA_OK:
        _again(st, "fa_cache_evict", _evict, cache, budget, weight_out, order_out, lens_out, kept, n_first, n_recent, stream)
    return kept


def _evict(cache, budget, weight_out, order_out, lens_out, kept, n_first, n_recent, stream) -> None:
    dev = cache.device
    _need(weight_out, "weight_out", torch.float32, cache.weight.shape, dev)
    if (order_out is None) != (cache.order is None):
        raise ValueError("order_out: needed with a cache that has an order and only with it")
    if order_out is not None:
        _need(order_out, "order_out", torch.int32, cache.weight.shape, dev)
    _need(lens_out, "lens_out", torch.int32, (cache.B,), dev)
    _need(kept, "kept", torch.int32, (cache.B, cache.Hkv, budget), dev)
    _launch("fa_cache_evict", _lib.fa_cache_evict, cache._index, stream, cache._ref, int(budget), int(n_first),
            int(n_recent), weight_out.data_ptr(), _ptr(order_out), lens_out.data_ptr(), kept.data_ptr())
