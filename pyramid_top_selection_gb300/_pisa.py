"""ctypes binding of libpisa.so: argument marshalling only.

Every step of the PISA hot path runs in the library's CUDA kernels. PyTorch supplies the
device memory (outputs and workspaces are torch tensors), the current CUDA stream and
the dtype/shape bookkeeping. There is no fallback: if the library cannot be loaded, every
call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpisa.so")

PISA_OK, PISA_EINVAL, PISA_EUNSUPPORTED, PISA_EWORKSPACE, PISA_ECUDA, PISA_ETIMEOUT = range(6)
WINDOW_FWD, WINDOW_BWD = range(2)
DOC_FWD, DOC_BWD = range(2)
OP_SELECT, OP_SELECT_FLAT, OP_ATTN_FWD, OP_ATTN_BWD, OP_SELECT_MEAN, OP_SELECT_MEANVAR = range(6)
STATUS_POS_RANGE, STATUS_TIMEOUT = 1, 2
MAX_LEVELS = 32
ABI_VERSION = 6          # PISA_VERSION of the header these argument lists follow

EXPORTS = (
    "pisa_version", "pisa_last_error", "pisa_pyramid_layout", "pisa_workspace_size",
    "pisa_build_pyramid", "pisa_select", "pisa_select_flat", "pisa_sparse_attn_fwd",
    "pisa_sparse_attn_bwd", "pisa_decode_pyramid_layout", "pisa_decode_build_pyramid",
    "pisa_decode_step", "pisa_profile_start", "pisa_profile_stop", "pisa_profile_read",
    "pisa_select_noalloc", "pisa_select_mean", "pisa_set_wait_limit", "pisa_test_stall",
    "pisa_select_meanvar", "pisa_window_workspace_size", "pisa_window_attn_fwd", "pisa_window_attn_bwd",
    "pisa_window_decode_step", "pisa_qk_norm_rope", "pisa_qk_norm_rope_workspace_size", "pisa_qk_norm_rope_bwd",
    "pisa_doc_workspace_size", "pisa_doc_attn_fwd", "pisa_doc_attn_bwd", "pisa_paged_append",
    "pisa_paged_workspace_size", "pisa_paged_attn",
)


class PisaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"PISA error {code}: {msg}")
        self.code = code


class Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "N", "Hq", "Hkv", "d", "C", "K", "g", "qtile")] + \
               [("scale", ctypes.c_float), ("per_head", ctypes.c_int32)]


class ProfileEntry(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int32), ("total_ms", ctypes.c_double)]


class DecodeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Ncap", "Hq", "Hkv", "d", "C", "K", "g")] + \
               [("scale", ctypes.c_float)]


class WindowShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Nq", "N", "Hq", "Hkv", "d", "window", "sinks")] + \
               [("scale", ctypes.c_float)] + \
               [(n, ctypes.c_int32) for n in ("q_stride", "k_stride", "v_stride")]


class WindowDecodeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Ncap", "Hq", "Hkv", "d", "window", "sinks")] + \
               [("scale", ctypes.c_float)]


class RopeShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "N", "Hq", "Hkv", "d", "rot", "interleaved", "norm")] + \
               [("eps", ctypes.c_float), ("rot_scale", ctypes.c_float)] + \
               [(n, ctypes.c_int32) for n in ("q_stride", "k_stride")]


class DocShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "Hq", "Hkv", "d", "n_docs", "max_len")] + \
               [("scale", ctypes.c_float), ("cap", ctypes.c_float)] + \
               [(n, ctypes.c_int32) for n in ("q_stride", "k_stride", "v_stride")]


class PagedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "d", "n_pages", "page", "max_pages", "bits", "nq")] + \
               [("scale", ctypes.c_float), ("cap", ctypes.c_float)]


class _PagedCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "k_amp", "v_amp")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libpisa.so (built by pyramid_top_selection_gb300.build) or raise."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libpisa.so not built at {LIB_PATH}: run pyramid_top_selection_gb300/build.py")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        P = ctypes.POINTER
        L.pisa_version.restype = ctypes.c_int
        if L.pisa_version() != ABI_VERSION:
            raise ImportError(f"libpisa.so has ABI version {L.pisa_version()}, this binding needs {ABI_VERSION}: "
                              "rebuild with pyramid_top_selection_gb300/build.py")
        L.pisa_last_error.restype = ctypes.c_char_p
        L.pisa_pyramid_layout.argtypes = [P(Shape), P(i32), P(i64), P(i64)]
        L.pisa_workspace_size.argtypes = [P(Shape), ctypes.c_int, P(sz)]
        L.pisa_build_pyramid.argtypes = [P(Shape), vp, vp, vp]
        L.pisa_select.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.pisa_select_flat.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, sz, vp]
        L.pisa_select_mean.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, sz, vp]
        L.pisa_select_meanvar.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, sz, vp]
        L.pisa_sparse_attn_fwd.argtypes = [P(Shape), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.pisa_sparse_attn_bwd.argtypes = [P(Shape)] + [vp] * 10 + [vp, sz, vp]
        L.pisa_decode_pyramid_layout.argtypes = [P(DecodeShape), P(i32), P(i64), P(i64)]
        L.pisa_decode_build_pyramid.argtypes = [P(DecodeShape), vp, vp, vp, vp]
        L.pisa_decode_step.argtypes = [P(DecodeShape)] + [vp] * 11 + [vp]
        L.pisa_window_workspace_size.argtypes = [P(WindowShape), ctypes.c_int, P(sz)]
        L.pisa_window_attn_fwd.argtypes = [P(WindowShape)] + [vp] * 7 + [sz, vp]
        L.pisa_window_attn_bwd.argtypes = [P(WindowShape)] + [vp] * 11 + [sz, vp]
        L.pisa_window_decode_step.argtypes = [P(WindowDecodeShape)] + [vp] * 10
        L.pisa_qk_norm_rope.argtypes = [P(RopeShape)] + [vp] * 9
        L.pisa_qk_norm_rope_workspace_size.argtypes = [P(RopeShape), P(sz)]
        L.pisa_qk_norm_rope_bwd.argtypes = [P(RopeShape)] + [vp] * 13 + [sz, vp]
        L.pisa_doc_workspace_size.argtypes = [P(DocShape), ctypes.c_int, P(sz)]
        L.pisa_doc_attn_fwd.argtypes = [P(DocShape)] + [vp] * 9 + [sz, vp]
        L.pisa_doc_attn_bwd.argtypes = [P(DocShape)] + [vp] * 13 + [sz, vp]
        L.pisa_paged_append.argtypes = [P(PagedShape), P(_PagedCache), P(RopeShape)] + [vp] * 3 + [i32] + [vp] * 9
        L.pisa_paged_workspace_size.argtypes = [P(PagedShape), P(sz)]
        L.pisa_paged_attn.argtypes = [P(PagedShape), P(_PagedCache)] + [vp] * 7 + [sz, vp]
        L.pisa_profile_start.argtypes = []
        L.pisa_profile_stop.argtypes = []
        L.pisa_profile_read.argtypes = [P(ProfileEntry), i32, P(i32)]
        L.pisa_set_wait_limit.argtypes = [ctypes.c_uint64]
        L.pisa_test_stall.argtypes = [ctypes.c_int]
        for f in EXPORTS:
            if f not in ("pisa_version", "pisa_last_error"):
                getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != PISA_OK:
        raise PisaError(rc, lib().pisa_last_error().decode())


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def make_shape(B, N, Hq, Hkv, d, C=64, K=16, g=2, qtile=1, scale=0.0, per_head=False) -> Shape:
    return Shape(B, N, Hq, Hkv, d, C, K, g, qtile, float(scale), 1 if per_head else 0)


def shape_of(Q: torch.Tensor, Kt: torch.Tensor, C=64, K=16, g=2, qtile=1, scale=0.0, per_head=False) -> Shape:
    B, N, Hq, d = Q.shape
    return make_shape(B, N, Hq, Kt.shape[2], d, C, K, g, qtile, scale, per_head)


def _units(shape: Shape) -> int:
    """Selection units per batch: the KV heads, or the query heads of a per-head selection."""
    return shape.Hq if shape.per_head else shape.Hkv


def pyramid_layout(shape: Shape):
    n = ctypes.c_int32()
    off = (ctypes.c_int64 * MAX_LEVELS)()
    nodes = ctypes.c_int64()
    _check(lib().pisa_pyramid_layout(ctypes.byref(shape), ctypes.byref(n), off, ctypes.byref(nodes)))
    return n.value, list(off[:n.value]), nodes.value


def workspace_size(shape: Shape, op: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().pisa_workspace_size(ctypes.byref(shape), op, ctypes.byref(b)))
    return b.value


def workspace(shape: Shape, op: int, device) -> torch.Tensor:
    """A device workspace of the size `op` needs (uint8 tensor)."""
    return _workspace(shape, op, device)


def _workspace(shape: Shape, op: int, device) -> torch.Tensor:
    return torch.empty(max(workspace_size(shape, op), 256), dtype=torch.uint8, device=device)


def _need(t: torch.Tensor, dtype, name: str) -> None:
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor (got {t.dtype}, "
                         f"cuda={t.is_cuda}, contiguous={t.is_contiguous()})")


def build_pyramid(Kt: torch.Tensor, shape: Shape, out: torch.Tensor | None = None) -> torch.Tensor:
    """fp32 key sums [B, Hkv, nodes, d] of K [B, N, Hkv, d] bf16."""
    _need(Kt, torch.bfloat16, "K")
    _, _, nodes = pyramid_layout(shape)
    pyr = out if out is not None else torch.empty(shape.B, shape.Hkv, nodes, shape.d, dtype=torch.float32,
                                                  device=Kt.device)
    _check(lib().pisa_build_pyramid(ctypes.byref(shape), _ptr(Kt), _ptr(pyr), _stream(Kt.device)))
    return pyr


def _select_out(Q, shape, want_score, idx, score):
    dev = Q.device
    if idx is None:
        idx = torch.empty(shape.B, _units(shape), shape.N, shape.K, dtype=torch.int32, device=dev)
    if score is None and want_score:
        score = torch.empty(shape.B, _units(shape), shape.N, shape.K, dtype=torch.float32, device=dev)
    return idx, score


def _select_in(Q, Kt, pyr):
    _need(Q, torch.bfloat16, "Q")
    _need(Kt, torch.bfloat16, "K")
    _need(pyr, torch.float32, "pyr_sum")


def select(Q, Kt, pyr, shape: Shape, ws=None, want_score=True, idx=None, score=None,
           want_head_lse=False, head_lse=None):
    """Pyramid Top-K selection: idx [B,Hkv,N,K] int32 (ascending, -1 pad), score fp32.

    With want_head_lse (or a head_lse buffer) also returns the per-head leaf LSEs
    [B,Hq,N,K] fp32 that sparse_attn_fwd takes to skip its normalisation pass."""
    _select_in(Q, Kt, pyr)
    dev = Q.device
    idx, score = _select_out(Q, shape, want_score, idx, score)
    if head_lse is None and want_head_lse:
        head_lse = torch.empty(shape.B, shape.Hq, shape.N, shape.K, dtype=torch.float32, device=dev)
    if ws is None:
        ws = _workspace(shape, OP_SELECT, dev)
    _check(lib().pisa_select(ctypes.byref(shape), _ptr(Q), _ptr(Kt), _ptr(pyr), _ptr(idx), _ptr(score),
                             _ptr(head_lse), _ptr(ws), ws.numel(), _stream(dev)))
    if head_lse is not None:
        return idx, score, head_lse
    return idx, score


def select_flat(Q, Kt, pyr, shape: Shape, ws=None, want_score=True, idx=None, score=None):
    """Flat O(N^2/C) block selection (comparator)."""
    _select_in(Q, Kt, pyr)
    dev = Q.device
    idx, score = _select_out(Q, shape, want_score, idx, score)
    if ws is None:
        ws = _workspace(shape, OP_SELECT_FLAT, dev)
    _check(lib().pisa_select_flat(ctypes.byref(shape), _ptr(Q), _ptr(Kt), _ptr(pyr), _ptr(idx), _ptr(score),
                                  _ptr(ws), ws.numel(), _stream(dev)))
    return idx, score


def select_mean(Q, Kt, pyr, shape: Shape, ws=None, want_score=True, idx=None, score=None):
    """PISA-1 ablation selection: the pyramid descent with every block scored by its mean key."""
    _select_in(Q, Kt, pyr)
    dev = Q.device
    idx, score = _select_out(Q, shape, want_score, idx, score)
    if ws is None:
        ws = _workspace(shape, OP_SELECT_MEAN, dev)
    _check(lib().pisa_select_mean(ctypes.byref(shape), _ptr(Q), _ptr(Kt), _ptr(pyr), _ptr(idx), _ptr(score),
                                  _ptr(ws), ws.numel(), _stream(dev)))
    return idx, score


def select_meanvar(Q, Kt, pyr, shape: Shape, ws=None, want_score=True, idx=None, score=None):
    """PISA-2 ablation selection: the pyramid descent with every block scored by mean + variance."""
    _select_in(Q, Kt, pyr)
    dev = Q.device
    idx, score = _select_out(Q, shape, want_score, idx, score)
    if ws is None:
        ws = _workspace(shape, OP_SELECT_MEANVAR, dev)
    _check(lib().pisa_select_meanvar(ctypes.byref(shape), _ptr(Q), _ptr(Kt), _ptr(pyr), _ptr(idx), _ptr(score),
                                     _ptr(ws), ws.numel(), _stream(dev)))
    return idx, score


def sparse_attn_fwd(Q, Kt, V, idx, shape: Shape, ws=None, out=None, lse=None, head_lse=None):
    """Causal attention over the selected leaves: O [B,N,Hq,d] bf16, lse [B,Hq,N] fp32.

    head_lse: the selection's per-head leaf LSEs for these idx (optional)."""
    for t, n in ((Q, "Q"), (Kt, "K"), (V, "V")):
        _need(t, torch.bfloat16, n)
    _need(idx, torch.int32, "idx")
    if head_lse is not None:
        _need(head_lse, torch.float32, "head_lse")
    dev = Q.device
    O = out if out is not None else torch.empty_like(Q)
    lse = lse if lse is not None else torch.empty(shape.B, shape.Hq, shape.N, dtype=torch.float32, device=dev)
    if ws is None:
        ws = _workspace(shape, OP_ATTN_FWD, dev)
    _check(lib().pisa_sparse_attn_fwd(ctypes.byref(shape), _ptr(Q), _ptr(Kt), _ptr(V), _ptr(idx),
                                      _ptr(head_lse), _ptr(O), _ptr(lse), _ptr(ws), ws.numel(), _stream(dev)))
    return O, lse


def sparse_attn_bwd(Q, Kt, V, O, lse, dO, idx, shape: Shape, ws=None):
    """Gradients through the selected attention only: dQ, dK, dV (bf16)."""
    for t, n in ((Q, "Q"), (Kt, "K"), (V, "V"), (O, "O"), (dO, "dO")):
        _need(t, torch.bfloat16, n)
    _need(lse, torch.float32, "lse")
    _need(idx, torch.int32, "idx")
    dev = Q.device
    dQ, dK, dV = torch.empty_like(Q), torch.empty_like(Kt), torch.empty_like(V)
    if ws is None:
        ws = _workspace(shape, OP_ATTN_BWD, dev)
    _check(lib().pisa_sparse_attn_bwd(ctypes.byref(shape), _ptr(Q), _ptr(Kt), _ptr(V), _ptr(O),
                                      _ptr(lse), _ptr(dO), _ptr(idx), _ptr(dQ), _ptr(dK), _ptr(dV),
                                      _ptr(ws), ws.numel(), _stream(dev)))
    return dQ, dK, dV


def make_decode_shape(B, Ncap, Hq, Hkv, d, C=64, K=16, g=2, scale=0.0) -> DecodeShape:
    return DecodeShape(B, Ncap, Hq, Hkv, d, C, K, g, float(scale))


def decode_pyramid_layout(shape: DecodeShape):
    n = ctypes.c_int32()
    off = (ctypes.c_int64 * MAX_LEVELS)()
    nodes = ctypes.c_int64()
    _check(lib().pisa_decode_pyramid_layout(ctypes.byref(shape), ctypes.byref(n), off, ctypes.byref(nodes)))
    return n.value, list(off[:n.value]), nodes.value


def decode_build_pyramid(Kcache, length, shape: DecodeShape) -> torch.Tensor:
    """Cached pyramid over Ncap from the first length[b] keys of each sequence."""
    _need(Kcache, torch.bfloat16, "Kcache")
    _need(length, torch.int32, "len")
    _, _, nodes = decode_pyramid_layout(shape)
    pyr = torch.empty(shape.B, shape.Hkv, nodes, shape.d, dtype=torch.float32, device=Kcache.device)
    _check(lib().pisa_decode_build_pyramid(ctypes.byref(shape), _ptr(Kcache), _ptr(length), _ptr(pyr),
                                           _stream(Kcache.device)))
    return pyr


def decode_step(shape: DecodeShape, pos, Kcache, Vcache, pyr, q, k_new, v_new, o=None, idx=None,
                score=None, status=None, rope: Rope | None = None):
    """One fused decode step (append + ancestor update + select + attend) for all sequences.

    With `rope`, q and k_new are raw projections (slices of a fused one, if need be): they are normed and
    rotated at `pos` first (qk_norm_rope, one more launch). What the step itself reads is contiguous."""
    dev = q.device
    _need(v_new, torch.bfloat16, "v_new")
    if rope is not None:
        q, k_new = _ready_token(rope, q, k_new, pos)
    _need(q, torch.bfloat16, "q")
    _need(k_new, torch.bfloat16, "k_new")
    o = o if o is not None else torch.empty_like(q)
    idx = idx if idx is not None else torch.empty(shape.B, shape.Hkv, shape.K, dtype=torch.int32, device=dev)
    status = status if status is not None else torch.zeros(4, dtype=torch.int32, device=dev)
    _check(lib().pisa_decode_step(ctypes.byref(shape), _ptr(pos), _ptr(Kcache), _ptr(Vcache), _ptr(pyr),
                                  _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(o), _ptr(idx), _ptr(score),
                                  _ptr(status), _stream(dev)))
    return o, idx, score, status


# ---------------------------------------------------------------------------------------
# Sliding-window attention with sinks; query/key norm with rotation

def _on(dev, fn, *args) -> None:
    """Call fn(*args, stream) on dev's current stream, with dev the current device."""
    if dev.type != "cuda":
        raise ValueError(f"the tensors must be CUDA tensors (got {dev})")
    stream = torch._C._cuda_getCurrentRawStream(dev.index)   # current_stream(dev).cuda_stream without its objects
    if dev.index == torch._C._cuda_getDevice():              # torch.cuda.current_device() of a context that exists
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != PISA_OK:
        _check(rc)


def _need_shaped(t, dtype, size, dev, name: str) -> None:
    """A contiguous tensor of this type and size on `dev` (the other tensors' device)."""
    if t.dtype is not dtype or t.shape != size or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(size)} on {dev} "
                         f"(got {t.dtype}, {tuple(t.shape)}, {t.device}, contiguous={t.is_contiguous()})")


def _token_stride(t: torch.Tensor, name: str) -> int:
    """Elements between consecutive tokens of [B, N, H, d] (0: contiguous), d and the heads contiguous."""
    if t.is_contiguous():
        return 0
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, N, H, d] (got {tuple(t.shape)})")
    B, N, H, d = t.shape
    sb, sn, sh, sd = t.stride()
    step = sn if N > 1 else sb if B > 1 else H * d
    if (d > 1 and sd != 1) or (H > 1 and sh != d) or (N > 1 and B > 1 and sb != N * sn) or not H * d <= step < 1 << 31:
        raise ValueError(f"{name} must have contiguous heads and evenly spaced tokens (strides {tuple(t.stride())})")
    return step if B * N > 1 else 0


def _need_tokens(t, size, stride: int, dev, name: str) -> None:
    if t.dtype is not torch.bfloat16 or t.shape != size or t.device != dev:
        raise ValueError(f"{name} must be a bfloat16 tensor {tuple(size)} on {dev} "
                         f"(got {t.dtype}, {tuple(t.shape)}, {t.device})")
    if stride or not t.is_contiguous():
        step, row = _token_stride(t, name), size[2] * size[3]
        if size[0] * size[1] > 1 and (step or row) != (stride or row):
            raise ValueError(f"{name} has strides {tuple(t.stride())}, the shape says {stride} elements a token")


def _need_ws(ws, dev) -> None:
    if ws.dtype is not torch.uint8 or ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on {dev} (got {ws.dtype}, {ws.device})")


def _need_int32(**sizes) -> None:
    """Sizes have to fit the C struct's int32 (ctypes would keep their low 32 bits)."""
    bad = [f"{n}={v}" for n, v in sizes.items() if not -0x80000000 <= v <= 0x7fffffff]
    if bad:
        raise ValueError(f"sizes must fit 32 bits (got {', '.join(bad)})")


def make_window_shape(B, Nq, N, Hq, Hkv, d, window, sinks=0, scale=0.0, q_stride=0, k_stride=0,
                      v_stride=0) -> WindowShape:
    if not 0 <= B | Nq | N | Hq | Hkv | d | window | sinks | q_stride | k_stride | v_stride <= 0x7fffffff:
        _need_int32(B=B, Nq=Nq, N=N, Hq=Hq, Hkv=Hkv, d=d, window=window, sinks=sinks, q_stride=q_stride, k_stride=k_stride,
                    v_stride=v_stride)
    return WindowShape(B, Nq, N, Hq, Hkv, d, window, sinks, float(scale), q_stride, k_stride, v_stride)


def window_shape_of(Q, K, V, window, sinks=0, scale=0.0) -> WindowShape:
    """The shape of Q [B,Nq,Hq,d], K, V [B,N,Hkv,d], which may be slices of a fused projection."""
    B, Nq, Hq, d = Q.shape
    return make_window_shape(B, Nq, K.shape[1], Hq, K.shape[2], d, window, sinks, scale, _token_stride(Q, "Q"),
                             _token_stride(K, "K"), _token_stride(V, "V"))


def window_workspace_size(shape: WindowShape, op: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().pisa_window_workspace_size(ctypes.byref(shape), op, ctypes.byref(b)))
    return b.value


def window_workspace(shape: WindowShape, op: int, device) -> torch.Tensor:
    """A device workspace of the size `op` (WINDOW_FWD, WINDOW_BWD) needs (uint8 tensor)."""
    return torch.empty(window_workspace_size(shape, op), dtype=torch.uint8, device=device)


def _need_window(Q, K, V, shape, lens) -> None:
    dev = Q.device
    kv = (shape.B, shape.N, shape.Hkv, shape.d)
    _need_tokens(Q, (shape.B, shape.Nq, shape.Hq, shape.d), shape.q_stride, dev, "Q")
    _need_tokens(K, kv, shape.k_stride, dev, "K")
    _need_tokens(V, kv, shape.v_stride, dev, "V")
    if lens is not None:
        _need_shaped(lens, torch.int32, (shape.B,), dev, "lens")


def window_attn_fwd(Q, K, V, shape: WindowShape, lens=None, ws=None, out=None, lse=None):
    """Causal sliding-window attention with sinks: O [B,Nq,Hq,d] bf16, lse [B,Hq,Nq] fp32.

    lens: valid tokens of each sequence, [B] int32 (None: all); rows past them get O = 0, lse = -inf.
    ws: a workspace whose status word the call writes (None: a timeout shows in the outputs only)."""
    _need_window(Q, K, V, shape, lens)
    dev = Q.device
    size = (shape.B, shape.Nq, shape.Hq, shape.d)
    if out is None:
        out = torch.empty(size, dtype=torch.bfloat16, device=dev)
    else:
        _need_shaped(out, torch.bfloat16, size, dev, "out")
    if lse is None:
        lse = torch.empty((shape.B, shape.Hq, shape.Nq), dtype=torch.float32, device=dev)
    else:
        _need_shaped(lse, torch.float32, (shape.B, shape.Hq, shape.Nq), dev, "lse")
    if ws is not None:
        _need_ws(ws, dev)
    _on(dev, lib().pisa_window_attn_fwd, ctypes.byref(shape), Q.data_ptr(), K.data_ptr(), V.data_ptr(), _ptr(lens),
        out.data_ptr(), lse.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel())
    return out, lse


def window_attn_bwd(Q, K, V, O, lse, dO, shape: WindowShape, lens=None, ws=None):
    """Gradients of window_attn_fwd: dQ, dK, dV (bf16), from its O and lse."""
    _need_window(Q, K, V, shape, lens)
    dev = Q.device
    size = (shape.B, shape.Nq, shape.Hq, shape.d)
    _need_shaped(O, torch.bfloat16, size, dev, "O")
    _need_shaped(dO, torch.bfloat16, size, dev, "dO")
    _need_shaped(lse, torch.float32, (shape.B, shape.Hq, shape.Nq), dev, "lse")
    dQ = torch.empty(size, dtype=torch.bfloat16, device=dev)
    dK = torch.empty((shape.B, shape.N, shape.Hkv, shape.d), dtype=torch.bfloat16, device=dev)
    dV = torch.empty_like(dK)
    if ws is None:
        ws = window_workspace(shape, WINDOW_BWD, dev)
    _need_ws(ws, dev)
    _on(dev, lib().pisa_window_attn_bwd, ctypes.byref(shape), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
        lse.data_ptr(), dO.data_ptr(), _ptr(lens), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), ws.data_ptr(),
        ws.numel())
    return dQ, dK, dV


def make_window_decode_shape(B, Ncap, Hq, Hkv, d, window, sinks=0, scale=0.0) -> WindowDecodeShape:
    if not 0 <= B | Ncap | Hq | Hkv | d | window | sinks <= 0x7fffffff:
        _need_int32(B=B, Ncap=Ncap, Hq=Hq, Hkv=Hkv, d=d, window=window, sinks=sinks)
    return WindowDecodeShape(B, Ncap, Hq, Hkv, d, window, sinks, float(scale))


def window_decode_step(shape: WindowDecodeShape, pos, Kcache, Vcache, q, k_new, v_new, o=None, lse=None,
                       status=None, rope: Rope | None = None):
    """One decode step of the window attention: append at the slot of pos, attend. Returns o, lse, status.

    The cache rolls once positions reach its capacity (see pisa.h). With `rope`, q and k_new are raw
    projections (slices of a fused one, if need be): they are normed and rotated at `pos` first
    (qk_norm_rope, one more launch). What the step itself reads is contiguous."""
    dev = q.device
    B, H = shape.B, (shape.B, shape.Hkv, shape.d)
    cache = (B, shape.Ncap, shape.Hkv, shape.d)
    _need_shaped(pos, torch.int32, (B,), dev, "pos")
    _need_shaped(Kcache, torch.bfloat16, cache, dev, "Kcache")
    _need_shaped(Vcache, torch.bfloat16, cache, dev, "Vcache")
    if rope is not None:
        q, k_new = _ready_token(rope, q, k_new, pos)
    _need_shaped(q, torch.bfloat16, (B, shape.Hq, shape.d), dev, "q")
    _need_shaped(k_new, torch.bfloat16, H, dev, "k_new")
    _need_shaped(v_new, torch.bfloat16, H, dev, "v_new")
    if o is None:
        o = torch.empty_like(q)
    else:
        _need_shaped(o, torch.bfloat16, (B, shape.Hq, shape.d), dev, "o")
    if lse is None:
        lse = torch.empty((B, shape.Hq), dtype=torch.float32, device=dev)
    else:
        _need_shaped(lse, torch.float32, (B, shape.Hq), dev, "lse")
    if status is None:
        status = torch.zeros(4, dtype=torch.int32, device=dev)
    elif status.dtype is not torch.int32 or status.device != dev or status.numel() < 1:
        raise ValueError(f"status must be an int32 tensor on {dev} (got {status.dtype}, {status.device})")
    _on(dev, lib().pisa_window_decode_step, ctypes.byref(shape), pos.data_ptr(), Kcache.data_ptr(), Vcache.data_ptr(),
        q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), o.data_ptr(), lse.data_ptr(), status.data_ptr())
    return o, lse, status


def make_rope_shape(B, N, Hq, Hkv, d, rot, interleaved=False, norm=True, eps=1e-6, rot_scale=1.0, q_stride=0,
                    k_stride=0) -> RopeShape:
    if not 0 <= B | N | Hq | Hkv | d | rot | q_stride | k_stride <= 0x7fffffff:
        _need_int32(B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, rot=rot, q_stride=q_stride, k_stride=k_stride)
    return RopeShape(B, N, Hq, Hkv, d, rot, 1 if interleaved else 0, 1 if norm else 0, float(eps), float(rot_scale),
                     q_stride, k_stride)


def rope_shape_of(Q, K, rot, interleaved=False, norm=True, eps=1e-6, rot_scale=1.0) -> RopeShape:
    """The shape of Q [B,N,Hq,d], K [B,N,Hkv,d], which may be slices of a fused projection."""
    B, N, Hq, d = Q.shape
    return make_rope_shape(B, N, Hq, K.shape[2], d, rot, interleaved, norm, eps, rot_scale, _token_stride(Q, "Q"),
                           _token_stride(K, "K"))


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained_len: int = 0, slow: float = 1.0, fast: float = 32.0):
    """Rotary frequencies (inv_freq [rot/2] fp32 on the CPU, radians per position) and rot_scale.

    scaling, for contexts `factor` times longer than the trained_len tokens of training:
      "none"    base ** (-2 c / rot)
      "linear"  every frequency divided by factor (position interpolation)
      "ntk"     the base raised by factor ** (rot / (rot - 2)): the lowest frequency is divided by
                factor, the highest stays
      "yarn"    by parts (YaRN): pairs that turn more than `fast` times within trained_len stay, those
                under `slow` turns are divided by factor, a linear ramp in the turns between, as the method's
                paper states it; and rot_scale = 0.1 ln(factor) + 1. (A model trained with a ramp over
                the pairs' index between rounded bounds has other frequencies in between: pass its own as
                inv_freq.)
    """
    if rot < 2 or rot % 2 or factor < 1 or base <= 0:
        raise ValueError(f"rot={rot} must be even and positive, factor={factor} at least 1, base={base} positive")
    c = torch.arange(0, rot, 2, dtype=torch.float64) / rot
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("ntk scaling needs rot >= 4")
        base = base * factor ** (rot / (rot - 2))
    f = base ** -c
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if trained_len < 1 or not 0 <= slow < fast:
            raise ValueError(f"yarn scaling needs trained_len and 0 <= slow < fast (got {trained_len}, {slow}, {fast})")
        keep = ((trained_len * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f / factor * (1 - keep) + f * keep
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(torch.float32), 0.1 * math.log(factor) + 1 if scaling == "yarn" and factor > 1 else 1.0


class Rope(NamedTuple):
    """What turns raw query and key projections into the heads the attentions take: device tensors
    (inv_freq [rot/2] fp32, the norm's weights [d] fp32 or None) and pisa_rope_shape_t's settings."""
    inv_freq: torch.Tensor | None
    rot: int
    interleaved: bool = False
    norm: bool = True
    eps: float = 1e-6
    rot_scale: float = 1.0
    q_weight: torch.Tensor | None = None
    k_weight: torch.Tensor | None = None


def _ready_token(rope: Rope, q, k_new, pos):
    """q [B,Hq,d] and k_new [B,Hkv,d] of one token per sequence, normed and rotated at pos [B]."""
    q4, k4 = q[:, None], k_new[:, None]
    shape = rope_shape_of(q4, k4, rope.rot, rope.interleaved, rope.norm, rope.eps, rope.rot_scale)
    q4, k4 = qk_norm_rope(q4, k4, rope.inv_freq, shape, rope.q_weight, rope.k_weight, pos[:, None])
    return q4[:, 0], k4[:, 0]


def _need_rope(Q, K, inv_freq, shape, q_weight, k_weight, pos) -> None:
    dev = Q.device
    _need_tokens(Q, (shape.B, shape.N, shape.Hq, shape.d), shape.q_stride, dev, "Q")
    _need_tokens(K, (shape.B, shape.N, shape.Hkv, shape.d), shape.k_stride, dev, "K")
    if inv_freq is not None:
        _need_shaped(inv_freq, torch.float32, (shape.rot // 2,), dev, "inv_freq")
    if q_weight is not None:
        _need_shaped(q_weight, torch.float32, (shape.d,), dev, "q_weight")
    if k_weight is not None:
        _need_shaped(k_weight, torch.float32, (shape.d,), dev, "k_weight")
    if pos is not None:
        _need_shaped(pos, torch.int32, (shape.B, shape.N), dev, "pos")


def qk_norm_rope(Q, K, inv_freq, shape: RopeShape, q_weight=None, k_weight=None, pos=None, q_out=None, k_out=None):
    """RMS norm of every head and rotation by position: Qr [B,N,Hq,d], Kr [B,N,Hkv,d] bf16.

    pos: [B,N] int32 (None: 0 .. N-1). q_out / k_out may be Q / K themselves where contiguous."""
    _need_rope(Q, K, inv_freq, shape, q_weight, k_weight, pos)
    dev = Q.device
    sizes = (shape.B, shape.N, shape.Hq, shape.d), (shape.B, shape.N, shape.Hkv, shape.d)
    if q_out is None:
        q_out = torch.empty(sizes[0], dtype=torch.bfloat16, device=dev)
    else:
        _need_shaped(q_out, torch.bfloat16, sizes[0], dev, "q_out")
    if k_out is None:
        k_out = torch.empty(sizes[1], dtype=torch.bfloat16, device=dev)
    else:
        _need_shaped(k_out, torch.bfloat16, sizes[1], dev, "k_out")
    _on(dev, lib().pisa_qk_norm_rope, ctypes.byref(shape), Q.data_ptr(), K.data_ptr(), _ptr(inv_freq), _ptr(q_weight),
        _ptr(k_weight), _ptr(pos), q_out.data_ptr(), k_out.data_ptr())
    return q_out, k_out


def qk_norm_rope_workspace(shape: RopeShape, device) -> torch.Tensor:
    """A device workspace for qk_norm_rope_bwd (uint8 tensor)."""
    b = ctypes.c_size_t()
    _check(lib().pisa_qk_norm_rope_workspace_size(ctypes.byref(shape), ctypes.byref(b)))
    return torch.empty(b.value, dtype=torch.uint8, device=device)


def qk_norm_rope_bwd(Q, K, dQr, dKr, inv_freq, shape: RopeShape, q_weight=None, k_weight=None, pos=None, ws=None):
    """Gradients of qk_norm_rope: dQ, dK (bf16) and the weights' dwq, dwk ([d] fp32; None without the norm)."""
    _need_rope(Q, K, inv_freq, shape, q_weight, k_weight, pos)
    dev = Q.device
    _need_shaped(dQr, torch.bfloat16, (shape.B, shape.N, shape.Hq, shape.d), dev, "dQr")
    _need_shaped(dKr, torch.bfloat16, (shape.B, shape.N, shape.Hkv, shape.d), dev, "dKr")
    dQ, dK = torch.empty_like(dQr), torch.empty_like(dKr)
    dwq = dwk = None
    if shape.norm:
        dwq = torch.empty(shape.d, dtype=torch.float32, device=dev)
        dwk = torch.empty(shape.d, dtype=torch.float32, device=dev)
    if ws is None:
        ws = qk_norm_rope_workspace(shape, dev)
    _need_ws(ws, dev)
    _on(dev, lib().pisa_qk_norm_rope_bwd, ctypes.byref(shape), Q.data_ptr(), K.data_ptr(), dQr.data_ptr(),
        dKr.data_ptr(), _ptr(inv_freq), _ptr(q_weight), _ptr(k_weight), _ptr(pos), dQ.data_ptr(), dK.data_ptr(),
        _ptr(dwq), _ptr(dwk), ws.data_ptr(), ws.numel())
    return dQ, dK, dwq, dwk


# ---------------------------------------------------------------------------------------
# Attention over packed documents; the paged key/value cache

def make_doc_shape(T, Hq, Hkv, d, n_docs, max_len=0, scale=0.0, cap=0.0, q_stride=0, k_stride=0, v_stride=0) -> DocShape:
    if not 0 <= T | Hq | Hkv | d | n_docs | max_len | q_stride | k_stride | v_stride <= 0x7fffffff:
        _need_int32(T=T, Hq=Hq, Hkv=Hkv, d=d, n_docs=n_docs, max_len=max_len, q_stride=q_stride, k_stride=k_stride,
                    v_stride=v_stride)
    return DocShape(T, Hq, Hkv, d, n_docs, max_len, float(scale), float(cap), q_stride, k_stride, v_stride)


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Elements between consecutive tokens of [T, H, d] (0: contiguous)."""
    if t.is_contiguous():
        return 0
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, H, d] (got {tuple(t.shape)})")
    T, H, d = t.shape
    step, head, one = t.stride()
    if T > 1 and head == d and one == 1 and H * d <= step < 1 << 31:
        return step
    return _token_stride(t[None], name)


def doc_shape_of(Q, K, V, starts, max_len=0, scale=0.0, cap=0.0) -> DocShape:
    """The shape of Q [T,Hq,d], K, V [T,Hkv,d] (slices of a fused projection, if need be) and starts [n_docs + 1].

    max_len: the longest document's tokens, where the caller knows them (0: not)."""
    T, Hq, d = Q.shape
    return make_doc_shape(T, Hq, K.shape[1], d, starts.numel() - 1, max_len, scale, cap, _row_stride(Q, "Q"),
                          _row_stride(K, "K"), _row_stride(V, "V"))


def doc_workspace_size(shape: DocShape, op: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().pisa_doc_workspace_size(ctypes.byref(shape), op, ctypes.byref(b)))
    return b.value


def doc_workspace(shape: DocShape, op: int, device) -> torch.Tensor:
    """A device workspace of the size `op` (DOC_FWD, DOC_BWD) needs (uint8 tensor)."""
    return torch.empty(doc_workspace_size(shape, op), dtype=torch.uint8, device=device)


def _need_rows(t, size, stride: int, dev, name: str) -> None:
    if t.dtype is not torch.bfloat16 or t.shape != size or t.device != dev:
        raise ValueError(f"{name} must be a bfloat16 tensor {tuple(size)} on {dev} "
                         f"(got {t.dtype}, {tuple(t.shape)}, {t.device})")
    if t.stride() != (stride or size[1] * size[2], size[2], 1):     # else as the shape says; sizes of one have any stride
        step, row = _row_stride(t, name), size[1] * size[2]
        if size[0] > 1 and (step or row) != (stride or row):
            raise ValueError(f"{name} has strides {tuple(t.stride())}, the shape says {stride} elements a token")


def _rows_stride(t, size, dev, name: str) -> int:
    """The stride of a tensor of this size, checked: elements between consecutive tokens (0: contiguous)."""
    stride = t.stride()
    if stride == (size[1] * size[2], size[2], 1):
        _need_rows(t, size, 0, dev, name)
        return 0
    step = _row_stride(t, name)
    _need_rows(t, size, step, dev, name)
    return step


def _need_docs(Q, K, V, starts, shape, prefix, slopes) -> None:
    dev = Q.device
    kv = (shape.T, shape.Hkv, shape.d)
    _need_rows(Q, (shape.T, shape.Hq, shape.d), shape.q_stride, dev, "Q")
    _need_rows(K, kv, shape.k_stride, dev, "K")
    _need_rows(V, kv, shape.v_stride, dev, "V")
    _need_shaped(starts, torch.int32, (shape.n_docs + 1,), dev, "starts")
    if prefix is not None:
        _need_shaped(prefix, torch.int32, (shape.n_docs,), dev, "prefix")
    if slopes is not None:
        _need_shaped(slopes, torch.float32, (shape.Hq,), dev, "slopes")


def doc_attn_fwd(Q, K, V, starts, shape: DocShape, prefix=None, slopes=None, ws=None, out=None, lse=None):
    """Attention over packed documents: O [T,Hq,d] bf16, lse [Hq,T] fp32.

    starts: the documents' first tokens and one past the last, [n_docs + 1] int32. prefix: leading tokens of each document
    that see one another, [n_docs] int32 (None: none). slopes: [Hq] fp32, what a score loses per token of
    distance (None: nothing). Rows outside every document get O = 0, lse = -inf.
    ws: a workspace whose status word the call writes (None: a timeout shows in the outputs only)."""
    _need_docs(Q, K, V, starts, shape, prefix, slopes)
    dev = Q.device
    size = (shape.T, shape.Hq, shape.d)
    if out is None:
        out = torch.empty(size, dtype=torch.bfloat16, device=dev)
    else:
        _need_shaped(out, torch.bfloat16, size, dev, "out")
    if lse is None:
        lse = torch.empty((shape.Hq, shape.T), dtype=torch.float32, device=dev)
    else:
        _need_shaped(lse, torch.float32, (shape.Hq, shape.T), dev, "lse")
    if ws is not None:
        _need_ws(ws, dev)
    else:
        n = doc_workspace_size(shape, DOC_FWD)
        if n > 256:                      # more than the status block
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _on(dev, lib().pisa_doc_attn_fwd, ctypes.byref(shape), Q.data_ptr(), K.data_ptr(), V.data_ptr(), starts.data_ptr(),
        _ptr(prefix), _ptr(slopes), out.data_ptr(), lse.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel())
    return out, lse


def doc_attn_bwd(Q, K, V, O, lse, dO, starts, shape: DocShape, prefix=None, slopes=None, ws=None):
    """Gradients of doc_attn_fwd: dQ, dK, dV (bf16), from its O and lse."""
    _need_docs(Q, K, V, starts, shape, prefix, slopes)
    dev = Q.device
    size = (shape.T, shape.Hq, shape.d)
    _need_shaped(O, torch.bfloat16, size, dev, "O")
    _need_shaped(dO, torch.bfloat16, size, dev, "dO")
    _need_shaped(lse, torch.float32, (shape.Hq, shape.T), dev, "lse")
    dQ = torch.empty(size, dtype=torch.bfloat16, device=dev)
    dK = torch.empty((shape.T, shape.Hkv, shape.d), dtype=torch.bfloat16, device=dev)
    dV = torch.empty_like(dK)
    if ws is None:
        ws = doc_workspace(shape, DOC_BWD, dev)
    _need_ws(ws, dev)
    _on(dev, lib().pisa_doc_attn_bwd, ctypes.byref(shape), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
        lse.data_ptr(), dO.data_ptr(), starts.data_ptr(), _ptr(prefix), _ptr(slopes), dQ.data_ptr(), dK.data_ptr(),
        dV.data_ptr(), ws.data_ptr(), ws.numel())
    return dQ, dK, dV


class PagedCache(NamedTuple):
    """A paged key/value cache's tensors: k, v [n_pages,Hkv,page,d] bf16, or uint8 [n_pages,Hkv,page,d/2] (two e2m1 codes a
    byte) with k_scale, v_scale [n_pages,Hkv,page,d/16] float8_e4m3fn and k_amp, v_amp [Hkv] fp32, 2^-64 to 2^64
    (None: ones)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None
    k_amp: torch.Tensor | None = None
    v_amp: torch.Tensor | None = None


def make_paged_shape(B, Hq, Hkv, d, n_pages, page, max_pages, bits=16, nq=1, scale=0.0, cap=0.0) -> PagedShape:
    if not 0 <= B | Hq | Hkv | d | n_pages | page | max_pages | bits | nq <= 0x7fffffff:
        _need_int32(B=B, Hq=Hq, Hkv=Hkv, d=d, n_pages=n_pages, page=page, max_pages=max_pages, bits=bits, nq=nq)
    return PagedShape(B, Hq, Hkv, d, n_pages, page, max_pages, bits, nq, float(scale), float(cap))


def paged_shape_of(cache: PagedCache, table, Hq, nq=1, scale=0.0, cap=0.0) -> PagedShape:
    """The shape of a cache and its page table [B, max_pages]."""
    n_pages, Hkv, page, row = cache.k.shape
    four = cache.k.dtype is torch.uint8
    return make_paged_shape(table.shape[0], Hq, Hkv, 2 * row if four else row, n_pages, page, table.shape[1],
                            4 if four else 16, nq, scale, cap)


def paged_cache(shape: PagedShape, device, k_amp=None, v_amp=None) -> PagedCache:
    """An empty cache of this shape (zeros)."""
    size = (shape.n_pages, shape.Hkv, shape.page)
    if shape.bits == 16:
        return PagedCache(*(torch.zeros(*size, shape.d, dtype=torch.bfloat16, device=device) for _ in range(2)))
    codes = (torch.zeros(*size, shape.d // 2, dtype=torch.uint8, device=device) for _ in range(2))
    scales = (torch.zeros(*size, shape.d // 16, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
    return PagedCache(*codes, *scales, k_amp, v_amp)


def _need_paged(shape, cache, table, dev):
    """The cache's C struct, its tensors checked."""
    k, v, k_scale, v_scale, k_amp, v_amp = cache
    n_pages, Hkv, page, d = shape.n_pages, shape.Hkv, shape.page, shape.d
    _need_shaped(table, torch.int32, (shape.B, shape.max_pages), dev, "table")
    if shape.bits != 4:
        _need_shaped(k, torch.bfloat16, (n_pages, Hkv, page, d), dev, "k")
        _need_shaped(v, torch.bfloat16, (n_pages, Hkv, page, d), dev, "v")
        if not k_scale is v_scale is k_amp is v_amp is None:
            raise ValueError("a cache in 16 bits has no scales")
        return _PagedCache(k.data_ptr(), v.data_ptr(), None, None, None, None)
    _need_shaped(k, torch.uint8, (n_pages, Hkv, page, d // 2), dev, "k")
    _need_shaped(v, torch.uint8, (n_pages, Hkv, page, d // 2), dev, "v")
    if k_scale is None or v_scale is None:
        raise ValueError("a cache in 4 bits needs k_scale and v_scale")
    _need_shaped(k_scale, torch.float8_e4m3fn, (n_pages, Hkv, page, d // 16), dev, "k_scale")
    _need_shaped(v_scale, torch.float8_e4m3fn, (n_pages, Hkv, page, d // 16), dev, "v_scale")
    if k_amp is not None:
        _need_shaped(k_amp, torch.float32, (Hkv,), dev, "k_amp")
    if v_amp is not None:
        _need_shaped(v_amp, torch.float32, (Hkv,), dev, "v_amp")
    return _PagedCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _ptr(k_amp), _ptr(v_amp))


def _need_status(status, dev):
    if status is None:
        return torch.zeros(4, dtype=torch.int32, device=dev)
    if status.dtype is not torch.int32 or status.device != dev or status.numel() < 1:
        raise ValueError(f"status must be an int32 tensor on {dev} (got {status.dtype}, {status.device})")
    return status


def paged_append(shape: PagedShape, cache: PagedCache, table, pos, K, V, Q=None, seq=None, rope: Rope | None = None,
                 q_out=None, status=None):
    """Appends tokens to a paged cache, keys normed and rotated on the way. Returns Qr (None without Q) and status.

    K, V [T,Hkv,d] bf16 and Q [T,Hq,d] (slices of a fused projection, if need be). pos [T] int32: each token's position in its
    sequence; seq [T] int32: its sequence, below 0 for padding (None: T / B tokens of each sequence, in order).
    rope (None: K as it is, and no Q): the norm and the rotation at pos, of K and of Q into q_out, which may be Q itself."""
    dev = K.device
    T = K.shape[0]
    if T < 1:
        raise ValueError("no tokens to append")
    B, N = (1, T) if seq is not None else (shape.B, T // shape.B)
    if B * N != T:
        raise ValueError(f"without seq the {T} tokens must be as many for each of {shape.B} sequences")
    if rope is None:
        if Q is not None:
            raise ValueError("Q is normed and rotated: it needs rope")
        rope = Rope(None, 0, norm=False)
    c = _need_paged(shape, cache, table, dev)
    kv = (T, shape.Hkv, shape.d)
    ks, vs, qs = _rows_stride(K, kv, dev, "K"), _rows_stride(V, kv, dev, "V"), 0
    _need_shaped(pos, torch.int32, (T,), dev, "pos")
    if seq is not None:
        _need_shaped(seq, torch.int32, (T,), dev, "seq")
    if rope.inv_freq is not None:
        _need_shaped(rope.inv_freq, torch.float32, (rope.rot // 2,), dev, "inv_freq")
    for t, n in ((rope.q_weight, "q_weight"), (rope.k_weight, "k_weight")):
        if t is not None:
            _need_shaped(t, torch.float32, (shape.d,), dev, n)
    if Q is not None:
        q = (T, shape.Hq, shape.d)
        qs = _rows_stride(Q, q, dev, "Q")
        if q_out is None:
            q_out = torch.empty(q, dtype=torch.bfloat16, device=dev)
        else:
            _need_shaped(q_out, torch.bfloat16, q, dev, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without Q")
    status = _need_status(status, dev)
    tokens = make_rope_shape(B, N, shape.Hq, shape.Hkv, shape.d, rope.rot, rope.interleaved, rope.norm, rope.eps,
                             rope.rot_scale, qs, ks)
    _on(dev, lib().pisa_paged_append, ctypes.byref(shape), ctypes.byref(c), ctypes.byref(tokens), _ptr(Q), K.data_ptr(),
        V.data_ptr(), vs, _ptr(rope.inv_freq), _ptr(rope.q_weight), _ptr(rope.k_weight), table.data_ptr(), _ptr(seq),
        pos.data_ptr(), _ptr(q_out), status.data_ptr())
    return q_out, status


def paged_workspace(shape: PagedShape, device) -> torch.Tensor:
    """A device workspace for paged_attn (uint8 tensor)."""
    b = ctypes.c_size_t()
    _check(lib().pisa_paged_workspace_size(ctypes.byref(shape), ctypes.byref(b)))
    return torch.empty(b.value, dtype=torch.uint8, device=device)


def paged_attn(shape: PagedShape, cache: PagedCache, table, lens, q, slopes=None, ws=None, o=None, lse=None):
    """The last nq tokens of every sequence against its pages: o [B,nq,Hq,d] bf16, lse [B,nq,Hq] fp32.

    lens: tokens of each sequence in the cache, the new ones included, [B] int32. slopes as in doc_attn_fwd. A query before its
    sequence's first token gets o = 0, lse = -inf. The workspace's status word tells of lengths and pages out of range."""
    dev = q.device
    c = _need_paged(shape, cache, table, dev)
    size = (shape.B, shape.nq, shape.Hq, shape.d)
    _need_shaped(lens, torch.int32, (shape.B,), dev, "lens")
    _need_shaped(q, torch.bfloat16, size, dev, "q")
    if slopes is not None:
        _need_shaped(slopes, torch.float32, (shape.Hq,), dev, "slopes")
    if o is None:
        o = torch.empty(size, dtype=torch.bfloat16, device=dev)
    else:
        _need_shaped(o, torch.bfloat16, size, dev, "o")
    if lse is None:
        lse = torch.empty(size[:3], dtype=torch.float32, device=dev)
    else:
        _need_shaped(lse, torch.float32, size[:3], dev, "lse")
    if ws is None:
        ws = paged_workspace(shape, dev)
    _need_ws(ws, dev)
    _on(dev, lib().pisa_paged_attn, ctypes.byref(shape), ctypes.byref(c), table.data_ptr(), lens.data_ptr(), q.data_ptr(),
        _ptr(slopes), o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel())
    return o, lse


def workspace_status(ws: torch.Tensor) -> int:
    """The status word of the last call that used workspace `ws` (its first 4 bytes, read after
    the current stream has passed the call): 0, or STATUS_* bits."""
    torch.cuda.current_stream(ws.device).synchronize()
    return int(ws[:4].view(torch.int32).item())


def check_status(ws: torch.Tensor) -> None:
    """Raise PisaError(PISA_ETIMEOUT) when the last call on `ws` reported a wait that gave up."""
    st = workspace_status(ws)
    if st & STATUS_TIMEOUT:
        raise PisaError(PISA_ETIMEOUT, f"a bounded device wait gave up (status word {st}); outputs are poisoned")


def set_wait_limit(ns: int) -> None:
    """Bound of every device-side pipeline wait in nanoseconds (0 restores the one-second default)."""
    _check(lib().pisa_set_wait_limit(int(ns)))


def set_test_stall(on: bool) -> None:
    """Test aid: make the tensor-core kernels wait on a barrier nothing signals (see pisa.h)."""
    _check(lib().pisa_test_stall(1 if on else 0))


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)


def profile_start() -> None:
    """Record CUDA events around every kernel launch of the library (on its stream)."""
    _check(lib().pisa_profile_start())


def profile_stop() -> None:
    _check(lib().pisa_profile_stop())


def profile_read() -> dict:
    """{kernel name: (launches, total ms)} since the last read; waits for the events."""
    buf = (ProfileEntry * 64)()
    n = ctypes.c_int32()
    _check(lib().pisa_profile_read(buf, 64, ctypes.byref(n)))
    return {buf[k].name.decode(): (buf[k].launches, buf[k].total_ms) for k in range(n.value)}
