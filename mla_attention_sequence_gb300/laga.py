"""Python binding of liblaga_mla.so (the C ABI in include/laga_mla.h).

Argument marshalling only: tensors are checked, outputs and workspace are
allocated with torch on the inputs' device, and every step of the computation
runs in the library's CUDA kernels on torch's current stream. There is no CPU
path: calling with CPU tensors, or without the built library, raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import NamedTuple

import torch

from .configs import Problem

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "liblaga_mla.so")

LAGA_OK = 0
STATUS_NAMES = {0: "LAGA_OK", 1: "LAGA_ERR_INVALID_ARG", 2: "LAGA_ERR_UNSUPPORTED", 3: "LAGA_ERR_WORKSPACE",
                4: "LAGA_ERR_CUDA", 5: "LAGA_ERR_TIMEOUT"}
DTYPES = {"f32": 0, "bf16": 1}
VARIANTS = {"auto": 0, "materialize": 1, "fused_recon": 2, "simt": 3}
FLAG_REUSE_KV = 1
FLAG_KV_PREBUILT = 2

EXPORTS = ("laga_mla_fwd_workspace_size", "laga_mla_bwd_workspace_size", "laga_mla_fwd", "laga_mla_bwd",
           "laga_mla_reconstruct", "laga_mla_check", "laga_status_string", "laga_mla_last_error",
           "laga_mla_version", "laga_mla_selftest_timeout", "laga_mla_absorbed_fwd",
           "laga_mla_absorbed_fwd_workspace_size", "laga_mla_reconstruct_rows", "laga_mla_masked_fwd",
           "laga_mla_masked_bwd", "laga_mla_masked_fwd_workspace_size", "laga_mla_masked_bwd_workspace_size",
           "laga_mla_key_bounds", "laga_mla_rope", "laga_mla_pack8", "laga_mla_unpack8", "laga_mla_norm_rope",
           "laga_mla_norm_rope_bwd", "laga_mla_norm_rope_bwd_workspace_size", "laga_mla_cache4_append",
           "laga_mla_cache4_read", "laga_mla_cache4_fwd", "laga_mla_cache4_fwd_workspace_size")


class LagaDesc(ctypes.Structure):
    """Mirror of laga_mla_desc."""
    _fields_ = [("batch", ctypes.c_int64), ("sq", ctypes.c_int64), ("skv", ctypes.c_int64),
                ("n_h", ctypes.c_int64), ("d_c", ctypes.c_int64), ("d_nope", ctypes.c_int64),
                ("d_rope", ctypes.c_int64), ("d_v", ctypes.c_int64), ("q_offset", ctypes.c_int64),
                ("causal", ctypes.c_int32), ("softmax_scale", ctypes.c_float), ("dtype", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("flags", ctypes.c_int32), ("q_split", ctypes.c_int64),
                ("q_offset2", ctypes.c_int64)]


class LagaMods(ctypes.Structure):
    """Mirror of laga_mla_mods."""
    _fields_ = [("key_lo", ctypes.c_void_p), ("key_hi", ctypes.c_void_p), ("slopes", ctypes.c_void_p),
                ("softcap", ctypes.c_float)]


class LagaPacked(ctypes.Structure):
    """Mirror of laga_mla_packed."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


ROPE_MAX_AXES = 4


class LagaRopeDesc(ctypes.Structure):
    """Mirror of laga_mla_rope_desc."""
    _fields_ = [("tokens", ctypes.c_int64), ("n_h", ctypes.c_int64), ("d_nope", ctypes.c_int64),
                ("d_rope", ctypes.c_int64), ("n_axes", ctypes.c_int64), ("sections", ctypes.c_int64 * ROPE_MAX_AXES),
                ("theta", ctypes.c_double), ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("pos64", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class LagaCache4(ctypes.Structure):
    """Mirror of laga_mla_cache4."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("k_rope", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("d_c", ctypes.c_int64),
                ("d_rope", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class LagaCache4Desc(ctypes.Structure):
    """Mirror of laga_mla_cache4_desc."""
    _fields_ = [("batch", ctypes.c_int64), ("sq", ctypes.c_int64), ("n_h", ctypes.c_int64), ("d_nope", ctypes.c_int64),
                ("d_v", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("causal", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("variant", ctypes.c_int32)]


class LagaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {detail}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load the library (built in-tree by the package's build step)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with mla_attention_sequence_gb300.build.build()")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    pd = ctypes.POINTER(LagaDesc)
    L.laga_mla_fwd_workspace_size.argtypes = [pd]
    L.laga_mla_fwd_workspace_size.restype = sz
    L.laga_mla_bwd_workspace_size.argtypes = [pd]
    L.laga_mla_bwd_workspace_size.restype = sz
    L.laga_mla_fwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.laga_mla_fwd.restype = st
    L.laga_mla_bwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.laga_mla_bwd.restype = st
    L.laga_mla_absorbed_fwd_workspace_size.argtypes = [pd]
    L.laga_mla_absorbed_fwd_workspace_size.restype = sz
    L.laga_mla_absorbed_fwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.laga_mla_absorbed_fwd.restype = st
    L.laga_mla_reconstruct.argtypes = [pd, vp, vp, vp, vp, vp, vp]
    L.laga_mla_reconstruct.restype = st
    L.laga_mla_reconstruct_rows.argtypes = [pd, vp, vp, vp, ctypes.c_int64, ctypes.c_int64, vp, sz, vp]
    L.laga_mla_reconstruct_rows.restype = st
    pm, pp = ctypes.POINTER(LagaMods), ctypes.POINTER(LagaPacked)
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    for f in (L.laga_mla_masked_fwd_workspace_size, L.laga_mla_masked_bwd_workspace_size):
        f.argtypes = [pd]
        f.restype = sz
    L.laga_mla_masked_fwd.argtypes = [pd, pm] + [vp] * 8 + [sz, vp]
    L.laga_mla_masked_bwd.argtypes = [pd, pm] + [vp] * 8 + [pp, pp] + [vp] * 6 + [sz, vp]
    L.laga_mla_key_bounds.argtypes = [i64] * 6 + [vp, i64, vp, i64, vp, vp, vp]
    L.laga_mla_rope.argtypes = [ctypes.POINTER(LagaRopeDesc)] + [vp] * 6
    L.laga_mla_pack8.argtypes = [i32, i64, i64, vp, vp, vp, vp]
    L.laga_mla_unpack8.argtypes = [i32, i64, i64, vp, vp, vp, vp]
    for f in (L.laga_mla_masked_fwd, L.laga_mla_masked_bwd, L.laga_mla_key_bounds, L.laga_mla_rope, L.laga_mla_pack8,
              L.laga_mla_unpack8):
        f.restype = st
    f32, pr, pc, pcd = ctypes.c_float, ctypes.POINTER(LagaRopeDesc), ctypes.POINTER(LagaCache4), \
        ctypes.POINTER(LagaCache4Desc)
    L.laga_mla_norm_rope.argtypes = [pr, f32] + [vp] * 8
    L.laga_mla_norm_rope_bwd.argtypes = [pr, f32] + [vp] * 12 + [sz, vp]
    L.laga_mla_norm_rope_bwd_workspace_size.argtypes = [pr]
    L.laga_mla_cache4_append.argtypes = [pc, i64, i64, i64] + [vp] * 6 + [f32, pr, vp, vp]
    L.laga_mla_cache4_read.argtypes = [pc, i64, i64, i64] + [vp] * 6
    L.laga_mla_cache4_fwd.argtypes = [pcd, pc, pm] + [vp] * 8 + [sz, vp]
    L.laga_mla_cache4_fwd_workspace_size.argtypes = [pcd, pc]
    for f in (L.laga_mla_norm_rope, L.laga_mla_norm_rope_bwd, L.laga_mla_cache4_append, L.laga_mla_cache4_read,
              L.laga_mla_cache4_fwd):
        f.restype = st
    for f in (L.laga_mla_norm_rope_bwd_workspace_size, L.laga_mla_cache4_fwd_workspace_size):
        f.restype = sz
    L.laga_mla_check.argtypes = [vp]
    L.laga_mla_check.restype = st
    L.laga_mla_selftest_timeout.argtypes = [vp]
    L.laga_mla_selftest_timeout.restype = st
    L.laga_status_string.argtypes = [st]
    L.laga_status_string.restype = ctypes.c_char_p
    L.laga_mla_last_error.argtypes = []
    L.laga_mla_last_error.restype = ctypes.c_char_p
    L.laga_mla_version.argtypes = []
    L.laga_mla_version.restype = ctypes.c_int
    _lib = L
    return L


def _raise_if(status: int):
    if status != LAGA_OK:
        raise LagaError(status, lib().laga_mla_last_error().decode(errors="replace"))


def make_desc(p: Problem, softmax_scale: float | None = None, variant: str = "auto", flags: int = 0) -> LagaDesc:
    return LagaDesc(p.B, p.Sq, p.S, p.n_h, p.d_c, p.d_nope, p.d_rope, p.d_v, p.q_offset, 1 if p.causal else 0,
                    float(softmax_scale) if softmax_scale else 0.0, DTYPES[p.dtype], VARIANTS[variant], flags,
                    p.q_split, p.q_offset2)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def problem_of(q, c_kv, k_rope, W_UK, W_UV, q_offset: int, causal: bool, q_split: int = 0,
               q_offset2: int = 0) -> Problem:
    """Infer and check the problem sizes from the input tensors. q_split > 0 makes
    rows [q_split, Sq) a second query segment starting at position q_offset2."""
    if q.dim() != 4 or c_kv.dim() != 3 or k_rope.dim() != 3 or W_UK.dim() != 2 or W_UV.dim() != 2:
        raise ValueError("expected q [B,Sq,n_h,d_qk], c_kv [B,S,d_c], k_rope [B,S,d_rope], W [d_c, n_h*d]")
    B, Sq, n_h, d_qk = q.shape
    _, S, d_c = c_kv.shape
    d_rope = k_rope.shape[2]
    if c_kv.shape[0] != B or k_rope.shape[:2] != (B, S) or W_UK.shape[0] != d_c or W_UV.shape[0] != d_c:
        raise ValueError("inconsistent batch / latent shapes")
    if W_UK.shape[1] % n_h or W_UV.shape[1] % n_h:
        raise ValueError("W_UK / W_UV columns must be n_h * head width")
    d_nope, d_v = W_UK.shape[1] // n_h, W_UV.shape[1] // n_h
    if d_nope + d_rope != d_qk:
        raise ValueError("q's last dim must be d_nope + d_rope")
    dt = {torch.float32: "f32", torch.bfloat16: "bf16"}.get(q.dtype)
    if dt is None:
        raise TypeError("tensors must be float32 or bfloat16")
    for t in (q, c_kv, k_rope, W_UK, W_UV):
        if t.dtype != q.dtype:
            raise TypeError("all inputs must share one dtype")
        if not t.is_cuda:
            raise RuntimeError("LAGA MLA runs on CUDA tensors only")
        if not t.is_contiguous():
            raise ValueError("inputs must be contiguous")
    return Problem(B=B, Sq=Sq, S=S, n_h=n_h, d_c=d_c, d_nope=d_nope, d_rope=d_rope, d_v=d_v,
                   q_offset=int(q_offset), causal=bool(causal), dtype=dt, q_split=int(q_split),
                   q_offset2=int(q_offset2))


def fwd_workspace_bytes(p: Problem, variant: str = "auto") -> int:
    d = make_desc(p, None, variant)
    return int(lib().laga_mla_fwd_workspace_size(ctypes.byref(d)))


def bwd_workspace_bytes(p: Problem, variant: str = "auto") -> int:
    d = make_desc(p, None, variant)
    return int(lib().laga_mla_bwd_workspace_size(ctypes.byref(d)))


def _workspace(nbytes: int, device, given: torch.Tensor | None) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    if given is not None:
        if given.numel() * given.element_size() < nbytes:
            raise ValueError("workspace too small")
        return given
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def fwd(q, c_kv, k_rope, W_UK, W_UV, q_offset: int = 0, causal: bool = True, softmax_scale: float | None = None,
        variant: str = "auto", workspace: torch.Tensor | None = None, out=None, lse=None, q_split: int = 0,
        q_offset2: int = 0, kv_prebuilt: bool = False):
    """laga_mla_fwd: returns (out [B,Sq,n_h,d_v], lse [B,n_h,Sq] fp32).

    kv_prebuilt=True (LAGA_FLAG_KV_PREBUILT): `workspace` already holds K_nope / V
    for every row the forward reads, from reconstruct_rows calls with the same
    arguments; the call runs the attention alone."""
    p = problem_of(q, c_kv, k_rope, W_UK, W_UV, q_offset, causal, q_split, q_offset2)
    if kv_prebuilt and workspace is None:
        raise ValueError("kv_prebuilt needs the workspace the rows were rebuilt into")
    d = make_desc(p, softmax_scale, variant, FLAG_KV_PREBUILT if kv_prebuilt else 0)
    L = lib()
    dev = q.device
    if out is None:
        out = torch.empty((p.B, p.Sq, p.n_h, p.d_v), dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((p.B, p.n_h, p.Sq), dtype=torch.float32, device=dev)
    nbytes = int(L.laga_mla_fwd_workspace_size(ctypes.byref(d)))
    ws = _workspace(nbytes, dev, workspace)
    _raise_if(L.laga_mla_fwd(ctypes.byref(d), _ptr(q), _ptr(c_kv), _ptr(k_rope), _ptr(W_UK), _ptr(W_UV),
                             _ptr(out), _ptr(lse), _ptr(ws), nbytes, _stream(dev)))
    return out, lse


def bwd(q, c_kv, k_rope, W_UK, W_UV, out, lse, dout, q_offset: int = 0, causal: bool = True,
        softmax_scale: float | None = None, variant: str = "auto", workspace: torch.Tensor | None = None,
        grads: dict | None = None, reuse_kv: bool = False, q_split: int = 0, q_offset2: int = 0):
    """laga_mla_bwd: returns dict dq, dc_kv, dk_rope, dW_UK, dW_UV.

    reuse_kv=True (LAGA_FLAG_REUSE_KV): `workspace` is the buffer the forward
    ran with, still holding the K_nope/V it rebuilt; the backward reads them
    instead of rebuilding them."""
    p = problem_of(q, c_kv, k_rope, W_UK, W_UV, q_offset, causal, q_split, q_offset2)
    for t in (out, lse, dout):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("out, lse and dout must be contiguous CUDA tensors")
    if reuse_kv and workspace is None:
        raise ValueError("reuse_kv needs the workspace the forward ran with")
    d = make_desc(p, softmax_scale, variant, FLAG_REUSE_KV if reuse_kv else 0)
    L = lib()
    dev = q.device
    g = grads if grads is not None else {
        "dq": torch.empty_like(q), "dc_kv": torch.empty_like(c_kv), "dk_rope": torch.empty_like(k_rope),
        "dW_UK": torch.empty_like(W_UK), "dW_UV": torch.empty_like(W_UV)}
    nbytes = int(L.laga_mla_bwd_workspace_size(ctypes.byref(d)))
    ws = _workspace(nbytes, dev, workspace)
    _raise_if(L.laga_mla_bwd(ctypes.byref(d), _ptr(q), _ptr(c_kv), _ptr(k_rope), _ptr(W_UK), _ptr(W_UV),
                             _ptr(out), _ptr(lse), _ptr(dout), _ptr(g["dq"]), _ptr(g["dc_kv"]), _ptr(g["dk_rope"]),
                             _ptr(g["dW_UK"]), _ptr(g["dW_UV"]), _ptr(ws), nbytes, _stream(dev)))
    return g


def reconstruct_rows(q, c_kv, k_rope, W_UK, W_UV, row0: int, rows: int, workspace: torch.Tensor,
                     q_offset: int = 0, causal: bool = True, q_split: int = 0, q_offset2: int = 0,
                     variant: str = "auto"):
    """laga_mla_reconstruct_rows: the forward's K/V rebuild for latent rows
    [row0, row0 + rows) into `workspace` (of at least fwd_workspace_bytes), for a
    later fwd(..., workspace=workspace, kv_prebuilt=True) with the same arguments.
    row0 a multiple of 128; row0 + rows a multiple of 128 or past the last row any
    query sees."""
    p = problem_of(q, c_kv, k_rope, W_UK, W_UV, q_offset, causal, q_split, q_offset2)
    d = make_desc(p, None, variant)
    nbytes = workspace.numel() * workspace.element_size()
    _raise_if(lib().laga_mla_reconstruct_rows(ctypes.byref(d), _ptr(c_kv), _ptr(W_UK), _ptr(W_UV), int(row0),
                                              int(rows), _ptr(workspace), nbytes, _stream(q.device)))


def absorbed_fwd(q, c_kv, k_rope, W_UK, W_UV, q_offset: int = 0, causal: bool = True,
                 softmax_scale: float | None = None, workspace: torch.Tensor | None = None, out=None, lse=None):
    """laga_mla_absorbed_fwd (the absorbed MLA form, for comparison): returns
    (out [B,Sq,n_h,d_v], lse [B,n_h,Sq] fp32). The workspace holds the form's
    intermediates q_lat and ctx ([B,Sq,n_h,d_c] each)."""
    p = problem_of(q, c_kv, k_rope, W_UK, W_UV, q_offset, causal)
    d = make_desc(p, softmax_scale)
    L = lib()
    dev = q.device
    if out is None:
        out = torch.empty((p.B, p.Sq, p.n_h, p.d_v), dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((p.B, p.n_h, p.Sq), dtype=torch.float32, device=dev)
    nbytes = int(L.laga_mla_absorbed_fwd_workspace_size(ctypes.byref(d)))
    if nbytes == 0:
        _raise_if(L.laga_mla_absorbed_fwd(ctypes.byref(d), None, None, None, None, None, None, None, None, 0,
                                          _stream(dev)))
    ws = _workspace(nbytes, dev, workspace)
    _raise_if(L.laga_mla_absorbed_fwd(ctypes.byref(d), _ptr(q), _ptr(c_kv), _ptr(k_rope), _ptr(W_UK), _ptr(W_UV),
                                      _ptr(out), _ptr(lse), _ptr(ws), nbytes, _stream(dev)))
    return out, lse


def absorbed_workspace_bytes(p: Problem) -> int:
    d = make_desc(p)
    return int(lib().laga_mla_absorbed_fwd_workspace_size(ctypes.byref(d)))


def reconstruct(c_kv, W_UK, W_UV, n_h: int, variant: str = "auto"):
    """laga_mla_reconstruct: per-head K_nope [B,S,n_h,d_nope] and V [B,S,n_h,d_v]."""
    B, S, d_c = c_kv.shape
    d_nope, d_v = W_UK.shape[1] // n_h, W_UV.shape[1] // n_h
    dt = {torch.float32: "f32", torch.bfloat16: "bf16"}[c_kv.dtype]
    p = Problem(B=B, Sq=1, S=S, n_h=n_h, d_c=d_c, d_nope=d_nope, d_rope=64 if dt == "bf16" else 0, d_v=d_v,
                q_offset=0, causal=False, dtype=dt)
    d = make_desc(p, None, variant)
    kn = torch.empty((B, S, n_h, d_nope), dtype=c_kv.dtype, device=c_kv.device)
    v = torch.empty((B, S, n_h, d_v), dtype=c_kv.dtype, device=c_kv.device)
    _raise_if(lib().laga_mla_reconstruct(ctypes.byref(d), _ptr(c_kv), _ptr(W_UK), _ptr(W_UV), _ptr(kn), _ptr(v),
                                         _stream(c_kv.device)))
    return kn, v


# ---------------------------------------------------------------- packed documents
#
# Every call below runs on the current stream of its tensors' device and makes that device
# current for its launches; all tensors of a call are on one device. The host's share of a
# small call is most of its time, so what depends on sizes alone is worked out once per sizes.

_TORCH_DTYPES = {torch.float32: "f32", torch.bfloat16: "bf16"}
_DTYPE_CODES = {torch.float32: 0, torch.bfloat16: 1}
_INT32, _FP32, _UINT8 = (torch.int32,), (torch.float32,), (torch.uint8,)


def _code_of(dtype: torch.dtype) -> int:
    if dtype not in _DTYPE_CODES:
        raise TypeError("tensors must be float32 or bfloat16")
    return _DTYPE_CODES[dtype]


def _expect(name: str, t: torch.Tensor, shape, dtypes, device) -> int:
    """The address of a contiguous CUDA tensor of that shape (None: any), type and device; an error that
    names it otherwise."""
    if isinstance(t, torch.Tensor) and t.get_device() == device.index and t.dtype in dtypes and t.is_contiguous() \
            and (shape is None or t.shape == shape):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise RuntimeError(f"{name}: LAGA MLA runs on CUDA tensors only")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


# The current stream's handle without the Stream object around it (2 us of a small call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(device, fn, *args):
    """fn(*args, stream) with `device` current, on its current stream."""
    index = device.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status != LAGA_OK:
        _raise_if(status)


def key_bounds(doc_starts, n_rows: int, q_offset: int = 0, prefix=None, window: int = 0, skv: int | None = None,
               q_split: int = 0, q_offset2: int = 0):
    """laga_mla_key_bounds: (key_lo, key_hi), int32 [B, n_rows], for masked_fwd / masked_bwd.

    doc_starts: int32 [B, n_docs + 1], ascending; document k holds the keys [doc_starts[k],
    doc_starts[k + 1]). A row sees the keys of its own document up to its position, at most
    the last `window` of them (0: all), or, with prefix (int32 [B, n_docs]), also all of the
    document's first prefix[k] keys (call the attention with causal=False then; not together
    with a window). Rows in no
    document see nothing. skv clamps the bounds (None: only the documents do)."""
    shape = doc_starts.shape
    if len(shape) != 2 or shape[1] < 2:
        raise ValueError("doc_starts must be [B, n_docs + 1]")
    B, n_docs = shape[0], shape[1] - 1
    dev = doc_starts.device
    starts = _expect("doc_starts", doc_starts, None, _INT32, dev)
    pre = None if prefix is None else _expect("prefix", prefix, (B, n_docs), _INT32, dev)
    lo = torch.empty((B, n_rows), dtype=torch.int32, device=dev)
    hi = torch.empty((B, n_rows), dtype=torch.int32, device=dev)
    _launch(dev, lib().laga_mla_key_bounds, B, n_rows, (1 << 30) - 1 if skv is None else int(skv), int(q_offset),
            int(q_split), int(q_offset2), starts, n_docs, pre, int(window), lo.data_ptr(), hi.data_ptr())
    return lo, hi


@dataclass
class Packed8:
    """A tensor saved in 8 bits: e4m3 codes (uint8, the tensor's shape), one biased power-of-two
    exponent per 32 values of the last dimension (uint8), and the type it is restored to."""
    codes: torch.Tensor
    scales: torch.Tensor
    dtype: torch.dtype

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device


def _scales_shape(shape):
    return (*shape[:-1], (shape[-1] + 31) // 32)


def _check_packed(name: str, p: Packed8):
    """(address of the codes, address of the scales)."""
    if p.dtype not in _DTYPE_CODES:
        raise TypeError(f"{name}: a checkpoint restores to float32 or bfloat16")
    shape, dev = p.codes.shape, p.codes.device
    if not shape:
        raise ValueError(f"{name}: a checkpoint has at least one dimension")
    return (_expect(name + ".codes", p.codes, None, _UINT8, dev),
            _expect(name + ".scales", p.scales, _scales_shape(shape), _UINT8, dev))


def pack8(x: torch.Tensor) -> Packed8:
    """laga_mla_pack8: saves a float32 or bfloat16 tensor in 8 bits along its last dimension. A q for
    masked_bwd is packed before the forward (see there)."""
    dt, shape, dev = x.dtype, x.shape, x.device
    code = _code_of(dt)
    if not shape:
        raise ValueError("pack8 needs at least one dimension")
    src = _expect("x", x, None, (dt,), dev)
    codes = torch.empty(shape, dtype=torch.uint8, device=dev)
    scales = torch.empty(_scales_shape(shape), dtype=torch.uint8, device=dev)
    n, cols = x.numel(), shape[-1]
    if n:
        _launch(dev, lib().laga_mla_pack8, code, n // cols, cols, src, codes.data_ptr(), scales.data_ptr())
    return Packed8(codes, scales, dt)


def unpack8(p: Packed8, out: torch.Tensor | None = None) -> torch.Tensor:
    """laga_mla_unpack8: the tensor a checkpoint stands for, in its own type."""
    codes, scales = _check_packed("p", p)
    shape, dev = p.codes.shape, p.codes.device
    if out is None:
        out = torch.empty(shape, dtype=p.dtype, device=dev)
    else:
        _expect("out", out, shape, (p.dtype,), dev)
    n, cols = out.numel(), shape[-1]
    if n:
        _launch(dev, lib().laga_mla_unpack8, _DTYPE_CODES[p.dtype], n // cols, cols, codes, scales, out.data_ptr())
    return out


@functools.lru_cache(maxsize=256)
def _rope_desc(q_shape, d_rope, sections, theta, interleaved, inverse, pos64, code):
    B, S, n_h, d_qk = q_shape
    if d_rope > d_qk:
        raise ValueError("q's last dim must be d_nope + d_rope")
    return LagaRopeDesc(B * S, n_h, d_qk - d_rope, d_rope, len(sections),
                        (ctypes.c_int64 * ROPE_MAX_AXES)(*sections), theta, interleaved, inverse, pos64, code)


def rope(q, k_rope, pos, sections=None, theta: float = 10000.0, interleaved: bool = True, inverse: bool = False,
         q_out=None, k_out=None):
    """laga_mla_rope: rotates the RoPE part of q [B, S, n_h, d_nope + d_rope] and k_rope
    [B, S, d_rope] by the positions pos [n_axes, B, S] (int32 or int64); returns (q, k_rope)
    rotated. sections: pairs per axis (None: one axis with all). The outputs are new tensors,
    or q_out / k_out, which may be q / k_rope themselves (in place). inverse=True rotates back:
    pass the gradients of the rotated tensors to get those of q and k_rope."""
    shape, dt, dev = q.shape, q.dtype, q.device
    if len(shape) != 4 or k_rope.dim() != 3 or pos.dim() != 3:
        raise ValueError("expected q [B,S,n_h,d_nope+d_rope], k_rope [B,S,d_rope], pos [n_axes,B,S]")
    d_rope, axes = k_rope.shape[2], pos.shape[0]
    code = _code_of(dt)
    k_shape = (shape[0], shape[1], d_rope)
    src = _expect("q", q, None, (dt,), dev)
    k_src = _expect("k_rope", k_rope, k_shape, (dt,), dev)
    at = _expect("pos", pos, (axes, shape[0], shape[1]), (torch.int32, torch.int64), dev)
    sections = (d_rope // 2,) if sections is None else tuple(map(int, sections))
    if len(sections) != axes or axes > ROPE_MAX_AXES:
        raise ValueError(f"one section per axis of pos, at most {ROPE_MAX_AXES}")
    if q_out is None:
        q_out = torch.empty(shape, dtype=dt, device=dev)
        q_at = q_out.data_ptr()
    else:
        q_at = _expect("q_out", q_out, shape, (dt,), dev)
    if k_out is None:
        k_out = torch.empty(k_shape, dtype=dt, device=dev)
        k_at = k_out.data_ptr()
    else:
        k_at = _expect("k_out", k_out, k_shape, (dt,), dev)
    if shape[0] * shape[1] == 0:  # no tokens: nothing turns
        return q_out, k_out
    d = _rope_desc(shape, d_rope, sections, float(theta), bool(interleaved), bool(inverse), pos.dtype == torch.int64,
                   code)
    _launch(dev, lib().laga_mla_rope, d, at, src, k_src, q_at, k_at)
    return q_out, k_out


@functools.lru_cache(maxsize=256)
def _masked_plan(q_shape, c_shape, r_shape, wk_shape, wv_shape, dtype, q_offset, causal, softmax_scale, variant,
                 q_split, q_offset2):
    """What a masked call's sizes decide: the other tensors' shapes, the descriptors without and with the reuse of K and
    V, the bytes of the forward's and the backward's workspace (0: refused)."""
    like = [_Sizes(s, dtype) for s in (q_shape, c_shape, r_shape, wk_shape, wv_shape)]
    p = problem_of(*like, q_offset, causal, q_split, q_offset2)
    d = make_desc(p, softmax_scale, variant)
    L = lib()
    shapes = _Shapes((p.B, p.Sq), (p.n_h,), (p.B, p.Sq, p.n_h, p.d_qk), (p.B, p.Sq, p.n_h, p.d_v), (p.B, p.n_h, p.Sq))
    return (shapes, d, make_desc(p, softmax_scale, variant, FLAG_REUSE_KV), int(L.laga_mla_masked_fwd_workspace_size(d)),
            int(L.laga_mla_masked_bwd_workspace_size(d)))


class _Shapes(NamedTuple):
    rows: tuple
    heads: tuple
    q: tuple
    out: tuple
    lse: tuple


class _Sizes:
    """A tensor's shape and type for problem_of, which asks no more of it."""
    is_cuda = True

    def __init__(self, shape, dtype):
        self.shape, self.dtype = shape, dtype

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True


class _MaskedCall:
    """The checked arguments that masked_fwd, masked_bwd and masked_workspace share."""
    __slots__ = ("shapes", "desc", "reuse", "fwd_bytes", "bwd_bytes", "q", "x", "dev", "dt", "dts")

    def __init__(self, q, c_kv, k_rope, W_UK, W_UV, q_offset, causal, softmax_scale, variant, q_split, q_offset2):
        self.dt, self.dev = dt, dev = c_kv.dtype, c_kv.device
        if dt not in _DTYPE_CODES:
            raise TypeError("tensors must be float32 or bfloat16")
        self.dts = dts = (dt,)
        if isinstance(q, Packed8):
            self.q = LagaPacked(*_check_packed("q", q))
            if q.dtype != dt:
                raise TypeError("all inputs must share one dtype")
            if q.device != dev:
                raise ValueError(f"q is on {q.device}, the other tensors on {dev}")
        else:
            self.q = _expect("q", q, None, dts, dev)
        self.x = (_expect("c_kv", c_kv, None, dts, dev), _expect("k_rope", k_rope, None, dts, dev),
                  _expect("W_UK", W_UK, None, dts, dev), _expect("W_UV", W_UV, None, dts, dev))
        self.shapes, self.desc, self.reuse, self.fwd_bytes, self.bwd_bytes = _masked_plan(
            q.shape, c_kv.shape, k_rope.shape, W_UK.shape, W_UV.shape, dt, int(q_offset), bool(causal),
            None if softmax_scale is None else float(softmax_scale), variant, int(q_split), int(q_offset2))

    def mods(self, key_lo, key_hi, softcap, slopes) -> LagaMods:
        shapes, dev = self.shapes, self.dev
        return LagaMods(None if key_lo is None else _expect("key_lo", key_lo, shapes.rows, _INT32, dev),
                        None if key_hi is None else _expect("key_hi", key_hi, shapes.rows, _INT32, dev),
                        None if slopes is None else _expect("slopes", slopes, shapes.heads, _FP32, dev),
                        softcap or 0.0)

    def workspace(self, nbytes, given):
        """(the tensor that keeps it alive, its address)."""
        if given is None:
            given = torch.empty(nbytes, dtype=torch.uint8, device=self.dev)
            return given, given.data_ptr()
        at = _expect("workspace", given, None, (given.dtype,), self.dev)
        if given.numel() * given.element_size() < nbytes:
            raise ValueError("workspace too small")
        return given, at

    def output(self, name, t, shape, dtypes):
        """(the output, its address): `t`, or a new tensor."""
        if t is None:
            t = torch.empty(shape, dtype=dtypes[0], device=self.dev)
            return t, t.data_ptr()
        return t, _expect(name, t, shape, dtypes, self.dev)


def masked_workspace(q, c_kv, k_rope, W_UK, W_UV, key_lo=None, key_hi=None, softcap: float = 0.0, slopes=None,
                     q_offset: int = 0, causal: bool = True, softmax_scale: float | None = None, variant: str = "auto",
                     q_split: int = 0, q_offset2: int = 0) -> torch.Tensor:
    """A workspace for masked_fwd and masked_bwd of these arguments; the forward's K and V stay in
    it for a backward with reuse_kv=True."""
    c = _MaskedCall(q, c_kv, k_rope, W_UK, W_UV, q_offset, causal, softmax_scale, variant, q_split, q_offset2)
    if c.bwd_bytes == 0:
        lib().laga_mla_masked_bwd_workspace_size(c.desc)  # the reason, for this thread
        _raise_if(2)
    return torch.empty(c.bwd_bytes, dtype=torch.uint8, device=c.dev)


def masked_fwd(q, c_kv, k_rope, W_UK, W_UV, key_lo=None, key_hi=None, softcap: float = 0.0, slopes=None,
               q_offset: int = 0, causal: bool = True, softmax_scale: float | None = None, variant: str = "auto",
               workspace: torch.Tensor | None = None, out=None, lse=None, q_split: int = 0, q_offset2: int = 0):
    """laga_mla_masked_fwd: (out [B,Sq,n_h,d_v], lse [B,n_h,Sq] fp32) where row i sees the keys
    key_lo[i] <= j < key_hi[i] (int32 [B, Sq], as key_bounds makes them; None: no bound) and, when
    causal, j <= its position. softcap > 0: scores become softcap tanh(s / softcap). slopes
    (float32 [n_h]): minus slopes[h] times the distance to the key. A row that sees nothing gets
    out 0 and lse -inf."""
    if isinstance(q, Packed8):
        raise ValueError("the forward takes q as a tensor")
    c = _MaskedCall(q, c_kv, k_rope, W_UK, W_UV, q_offset, causal, softmax_scale, variant, q_split, q_offset2)
    m = c.mods(key_lo, key_hi, softcap, slopes)
    out, out_at = c.output("out", out, c.shapes.out, c.dts)
    lse, lse_at = c.output("lse", lse, c.shapes.lse, _FP32)
    ws, at = c.workspace(c.fwd_bytes, workspace)
    _launch(c.dev, lib().laga_mla_masked_fwd, c.desc, m, c.q, *c.x, out_at, lse_at, at, c.fwd_bytes)
    return out, lse


def masked_bwd(q, c_kv, k_rope, W_UK, W_UV, out, lse, dout, key_lo=None, key_hi=None, softcap: float = 0.0,
               slopes=None, q_offset: int = 0, causal: bool = True, softmax_scale: float | None = None,
               variant: str = "auto", workspace: torch.Tensor | None = None, grads: dict | None = None,
               reuse_kv: bool = False, q_split: int = 0, q_offset2: int = 0):
    """laga_mla_masked_bwd: dict dq, dc_kv, dk_rope, dW_UK, dW_UV of <dout, out>, with the forward's
    arguments. q and out may both be Packed8 checkpoints: the backward reads them in 8 bits. Pack q
    before the forward and run it on unpack8 of the checkpoint, so that lse belongs to the q that the
    backward sees; with lse of the q before its rounding the weights exp(s - lse) do not sum to 1, the
    further off the larger the scores. reuse_kv=True: `workspace` is the one the forward ran with, its
    K and V intact."""
    packed = isinstance(q, Packed8)
    if packed != isinstance(out, Packed8):
        raise ValueError("q and out come either both as tensors or both as 8-bit checkpoints")
    c = _MaskedCall(q, c_kv, k_rope, W_UK, W_UV, q_offset, causal, softmax_scale, variant, q_split, q_offset2)
    dev, dts, shapes = c.dev, c.dts, c.shapes
    if packed:
        out8 = LagaPacked(*_check_packed("out", out))
        if out.dtype != c.dt:
            raise TypeError("all inputs must share one dtype")
        _expect("out.codes", out.codes, shapes.out, _UINT8, dev)
        q_at, out_at, q8 = None, None, c.q
    else:
        q_at, out_at, q8, out8 = c.q, _expect("out", out, shapes.out, dts, dev), None, None
    lse_at = _expect("lse", lse, shapes.lse, _FP32, dev)
    dout_at = _expect("dout", dout, shapes.out, dts, dev)
    if reuse_kv and workspace is None:
        raise ValueError("reuse_kv needs the workspace the forward ran with")
    m = c.mods(key_lo, key_hi, softcap, slopes)
    given = (grads or {}).get
    dq, a0 = c.output("dq", given("dq"), shapes.q, dts)
    dc_kv, a1 = c.output("dc_kv", given("dc_kv"), c_kv.shape, dts)
    dk_rope, a2 = c.output("dk_rope", given("dk_rope"), k_rope.shape, dts)
    dW_UK, a3 = c.output("dW_UK", given("dW_UK"), W_UK.shape, dts)
    dW_UV, a4 = c.output("dW_UV", given("dW_UV"), W_UV.shape, dts)
    ws, at = c.workspace(c.bwd_bytes, workspace)
    _launch(dev, lib().laga_mla_masked_bwd, c.reuse if reuse_kv else c.desc, m, q_at, *c.x, out_at, lse_at, dout_at, q8,
            out8, a0, a1, a2, a3, a4, at, c.bwd_bytes)
    return {"dq": dq, "dc_kv": dc_kv, "dk_rope": dk_rope, "dW_UK": dW_UK, "dW_UV": dW_UV}


# ---------------------------------------------------------------- norms with rotation, the 4-bit cache


def _norm_call(q, k_rope, pos, q_weight, k_weight, sections, theta, interleaved):
    """(descriptor, shapes of q and k_rope or None, addresses of pos, q, k_rope, q_weight, k_weight, type, device)."""
    like = q if q is not None else k_rope
    if like is None:
        raise ValueError("give q, k_rope or both")
    dt, dev = like.dtype, like.device
    code = _code_of(dt)
    dts = (dt,)
    if pos.dim() != 3 or (q is not None and q.dim() != 4) or (k_rope is not None and k_rope.dim() != 3):
        raise ValueError("expected q [B,S,n_h,d_nope+d_rope], k_rope [B,S,d_rope], pos [n_axes,B,S]")
    B, S = like.shape[:2]
    if k_rope is not None:
        d_rope = k_rope.shape[2]
    elif sections is None:
        raise ValueError("without k_rope the sections say how much of a head turns")
    else:
        d_rope = 2 * sum(map(int, sections))
    sections = (d_rope // 2,) if sections is None else tuple(map(int, sections))
    axes = pos.shape[0]
    if len(sections) != axes or axes > ROPE_MAX_AXES:
        raise ValueError(f"one section per axis of pos, at most {ROPE_MAX_AXES}")
    q_at = k_at = wq_at = wk_at = None
    if q is not None:
        q_at = _expect("q", q, None, dts, dev)
        wq_at = _expect("q_weight", q_weight, (q.shape[3],), dts, dev)
    elif q_weight is not None:
        raise ValueError("q_weight without q")
    if k_rope is not None:
        k_at = _expect("k_rope", k_rope, (B, S, d_rope), dts, dev)
        wk_at = _expect("k_weight", k_weight, (d_rope,), dts, dev)
    elif k_weight is not None:
        raise ValueError("k_weight without k_rope")
    at = _expect("pos", pos, (axes, B, S), (torch.int32, torch.int64), dev)
    d = _rope_desc(tuple(q.shape) if q is not None else (B, S, 1, d_rope), d_rope, sections, float(theta),
                   bool(interleaved), False, pos.dtype == torch.int64, code) if B * S else None
    return d, (at, q_at, k_at, wq_at, wk_at), dts, dev


def _made(name, t, like, dts, dev):
    """(the output, its address): `t`, or a new tensor of like's shape; (None, None) where like is None."""
    if like is None:
        if t is not None:
            raise ValueError(f"{name} without its input")
        return None, None
    if t is None:
        t = torch.empty_like(like)  # contiguous and of the calls' type, as `like` has been found to be
        return t, t.data_ptr()
    return t, _expect(name, t, like.shape, dts, dev)


def norm_rope(q, k_rope, pos, q_weight, k_weight=None, eps: float = 1e-6, sections=None, theta: float = 10000.0,
              interleaved: bool = True, q_out=None, k_out=None):
    """laga_mla_norm_rope: RMS norms of the query heads (over d_nope + d_rope, times q_weight) and of the
    shared RoPE key (times k_weight), and the rotation of rope in the same pass; returns (q, k_rope).
    Either may be None, with its weight (without k_rope, sections say how much of a head turns). q_out /
    k_out may be q / k_rope themselves."""
    d, (at, q_at, k_at, wq, wk), dts, dev = _norm_call(q, k_rope, pos, q_weight, k_weight, sections, theta, interleaved)
    q_out, qo = _made("q_out", q_out, q, dts, dev)
    k_out, ko = _made("k_out", k_out, k_rope, dts, dev)
    if d is not None:
        _launch(dev, lib().laga_mla_norm_rope, d, eps, at, q_at, k_at, wq, wk, qo, ko)
    return q_out, k_out


def norm_rope_bwd(dq_out, dk_out, q, k_rope, pos, q_weight, k_weight=None, eps: float = 1e-6, sections=None,
                  theta: float = 10000.0, interleaved: bool = True, workspace: torch.Tensor | None = None,
                  grads: dict | None = None):
    """laga_mla_norm_rope_bwd: dict dq, dk_rope, dw_q, dw_k from the gradients of norm_rope's results and
    its arguments (q and k_rope before the norm); what belongs to a None is left out. grads: tensors to
    write to by those names (dq may be dq_out or q, dk_rope may be dk_out or k_rope)."""
    d, (at, q_at, k_at, wq, wk), dts, dev = _norm_call(q, k_rope, pos, q_weight, k_weight, sections, theta, interleaved)
    zq = zk = None
    if q is not None:
        zq = _expect("dq_out", dq_out, q.shape, dts, dev)
    elif dq_out is not None:
        raise ValueError("dq_out without q")
    if k_rope is not None:
        zk = _expect("dk_out", dk_out, k_rope.shape, dts, dev)
    elif dk_out is not None:
        raise ValueError("dk_out without k_rope")
    given = (grads or {}).get
    res, to = {}, []
    for name, like in (("dq", q), ("dk_rope", k_rope), ("dw_q", q_weight), ("dw_k", k_weight)):
        t, address = _made(name, given(name), like, dts, dev)
        to.append(address)
        if t is not None:
            res[name] = t
    if d is None:  # no rows: nothing to sum
        for name in ("dw_q", "dw_k"):
            if name in res:
                res[name].zero_()
        return res
    nbytes = _norm_bwd_bytes(bytes(d))
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ws = workspace.data_ptr()
    else:
        ws = _expect("workspace", workspace, None, (workspace.dtype,), dev)
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
    _launch(dev, lib().laga_mla_norm_rope_bwd, d, eps, at, zq, zk, q_at, k_at, wq, wk, *to, ws, nbytes)
    return res


@functools.lru_cache(maxsize=256)
def _norm_bwd_bytes(desc: bytes) -> int:
    return int(lib().laga_mla_norm_rope_bwd_workspace_size(LagaRopeDesc.from_buffer_copy(desc)))


CACHE4_BLOCK = 16


@dataclass
class Cache4:
    """A paged pool of cached tokens: latents in 4 bits (codes uint8 [pages, page_size, ceil(d_c / 2)], scales
    uint8 [pages, page_size, ceil(d_c / 16)]; the format stands in laga_mla.h) and rotated RoPE keys
    [pages, page_size, d_rope], in the type of the calls' tensors."""
    codes: torch.Tensor
    scales: torch.Tensor
    k_rope: torch.Tensor
    d_c: int

    @property
    def page_size(self):
        return self.codes.shape[1]

    @property
    def device(self):
        return self.codes.device


def cache4(pages: int, page_size: int, d_c: int, d_rope: int, dtype=torch.bfloat16, device="cuda") -> Cache4:
    """An empty pool of `pages` pages."""
    _code_of(dtype)
    return Cache4(torch.zeros(pages, page_size, (d_c + 1) // 2, dtype=torch.uint8, device=device),
                  torch.zeros(pages, page_size, -(-d_c // CACHE4_BLOCK), dtype=torch.uint8, device=device),
                  torch.zeros(pages, page_size, d_rope, dtype=dtype, device=device), d_c)


def _check_cache(c: Cache4):
    """(descriptor, the tensors' allowed types, device)."""
    if c.codes.dim() != 3 or c.k_rope.dim() != 3:
        raise ValueError("a cache's tensors are [pages, page_size, ...]")
    pages, page = c.codes.shape[:2]
    dev, dt = c.codes.device, c.k_rope.dtype
    code = _code_of(dt)
    d_rope = c.k_rope.shape[2]
    codes = _expect("cache.codes", c.codes, (pages, page, (c.d_c + 1) // 2), _UINT8, dev)
    scales = _expect("cache.scales", c.scales, (pages, page, -(-c.d_c // CACHE4_BLOCK)), _UINT8, dev)
    keys = _expect("cache.k_rope", c.k_rope, (pages, page, d_rope), (dt,), dev)
    return LagaCache4(codes, scales, keys if d_rope else None, pages, page, c.d_c, d_rope, code), (dt,), dev


def _table(table, dev):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [B, max_pages]")
    return _expect("table", table, None, _INT32, dev)


def cache4_append(cache: Cache4, c_kv, k_rope, table, starts, counts=None, k_weight=None, eps: float = 1e-6, pos=None,
                  sections=None, theta: float | None = 10000.0, interleaved: bool = True) -> None:
    """laga_mla_cache4_append: writes rows i < counts[b] (None: all) of c_kv [B, S, d_c] and k_rope [B, S, d_rope]
    to positions starts[b] + i of sequence b, whose pages are table[b] (int32 [B, max_pages]; starts, counts int32
    [B]). The latents are stored in 4 bits; the keys are normed with k_weight (None: not) and rotated as by rope,
    by pos [n_axes, B, S] or by their positions in the sequence (theta None: stored as they come)."""
    d, dts, dev = _check_cache(cache)
    d_rope = d.d_rope
    if c_kv.dim() != 3:
        raise ValueError("expected c_kv [B,S,d_c]")
    B, S = c_kv.shape[:2]
    c_at = _expect("c_kv", c_kv, (B, S, cache.d_c), dts, dev)
    k_at = _expect("k_rope", k_rope, (B, S, d_rope), dts, dev)
    t_at = _table(table, dev)
    if table.shape[0] != B:
        raise ValueError("table has a row for each sequence")
    s_at = _expect("starts", starts, (B,), _INT32, dev)
    n_at = None if counts is None else _expect("counts", counts, (B,), _INT32, dev)
    w_at = None if k_weight is None else _expect("k_weight", k_weight, (d_rope,), dts, dev)
    rope_desc = p_at = None
    if theta is not None and d_rope and B * S:
        axes = 1 if pos is None else pos.shape[0]
        sections = (d_rope // 2,) if sections is None else tuple(map(int, sections))
        if len(sections) != axes or axes > ROPE_MAX_AXES:
            raise ValueError(f"one section per axis of pos (one without pos), at most {ROPE_MAX_AXES}")
        if pos is not None:
            p_at = _expect("pos", pos, (axes, B, S), (torch.int32, torch.int64), dev)
        rope_desc = _rope_desc((B, S, 1, d_rope), d_rope, sections, float(theta), bool(interleaved), False,
                               pos is not None and pos.dtype == torch.int64, d.dtype)
    elif pos is not None:
        raise ValueError("pos without a rotation")
    if B * S:
        _launch(dev, lib().laga_mla_cache4_append, d, B, S, table.shape[1], t_at, s_at, n_at, c_at,
                k_at if d_rope else None, w_at, eps, rope_desc, p_at)


def cache4_read(cache: Cache4, table, starts, rows: int, counts=None, c_kv=None, k_rope=None):
    """laga_mla_cache4_read: (c_kv [B, rows, d_c], k_rope [B, rows, d_rope]), the values that positions
    starts[b] + i, i < counts[b] (None: rows), of the cache stand for; zeros past counts[b]. c_kv / k_rope: tensors
    to write to."""
    d, dts, dev = _check_cache(cache)
    t_at = _table(table, dev)
    B, rows = table.shape[0], int(rows)
    s_at = _expect("starts", starts, (B,), _INT32, dev)
    n_at = None if counts is None else _expect("counts", counts, (B,), _INT32, dev)
    if c_kv is None:
        c_kv = torch.empty((B, rows, cache.d_c), dtype=dts[0], device=dev)
    if k_rope is None:
        k_rope = torch.empty((B, rows, d.d_rope), dtype=dts[0], device=dev)
    c_at = _expect("c_kv", c_kv, (B, rows, cache.d_c), dts, dev)
    k_at = _expect("k_rope", k_rope, (B, rows, d.d_rope), dts, dev)
    if B * rows:
        _launch(dev, lib().laga_mla_cache4_read, d, B, rows, table.shape[1], t_at, s_at, n_at, c_at,
                k_at if d.d_rope else None)
    return c_kv, k_rope


@functools.lru_cache(maxsize=256)
def _cache4_plan(q_shape, wk_shape, wv_shape, pages, page_size, d_c, d_rope, code, max_pages, causal, softmax_scale,
                 variant):
    """What a cached call's sizes decide: the descriptor, d_nope, d_v and the workspace's bytes."""
    if len(q_shape) != 4 or len(wk_shape) != 2 or len(wv_shape) != 2:
        raise ValueError("expected q [B,Sq,n_h,d_nope+d_rope], W_UK [d_c,n_h*d_nope], W_UV [d_c,n_h*d_v]")
    B, Sq, n_h, d_qk = q_shape
    if wk_shape[0] != d_c or wv_shape[0] != d_c:
        raise ValueError("W_UK and W_UV have a row for each latent column of the cache")
    if n_h < 1 or wk_shape[1] % n_h or wv_shape[1] % n_h:
        raise ValueError("W_UK / W_UV columns must be n_h * head width")
    d_nope, d_v = wk_shape[1] // n_h, wv_shape[1] // n_h
    if d_nope + d_rope != d_qk:
        raise ValueError("q's last dim must be d_nope + the cache's d_rope")
    d = LagaCache4Desc(B, Sq, n_h, d_nope, d_v, max_pages, causal, softmax_scale or 0.0, VARIANTS[variant])
    nbytes = 0
    if B * Sq:
        nbytes = int(lib().laga_mla_cache4_fwd_workspace_size(d, LagaCache4(None, None, None, pages, page_size, d_c,
                                                                              d_rope, code)))
        if nbytes == 0:
            _raise_if(2)
    return d, d_v, nbytes


def _cache4_call(q, cache, W_UK, W_UV, table, causal, softmax_scale, variant):
    c, dts, dev = _check_cache(cache)
    at = (_expect("q", q, None, dts, dev), _expect("W_UK", W_UK, None, dts, dev), _expect("W_UV", W_UV, None, dts, dev))
    t_at = _table(table, dev)
    d, d_v, nbytes = _cache4_plan(tuple(q.shape), tuple(W_UK.shape), tuple(W_UV.shape), c.pages, c.page_size, c.d_c,
                                  c.d_rope, c.dtype, table.shape[1], bool(causal),
                                  None if softmax_scale is None else float(softmax_scale), variant)
    if table.shape[0] != q.shape[0]:
        raise ValueError("table has a row for each sequence")
    return c, dts, dev, at, t_at, d, d_v, nbytes


def cache4_workspace(q, cache: Cache4, W_UK, W_UV, table, causal: bool = True, softmax_scale: float | None = None,
                     variant: str = "auto") -> torch.Tensor:
    """A workspace for cache4_fwd of these sizes. Calls in flight at the same time, replayed graphs among them, need
    one each."""
    *_, dev, _, _, _, _, nbytes = _cache4_call(q, cache, W_UK, W_UV, table, causal, softmax_scale, variant)
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def cache4_fwd(q, cache: Cache4, W_UK, W_UV, table, lengths, key_lo=None, key_hi=None, softcap: float = 0.0, slopes=None,
               causal: bool = True, softmax_scale: float | None = None, variant: str = "auto",
               workspace: torch.Tensor | None = None, out=None, lse=None):
    """laga_mla_cache4_fwd: (out [B,Sq,n_h,d_v], lse [B,n_h,Sq] fp32) of the last Sq tokens of each sequence over its
    lengths[b] cached tokens (int32 [B]; the call's own among them), q normed and rotated. Query i is at position
    lengths[b] - Sq + i; causal, key_lo / key_hi (int32 [B, Sq]), softcap and slopes as for masked_fwd. The table
    (int32 [B, max_pages]) names each sequence's pages."""
    c, dts, dev, at, t_at, d, d_v, nbytes = _cache4_call(q, cache, W_UK, W_UV, table, causal, softmax_scale, variant)
    B, Sq, n_h, _ = q.shape
    n_at = _expect("lengths", lengths, (B,), _INT32, dev)
    m = LagaMods(None if key_lo is None else _expect("key_lo", key_lo, (B, Sq), _INT32, dev),
                 None if key_hi is None else _expect("key_hi", key_hi, (B, Sq), _INT32, dev),
                 None if slopes is None else _expect("slopes", slopes, (n_h,), _FP32, dev), softcap or 0.0)
    if out is None:
        out = torch.empty((B, Sq, n_h, d_v), dtype=dts[0], device=dev)
        o_at = out.data_ptr()
    else:
        o_at = _expect("out", out, (B, Sq, n_h, d_v), dts, dev)
    if lse is None:
        lse = torch.empty((B, n_h, Sq), dtype=torch.float32, device=dev)
        l_at = lse.data_ptr()
    else:
        l_at = _expect("lse", lse, (B, n_h, Sq), _FP32, dev)
    if B * Sq == 0:
        return out, lse
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ws = workspace.data_ptr()
    else:
        ws = _expect("workspace", workspace, None, (workspace.dtype,), dev)
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
    _launch(dev, lib().laga_mla_cache4_fwd, d, c, m, t_at, n_at, at[0], at[1], at[2], o_at, l_at, ws, nbytes)
    return out, lse


def check(device=None) -> None:
    """laga_mla_check on the current stream: raise on a device-side timeout, a cached position without a page, or a
    CUDA error."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    _raise_if(lib().laga_mla_check(_stream(dev)))


def selftest_timeout(device=None) -> None:
    """laga_mla_selftest_timeout on the current stream: enqueue a kernel whose
    bounded wait expires (about 2 s); the next check() raises LAGA_ERR_TIMEOUT."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    _raise_if(lib().laga_mla_selftest_timeout(_stream(dev)))


@dataclass
class StepBuffers:
    """Preallocated device buffers for repeated forward+backward steps of one
    problem. One workspace serves both calls: the backward reuses the K_nope/V
    the forward left in it."""
    p: Problem
    inputs: dict
    out: torch.Tensor
    lse: torch.Tensor
    grads: dict
    ws: torch.Tensor | None


def alloc_step(p: Problem, inputs: dict, variant: str = "auto") -> StepBuffers:
    dev = inputs["q"].device
    dt = inputs["q"].dtype
    out = torch.empty((p.B, p.Sq, p.n_h, p.d_v), dtype=dt, device=dev)
    lse = torch.empty((p.B, p.n_h, p.Sq), dtype=torch.float32, device=dev)
    grads = {"dq": torch.empty_like(inputs["q"]), "dc_kv": torch.empty_like(inputs["c_kv"]),
             "dk_rope": torch.empty_like(inputs["k_rope"]), "dW_UK": torch.empty_like(inputs["W_UK"]),
             "dW_UV": torch.empty_like(inputs["W_UV"])}
    nb = max(fwd_workspace_bytes(p, variant), bwd_workspace_bytes(p, variant))
    ws = torch.empty(nb, dtype=torch.uint8, device=dev) if nb else None
    return StepBuffers(p, inputs, out, lse, grads, ws)


def step(buf: StepBuffers, variant: str = "auto"):
    """One forward + backward pass of the attention block into preallocated buffers."""
    x, p = buf.inputs, buf.p
    fwd(x["q"], x["c_kv"], x["k_rope"], x["W_UK"], x["W_UV"], p.q_offset, p.causal, None, variant,
        buf.ws, buf.out, buf.lse, p.q_split, p.q_offset2)
    bwd(x["q"], x["c_kv"], x["k_rope"], x["W_UK"], x["W_UV"], buf.out, buf.lse, x["dout"], p.q_offset, p.causal,
        None, variant, buf.ws, buf.grads, reuse_kv=buf.ws is not None, q_split=p.q_split, q_offset2=p.q_offset2)
    return buf.out, buf.lse, buf.grads
