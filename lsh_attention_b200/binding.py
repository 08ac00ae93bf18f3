"""Thin Python binding of the C ABI in include/lsh_attn.h.

Argument marshalling only: every step of the computation runs in the CUDA
library liblshattn.so. PyTorch supplies device memory (inputs, outputs and
the workspace) and the current CUDA stream. There is no fallback: if the
library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblshattn.so")

LSH_F32, LSH_BF16 = 0, 1
PROFILE_EVENTS = 10  # LSH_ATTN_PROFILE_EVENTS
#: what ends at each profiling event after the first
PROFILE_KERNELS = ("hash_prep", "hash_mma", "hash_refine", "sort_hist", "sort_scan",
                   "sort_rank", "gather_or_norm", "chunk_attention", "unsort_merge")
_DTYPES = {torch.float32: LSH_F32, torch.bfloat16: LSH_BF16}

#: every symbol the header declares
EXPORTS = ("lsh_attn_workspace_size", "lsh_attn_hash", "lsh_attn_sort", "lsh_attn_forward",
           "lsh_attn_forward_profiled", "lsh_attn_get_device_status", "lsh_attn_get_diag",
           "lsh_attn_sort_noalloc", "lsh_attn_selftest_wait_timeout",
           "lsh_attn_dense_workspace_size", "lsh_attn_dense_forward",
           "lsh_attn_backward_workspace_size", "lsh_attn_backward", "lsh_rev_workspace_size",
           "lsh_rev_block", "lsh_topk_workspace_size", "lsh_topk_forward", "lsh_rope",
           "lsh_cache_append", "lsh_cache_gather", "lsh_cache_attend_workspace_size",
           "lsh_cache_attend",
           "lsh_attn_status_string")


class LshAttnDesc(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in
                ("batch", "heads", "n", "d", "n_buckets", "chunk", "rounds", "causal", "dtype")]


class LshAttnDiag(ctypes.Structure):
    _fields_ = [(k, ctypes.c_uint32) for k in
                ("status", "hash_refined", "bad_bucket_ids", "reserved")]


class LshRevDesc(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in
                ("batch", "n", "d_model", "heads", "d_head", "d_ff", "ffn_chunk", "n_buckets",
                 "chunk", "rounds", "causal", "hash_buckets")]


class LshRevWeights(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("w_qk", "w_v", "w_o", "w1", "b1", "w2", "b2")]


class LshTopkDesc(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in
                ("batch", "heads", "n", "d", "n_buckets", "n_bits", "top_k", "rounds", "causal")]


LSH_CACHE_BF16, LSH_CACHE_I8 = 0, 1
ROPE_MAX_AXES = 4  # LSH_ROPE_MAX_AXES


class LshRopeAxes(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int32), ("dims", ctypes.c_int32 * ROPE_MAX_AXES),
                ("adjacent", ctypes.c_int32)]


class LshRopeDesc(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_int32) for k in
                 ("batch", "heads", "n", "d", "dtype", "inverse", "pos_batched")] +
                [("rot", LshRopeAxes), ("x_stride", ctypes.c_int64 * 3),
                 ("out_stride", ctypes.c_int64 * 3)])


class LshCacheDesc(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("pages", "heads", "page_size", "d", "format")]


class LshCacheMemory(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in
                ("k", "v", "key_inv_norm", "k_scale", "v_scale", "status")]


class LshCacheRows(ctypes.Structure):
    _fields_ = ([(k, ctypes.c_int32) for k in ("batch", "n", "max_pages", "pos_batched")] +
                [(k, ctypes.c_int64 * 3) for k in ("x_stride", "v_stride", "out_stride")])


class LshAttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load liblshattn.so; raise if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise ImportError(f"{_LIB_PATH} is missing: build it with "
                                  "`python -m lsh_attention_b200.build`")
            lib = ctypes.CDLL(_LIB_PATH)
            vp, sz = ctypes.c_void_p, ctypes.c_size_t
            dp = ctypes.POINTER(LshAttnDesc)
            lib.lsh_attn_workspace_size.argtypes = [dp, ctypes.POINTER(sz)]
            lib.lsh_attn_hash.argtypes = [dp, vp, vp, vp, vp, sz, vp]
            lib.lsh_attn_sort.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            lib.lsh_attn_forward.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            lib.lsh_attn_forward_profiled.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                                      ctypes.POINTER(ctypes.c_void_p)]
            lib.lsh_attn_get_device_status.argtypes = [vp, vp]
            lib.lsh_attn_sort_noalloc.argtypes = [dp, vp, vp, vp]
            lib.lsh_attn_get_diag.argtypes = [vp, vp, ctypes.POINTER(LshAttnDiag)]
            lib.lsh_attn_selftest_wait_timeout.argtypes = [vp, sz, ctypes.c_uint32, vp]
            lib.lsh_attn_dense_workspace_size.argtypes = [dp, ctypes.POINTER(sz)]
            lib.lsh_attn_dense_forward.argtypes = [dp, vp, vp, vp, vp, vp, sz, vp]
            lib.lsh_attn_backward_workspace_size.argtypes = [dp, ctypes.POINTER(sz)]
            lib.lsh_attn_backward.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
            lib.lsh_rev_workspace_size.argtypes = [ctypes.POINTER(LshRevDesc),
                                                   ctypes.POINTER(sz)]
            lib.lsh_rev_block.argtypes = [ctypes.POINTER(LshRevDesc), ctypes.c_int, vp, vp,
                                          ctypes.POINTER(LshRevWeights), vp, vp, vp, vp, vp, sz,
                                          vp]
            lib.lsh_topk_workspace_size.argtypes = [ctypes.POINTER(LshTopkDesc),
                                                    ctypes.POINTER(sz)]
            lib.lsh_topk_forward.argtypes = [ctypes.POINTER(LshTopkDesc), vp, vp, vp, vp, vp, vp,
                                             vp, sz, vp]
            lib.lsh_rope.argtypes = [ctypes.POINTER(LshRopeDesc), vp, vp, vp, vp, vp]
            cp, mp, rp = (ctypes.POINTER(t) for t in (LshCacheDesc, LshCacheMemory, LshCacheRows))
            lib.lsh_cache_append.argtypes = [cp, mp, rp, ctypes.POINTER(LshRopeAxes)] + [vp] * 9
            lib.lsh_cache_gather.argtypes = [cp, mp, rp] + [vp] * 6
            lib.lsh_cache_attend_workspace_size.argtypes = [cp, rp, ctypes.POINTER(sz)]
            lib.lsh_cache_attend.argtypes = [cp, mp, rp] + [vp] * 7 + [sz, vp]
            lib.lsh_attn_status_string.argtypes = [ctypes.c_int]
            lib.lsh_attn_status_string.restype = ctypes.c_char_p
            for f in EXPORTS[:-1]:
                getattr(lib, f).restype = ctypes.c_int
            _lib = lib
    return _lib


def _check(status: int) -> None:
    if status != 0:
        msg = load().lsh_attn_status_string(status).decode()
        raise LshAttnError(status, msg)


def make_desc(batch, heads, n, d, n_buckets, chunk, rounds, causal, dtype) -> LshAttnDesc:
    if isinstance(dtype, torch.dtype):
        if dtype not in _DTYPES:
            raise TypeError(f"unsupported dtype {dtype}")
        dtype = _DTYPES[dtype]
    return LshAttnDesc(batch, heads, n, d, n_buckets, chunk, rounds, int(bool(causal)), dtype)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _on_current_device(stream=None, **tensors) -> None:
    """The library launches on the current CUDA device and dereferences every
    pointer there: raise ValueError, before anything is launched, unless every
    given tensor (and the stream, if one is given) lives on that device."""
    cur = torch.cuda.current_device()
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device.index != cur:
            raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{cur}; "
                             f"call inside `with torch.cuda.device({t.device})`")
    if stream is not None and stream.device.index != cur:
        raise ValueError(f"stream is on {stream.device}, but the current device is cuda:{cur}")


def _require(t: torch.Tensor, name: str, dtype, shape) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def lsh_attn_workspace_size(desc: LshAttnDesc) -> int:
    out = ctypes.c_size_t(0)
    _check(load().lsh_attn_workspace_size(ctypes.byref(desc), ctypes.byref(out)))
    return out.value


_ws_cache: dict = {}


def workspace(desc: LshAttnDesc, device, stream=None) -> torch.Tensor:
    """A cached workspace of at least the size `desc` needs, one per
    (device, stream): calls that may run concurrently must not share one."""
    return _scratch(device, stream, lsh_attn_workspace_size(desc))


def lsh_attn_hash(x, R, n_buckets: int, buckets=None, ws=None, stream=None):
    """Bucket ids [B, H, rounds, n] int32 of x [B, H, n, d] under R [rounds, d, nb/2]."""
    _on_current_device(stream, x=x, R=R, buckets=buckets, ws=ws)
    B, H, n, d = x.shape
    rounds = R.shape[0]
    _require(x, "x", None, None)
    _require(R, "R", x.dtype, (rounds, d, n_buckets // 2))
    desc = make_desc(B, H, n, d, n_buckets, 1, rounds, False, x.dtype)
    if buckets is None:
        buckets = torch.empty((B, H, rounds, n), dtype=torch.int32, device=x.device)
    _require(buckets, "buckets", torch.int32, (B, H, rounds, n))
    if ws is None:
        ws = workspace(desc, x.device, stream)
    _check(load().lsh_attn_hash(ctypes.byref(desc), _ptr(x), _ptr(R), _ptr(buckets), _ptr(ws),
                                ws.numel(), _stream(stream)))
    return buckets


def lsh_attn_sort(buckets, n_buckets: int, x=None, v=None, perm=None, xs=None, vs=None, ws=None,
                  stream=None, d: int = 64, dtype=torch.bfloat16):
    """Stable sort by (bucket, position) of every (batch, head, round).
    Returns perm [B, H, rounds, n] int32, and (xs, vs) sorted row copies when
    x and v are given."""
    _on_current_device(stream, buckets=buckets, x=x, v=v, perm=perm, xs=xs, vs=vs, ws=ws)
    B, H, rounds, n = buckets.shape
    _require(buckets, "buckets", torch.int32, None)
    if x is not None:
        _require(x, "x", None, (B, H, n, x.shape[-1]))
        _require(v, "v", x.dtype, tuple(x.shape))
        d, dtype = x.shape[-1], x.dtype
    desc = make_desc(B, H, n, d, n_buckets, 1, rounds, False, dtype)
    if perm is None:
        perm = torch.empty((B, H, rounds, n), dtype=torch.int32, device=buckets.device)
    _require(perm, "perm", torch.int32, (B, H, rounds, n))
    if x is not None:
        if xs is None:
            xs = torch.empty((B, H, rounds, n, d), dtype=dtype, device=x.device)
        if vs is None:
            vs = torch.empty((B, H, rounds, n, d), dtype=dtype, device=x.device)
        _require(xs, "xs", dtype, (B, H, rounds, n, d))
        _require(vs, "vs", dtype, (B, H, rounds, n, d))
    if ws is None:
        ws = workspace(desc, buckets.device, stream)
    _check(load().lsh_attn_sort(ctypes.byref(desc), _ptr(buckets), _ptr(x), _ptr(v), _ptr(perm),
                                _ptr(xs), _ptr(vs), _ptr(ws), ws.numel(), _stream(stream)))
    return (perm, xs, vs) if x is not None else perm


def lsh_attn_forward(x, v, R=None, *, n_buckets: int, chunk: int, causal: bool, rounds=None,
                     buckets=None, out=None, lse=None, ws=None, stream=None, events=None):
    """LSH-attention forward. x, v [B, H, n, d]; R [rounds, d, nb/2] (or
    caller buckets [B, H, rounds, n]). Returns (out [B, H, n, d], lse
    [B, H, rounds, n] fp32). `events`: PROFILE_EVENTS recorded
    torch.cuda.Event objects marking the kernel boundaries
    (lsh_attn_forward_profiled)."""
    _on_current_device(stream, x=x, v=v, R=R, buckets=buckets, out=out, lse=lse, ws=ws)
    B, H, n, d = x.shape
    _require(x, "x", None, None)
    _require(v, "v", x.dtype, tuple(x.shape))
    if buckets is not None:
        rounds = buckets.shape[2]
        _require(buckets, "buckets", torch.int32, (B, H, rounds, n))
    else:
        if R is None:
            raise ValueError("either R or buckets is required")
        rounds = R.shape[0]
        _require(R, "R", x.dtype, (rounds, d, n_buckets // 2))
    desc = make_desc(B, H, n, d, n_buckets, chunk, rounds, causal, x.dtype)
    if out is None:
        out = torch.empty_like(x)
    if lse is None:
        lse = torch.empty((B, H, rounds, n), dtype=torch.float32, device=x.device)
    _require(out, "out", x.dtype, tuple(x.shape))
    _require(lse, "lse", torch.float32, (B, H, rounds, n))
    if ws is None:
        ws = workspace(desc, x.device, stream)
    args = (ctypes.byref(desc), _ptr(x), _ptr(v), _ptr(R), _ptr(buckets), _ptr(out), _ptr(lse),
            _ptr(ws), ws.numel(), _stream(stream))
    if events is None:
        _check(load().lsh_attn_forward(*args))
    else:
        if len(events) != PROFILE_EVENTS or any(e.cuda_event == 0 for e in events):
            raise ValueError(f"events: {PROFILE_EVENTS} torch.cuda.Event objects, each recorded once")
        ev = (ctypes.c_void_p * PROFILE_EVENTS)(*[e.cuda_event for e in events])
        _check(load().lsh_attn_forward_profiled(*args, ev))
    return out, lse


def lsh_attn_dense_forward(x, v, *, causal: bool, out=None, lse=None, ws=None, stream=None):
    """Dense shared-QK attention (the full-attention baseline) of x, v
    [B, H, n, d] bf16. Returns (out [B, H, n, d], lse [B, H, n] fp32)."""
    _on_current_device(stream, x=x, v=v, out=out, lse=lse, ws=ws)
    B, H, n, d = x.shape
    _require(x, "x", torch.bfloat16, None)
    _require(v, "v", torch.bfloat16, tuple(x.shape))
    desc = make_desc(B, H, n, d, 2, 1, 1, causal, x.dtype)
    if out is None:
        out = torch.empty_like(x)
    if lse is None:
        lse = torch.empty((B, H, n), dtype=torch.float32, device=x.device)
    _require(out, "out", torch.bfloat16, tuple(x.shape))
    _require(lse, "lse", torch.float32, (B, H, n))
    need = ctypes.c_size_t(0)
    _check(load().lsh_attn_dense_workspace_size(ctypes.byref(desc), ctypes.byref(need)))
    if ws is None:
        ws = _scratch(x.device, stream, need.value)
    elif ws.numel() < need.value:
        raise ValueError(f"ws: {need.value} bytes needed, {ws.numel()} given")
    _check(load().lsh_attn_dense_forward(ctypes.byref(desc), _ptr(x), _ptr(v), _ptr(out),
                                         _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))
    return out, lse


def lsh_attn_backward(x, v, buckets, out, lse, dout, *, n_buckets: int, chunk: int,
                      causal: bool, dlse=None, dx=None, dv=None, ws=None, stream=None):
    """Gradients (dx, dv) [B, H, n, d] of lsh_attn_forward(x, v, buckets=...)
    for upstream dout [B, H, n, d] (and dlse [B, H, rounds, n], or None),
    given that forward's out and lse."""
    _on_current_device(stream, x=x, v=v, buckets=buckets, out=out, lse=lse, dout=dout, dlse=dlse,
                       dx=dx, dv=dv, ws=ws)
    B, H, n, d = x.shape
    rounds = buckets.shape[2]
    _require(x, "x", None, None)
    for name, t in (("v", v), ("out", out), ("dout", dout)):
        _require(t, name, x.dtype, tuple(x.shape))
    _require(buckets, "buckets", torch.int32, (B, H, rounds, n))
    _require(lse, "lse", torch.float32, (B, H, rounds, n))
    if dlse is not None:
        _require(dlse, "dlse", torch.float32, (B, H, rounds, n))
    desc = make_desc(B, H, n, d, n_buckets, chunk, rounds, causal, x.dtype)
    if dx is None:
        dx = torch.empty_like(x)
    if dv is None:
        dv = torch.empty_like(x)
    _require(dx, "dx", x.dtype, tuple(x.shape))
    _require(dv, "dv", x.dtype, tuple(x.shape))
    need = ctypes.c_size_t(0)
    _check(load().lsh_attn_backward_workspace_size(ctypes.byref(desc), ctypes.byref(need)))
    if ws is None:
        ws = _scratch(x.device, stream, need.value)
    elif ws.numel() < need.value:
        raise ValueError(f"ws: {need.value} bytes needed, {ws.numel()} given")
    _check(load().lsh_attn_backward(ctypes.byref(desc), _ptr(x), _ptr(v), _ptr(buckets),
                                    _ptr(out), _ptr(lse), _ptr(dout), _ptr(dlse), _ptr(dx),
                                    _ptr(dv), _ptr(ws), ws.numel(), _stream(stream)))
    return dx, dv


def lsh_rev_block(in1, in2, weights: dict, *, heads: int, n_buckets: int, rounds: int,
                  causal: bool, ffn_chunk: int, R=None, buckets=None, inverse: bool = False,
                  out1=None, out2=None, ws=None, stream=None, chunk: int = 64):
    """Reversible layer: forward (x1, x2) -> (y1, y2), or inverse (y1, y2) ->
    (x1, x2), [B, n, d_model] bf16. weights: w_qk, w_v, w_o [d_model][d_model],
    w1 [d_ff][d_model], b1 [d_ff], w2 [d_model][d_ff], b2 [d_model] (bf16
    weights, fp32 biases). Forward without `buckets` hashes them (R needed)
    and returns them. Returns (out1, out2, buckets)."""
    W = weights
    _on_current_device(stream, in1=in1, in2=in2, R=R, buckets=buckets, out1=out1, out2=out2,
                       ws=ws, **W)
    B, n, dm = in1.shape
    dh = dm // heads
    d_ff = W["w1"].shape[0]
    for name, t in (("in1", in1), ("in2", in2)):
        _require(t, name, torch.bfloat16, (B, n, dm))
    for name, shape in (("w_qk", (dm, dm)), ("w_v", (dm, dm)), ("w_o", (dm, dm)),
                        ("w1", (d_ff, dm)), ("w2", (dm, d_ff))):
        _require(W[name], name, torch.bfloat16, shape)
    for name, shape in (("b1", (d_ff,)), ("b2", (dm,))):
        if W.get(name) is not None:
            _require(W[name], name, torch.float32, shape)
    hash_buckets = not inverse and buckets is None
    if buckets is None:
        if inverse:
            raise ValueError("the inverse needs the forward's bucket ids")
        if R is None:
            raise ValueError("either R or buckets is required")
        buckets = torch.empty((B, heads, rounds, n), dtype=torch.int32, device=in1.device)
    _require(buckets, "buckets", torch.int32, (B, heads, rounds, n))
    if R is not None:
        _require(R, "R", torch.bfloat16, (rounds, dh, n_buckets // 2))
    desc = LshRevDesc(B, n, dm, heads, dh, d_ff, ffn_chunk, n_buckets, chunk, rounds,
                      int(bool(causal)), int(hash_buckets))
    wts = LshRevWeights(*[ctypes.c_void_p(0 if W.get(k) is None else W[k].data_ptr())
                          for k in ("w_qk", "w_v", "w_o", "w1", "b1", "w2", "b2")])
    out1 = torch.empty_like(in1) if out1 is None else out1
    out2 = torch.empty_like(in2) if out2 is None else out2
    _require(out1, "out1", torch.bfloat16, (B, n, dm))
    _require(out2, "out2", torch.bfloat16, (B, n, dm))
    need = ctypes.c_size_t(0)
    _check(load().lsh_rev_workspace_size(ctypes.byref(desc), ctypes.byref(need)))
    if ws is None:
        ws = _scratch(in1.device, stream, need.value)
    elif ws.numel() < need.value:
        raise ValueError(f"ws: {need.value} bytes needed, {ws.numel()} given")
    _check(load().lsh_rev_block(ctypes.byref(desc), int(bool(inverse)), _ptr(in1), _ptr(in2),
                                ctypes.byref(wts), _ptr(R), _ptr(buckets), _ptr(out1), _ptr(out2),
                                _ptr(ws), ws.numel(), _stream(stream)))
    return out1, out2, buckets


def lsh_topk_forward(x, v, proj, *, n_buckets: int, top_k: int, causal: bool,
                     return_candidates: bool = False, out=None, lse=None, ws=None, stream=None):
    """The in-bucket top-k variant: x, v [B, H, n, d] bf16, proj [rounds, d,
    n_bits] bf16. Returns (out, lse [B, H, n]) and, if asked, the candidates
    [B, H, rounds, n, top_k] int32 (-1 past the kept ones)."""
    _on_current_device(stream, x=x, v=v, proj=proj, out=out, lse=lse, ws=ws)
    B, H, n, d = x.shape
    L, _, m = proj.shape
    _require(x, "x", torch.bfloat16, None)
    _require(v, "v", torch.bfloat16, tuple(x.shape))
    _require(proj, "proj", torch.bfloat16, (L, d, m))
    desc = LshTopkDesc(B, H, n, d, n_buckets, m, top_k, L, int(bool(causal)))
    out = torch.empty_like(x) if out is None else out
    lse = torch.empty((B, H, n), dtype=torch.float32, device=x.device) if lse is None else lse
    _require(out, "out", torch.bfloat16, tuple(x.shape))
    _require(lse, "lse", torch.float32, (B, H, n))
    cand = (torch.empty((B, H, L, n, top_k), dtype=torch.int32, device=x.device)
            if return_candidates else None)
    need = ctypes.c_size_t(0)
    _check(load().lsh_topk_workspace_size(ctypes.byref(desc), ctypes.byref(need)))
    if ws is None:
        ws = _scratch(x.device, stream, need.value)
    elif ws.numel() < need.value:
        raise ValueError(f"ws: {need.value} bytes needed, {ws.numel()} given")
    _check(load().lsh_topk_forward(ctypes.byref(desc), _ptr(x), _ptr(v), _ptr(proj), _ptr(out),
                                   _ptr(lse), _ptr(cand), _ptr(ws), ws.numel(), _stream(stream)))
    return (out, lse, cand) if return_candidates else (out, lse)


def _rows_strides(t, name: str, dtype, shape) -> tuple:
    """(batch, head, position) strides of rows [B, H, n, d] whose d values are contiguous."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # an axis of one entry is never stepped along; torch gives it any stride
    return (s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0, s[2] if shape[2] > 1 else 0)


@functools.lru_cache(maxsize=None)
def _axes(axis_dims: tuple, adjacent: bool) -> LshRopeAxes:
    return LshRopeAxes(len(axis_dims), (ctypes.c_int32 * ROPE_MAX_AXES)(*axis_dims),
                       int(adjacent))


def _check_angles(positions, freqs, axis_dims: tuple, B: int, n: int) -> bool:
    """Check positions [axes, B, n] or [axes, n] and freqs; whether positions have a batch axis."""
    if len(axis_dims) > ROPE_MAX_AXES:
        raise ValueError(f"axis_dims: at most {ROPE_MAX_AXES} axes, got {len(axis_dims)}")
    batched = positions.dim() == 3
    _require(positions, "positions", torch.int32,
             (len(axis_dims), B, n) if batched else (len(axis_dims), n))
    _require(freqs, "freqs", torch.float32, (sum(a // 2 for a in axis_dims),))
    return batched


def _raw_stream(device) -> int:
    """Handle of the device's current stream: what _stream(None) gives, without making a Stream
    object (which takes longer than a small kernel)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _on_stream(stream, call, *tensors):
    """Run call() with `stream` current, its results made in that stream's memory; the tensors
    are not handed out again before the stream has passed."""
    with torch.cuda.stream(stream):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return call()


#: what a call's checks found, by what they looked at: shapes, strides, types and devices of its
#: tensors (nothing of their memory). A step of a loop is checked once.
_plans: dict = {}


def _seen(*tensors) -> tuple:
    """What the checks look at of every tensor."""
    return tuple([None if t is None else (t.shape, t.stride(), t.dtype, t.device)
                  for t in tensors])


def _keep(key, plan):
    if len(_plans) >= 4096:
        _plans.clear()
    _plans[key] = plan
    return plan


def lsh_rope(x, positions, freqs, *, axis_dims, adjacent: bool = False, inverse: bool = False,
             out=None, stream=None):
    """Rotary positions on the rows of x [B, H, n, d] (fp32 or bf16; any strides with the last
    dimension contiguous). Axis a turns axis_dims[a] dimensions by positions[a] * freqs;
    positions int32 [axes, B, n] or [axes, n], freqs fp32 [sum(axis_dims) / 2] (one frequency
    for each pair). `adjacent`: pairs are neighbouring dimensions, else the halves of an axis.
    `inverse` turns back, which is the gradient with respect to x. Returns out [B, H, n, d];
    out may be x itself."""
    if stream is not None:
        _on_current_device(stream, x=x, positions=positions, freqs=freqs, out=out)
        return _on_stream(stream, lambda: lsh_rope(x, positions, freqs, axis_dims=axis_dims,
                                                   adjacent=adjacent, inverse=inverse, out=out),
                          x, positions, freqs, out)
    key = ("rope", torch.cuda.current_device(), tuple(axis_dims), adjacent, inverse,
           _seen(x, positions, freqs, out))
    desc = _plans.get(key) or _keep(key, _plan_rope(x, positions, freqs, key[2], adjacent, inverse,
                                                    out))
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    _check((_lib or load()).lsh_rope(desc, x.data_ptr(), positions.data_ptr(), freqs.data_ptr(),
                                     out.data_ptr(), _raw_stream(x.device)))
    return out


def _plan_rope(x, positions, freqs, axis_dims, adjacent, inverse, out):
    _on_current_device(None, x=x, positions=positions, freqs=freqs, out=out)
    B, H, n, d = shape = tuple(x.shape)
    if x.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    xs = _rows_strides(x, "x", x.dtype, shape)
    batched = _check_angles(positions, freqs, axis_dims, B, n)
    three = ctypes.c_int64 * 3
    os_ = (H * n * d, n * d, d) if out is None else _rows_strides(out, "out", x.dtype, shape)
    return ctypes.byref(LshRopeDesc(B, H, n, d, _DTYPES[x.dtype], int(inverse), batched,
                                    _axes(axis_dims, adjacent), three(*xs), three(*os_)))


class LshCache:
    """A paged cache of rows of x and v for every head, bf16 or int8 (see lsh_cache in
    lsh_attn.h for the layouts):

    k [pages, heads, page_size, d], v [pages, heads, page_size / 16, d, 16],
    key_inv_norm [pages, heads, page_size] fp32, and for int8 k_scale and v_scale
    [pages, heads] fp32. status: int32 [64], zeroed here; the calls record the first error they
    meet on the device there. `LshCache.empty` makes one."""

    def __init__(self, k, v, key_inv_norm, k_scale=None, v_scale=None, status=None):
        pages, heads, page, d = k.shape
        if k.dtype not in (torch.bfloat16, torch.int8):
            raise TypeError(f"k must be torch.bfloat16 or torch.int8, got {k.dtype}")
        self.int8 = k.dtype == torch.int8
        _require(k, "k", None, None)
        _require(v, "v", k.dtype, (pages, heads, page // 16, d, 16))
        _require(key_inv_norm, "key_inv_norm", torch.float32, (pages, heads, page))
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if self.int8 != (t is not None):
                raise ValueError(f"{name} belongs to an int8 cache, and to no other")
            if t is not None:
                _require(t, name, torch.float32, (pages, heads))
        if status is None:
            status = torch.zeros(64, dtype=torch.int32, device=k.device)
        _require(status, "status", torch.int32, (64,))
        self.k, self.v, self.key_inv_norm = k, v, key_inv_norm
        self.k_scale, self.v_scale, self.status = k_scale, v_scale, status
        self.tensors = {"k": k, "v": v, "key_inv_norm": key_inv_norm, "k_scale": k_scale,
                        "v_scale": v_scale, "status": status}
        if any(t is not None and t.device != k.device for t in self.tensors.values()):
            raise ValueError("all of a cache lies on one device")
        self.pages, self.heads, self.page_size, self.d = pages, heads, page, d
        self.desc = LshCacheDesc(pages, heads, page, d,
                                 LSH_CACHE_I8 if self.int8 else LSH_CACHE_BF16)
        self.memory = LshCacheMemory(*[None if t is None else t.data_ptr()
                                       for t in self.tensors.values()])
        self.desc_ref, self.memory_ref = ctypes.byref(self.desc), ctypes.byref(self.memory)
        self.kind = (pages, heads, page, d, self.int8, k.device)

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, d: int, *, int8: bool = False,
              device="cuda") -> "LshCache":
        """A cache whose pages hold nothing yet."""
        dt = torch.int8 if int8 else torch.bfloat16
        scales = [torch.empty((pages, heads), dtype=torch.float32, device=device)
                  for _ in range(2)] if int8 else []
        return cls(torch.empty((pages, heads, page_size, d), dtype=dt, device=device),
                   torch.empty((pages, heads, page_size // 16, d, 16), dtype=dt, device=device),
                   torch.empty((pages, heads, page_size), dtype=torch.float32, device=device),
                   *scales)

    def get_device_status(self, stream=None) -> int:
        """Synchronise and return the first error recorded since the status was cleared."""
        return lsh_attn_get_device_status(self.status, stream)

    def clear_status(self) -> None:
        self.status.zero_()


def _check_tables(B: int, page_table, seq_len, n_valid, what: str = "seq_len") -> None:
    _require(page_table, "page_table", torch.int32, (B, page_table.shape[-1]))
    _require(seq_len, what, torch.int32, (B,))
    if n_valid is not None:
        _require(n_valid, "n_valid", torch.int32, (B,))


def _opt(t):
    return None if t is None else t.data_ptr()


def _cache_rows(B, n, max_pages, batched=False, xs=(0, 0, 0), vs=(0, 0, 0), os_=(0, 0, 0)):
    three = ctypes.c_int64 * 3
    return LshCacheRows(B, n, max_pages, batched, three(*xs), three(*vs), three(*os_))


def _new_rows(shape, t, name: str) -> tuple:
    """Strides of rows that the call returns: those of `t`, or of a new tensor."""
    B, H, n, d = shape
    return (H * n * d, n * d, d) if t is None else _rows_strides(t, name, torch.bfloat16, shape)


def lsh_cache_append(cache: LshCache, x, v, page_table, seq_len, *, n_valid=None, positions=None,
                     freqs=None, axis_dims=(), adjacent: bool = False, xr=None, stream=None):
    """Append the rows x, v [B, H, n, d] (bf16, any strides with the last dimension contiguous)
    as tokens seq_len .. of every sequence, x rotated on the way if `axis_dims` is given (as
    lsh_rope). page_table int32 [B, max_pages], seq_len int32 [B], n_valid int32 [B] or None
    (all n rows). Returns the rotated rows [B, H, n, d] (zeros past n_valid), the queries of
    lsh_cache_attend; without a rotation and without `xr`, x itself. xr may be x."""
    if stream is not None:
        _on_current_device(stream, x=x, v=v, page_table=page_table, seq_len=seq_len,
                           n_valid=n_valid, positions=positions, freqs=freqs, xr=xr, cache=cache.k)
        return _on_stream(
            stream, lambda: lsh_cache_append(
                cache, x, v, page_table, seq_len, n_valid=n_valid, positions=positions,
                freqs=freqs, axis_dims=axis_dims, adjacent=adjacent, xr=xr),
            x, v, page_table, seq_len, n_valid, positions, freqs, xr, *cache.tensors.values())
    key = ("append", torch.cuda.current_device(), cache.kind, tuple(axis_dims), adjacent,
           _seen(x, v, page_table, seq_len, n_valid, positions, freqs, xr))
    rows, rot = _plans.get(key) or _keep(key, _plan_append(
        cache, x, v, page_table, seq_len, n_valid, positions, freqs, key[3], adjacent, xr))
    if xr is None and axis_dims:
        xr = torch.empty_like(x, memory_format=torch.contiguous_format)
    _check((_lib or load()).lsh_cache_append(
        cache.desc_ref, cache.memory_ref, rows, rot, x.data_ptr(), v.data_ptr(), _opt(positions),
        _opt(freqs), page_table.data_ptr(), seq_len.data_ptr(), _opt(n_valid), _opt(xr),
        _raw_stream(x.device)))
    return x if xr is None else xr


def _plan_append(cache, x, v, page_table, seq_len, n_valid, positions, freqs, axis_dims, adjacent,
                 xr):
    _on_current_device(None, x=x, v=v, page_table=page_table, seq_len=seq_len, n_valid=n_valid,
                       positions=positions, freqs=freqs, xr=xr, cache=cache.k)
    B, H, n, d = shape = tuple(x.shape)
    if (H, d) != (cache.heads, cache.d):
        raise ValueError(f"x has {H} heads of {d}, the cache {cache.heads} of {cache.d}")
    xs = _rows_strides(x, "x", torch.bfloat16, shape)
    vs = _rows_strides(v, "v", torch.bfloat16, shape)
    _check_tables(B, page_table, seq_len, n_valid)
    batched, os_ = False, (0, 0, 0)
    if axis_dims:
        if positions is None or freqs is None:
            raise ValueError("a rotation needs positions and freqs")
        batched = _check_angles(positions, freqs, axis_dims, B, n)
    if axis_dims or xr is not None:
        os_ = _new_rows(shape, xr, "xr")
    return (ctypes.byref(_cache_rows(B, n, page_table.shape[1], batched, xs, vs, os_)),
            ctypes.byref(_axes(axis_dims, adjacent)))


def lsh_cache_gather(cache: LshCache, page_table, start, n: int, *, n_valid=None, x=None, v=None,
                     stream=None):
    """Read n rows from position start[b] of every sequence back as values. start int32 [B],
    n_valid int32 [B] or None. Returns x, v [B, H, n, d] bf16, zeros past n_valid."""
    if stream is not None:
        _on_current_device(stream, page_table=page_table, start=start, n_valid=n_valid, x=x, v=v,
                           cache=cache.k)
        return _on_stream(stream, lambda: lsh_cache_gather(cache, page_table, start, n,
                                                           n_valid=n_valid, x=x, v=v),
                          page_table, start, n_valid, x, v, *cache.tensors.values())
    key = ("gather", torch.cuda.current_device(), cache.kind, n,
           _seen(page_table, start, n_valid, x, v))
    rows, shape = _plans.get(key) or _keep(key, _plan_gather(cache, page_table, start, n, n_valid,
                                                             x, v))
    if x is None:
        x = torch.empty(shape, dtype=torch.bfloat16, device=page_table.device)
    if v is None:
        v = torch.empty(shape, dtype=torch.bfloat16, device=page_table.device)
    _check((_lib or load()).lsh_cache_gather(
        cache.desc_ref, cache.memory_ref, rows, page_table.data_ptr(), start.data_ptr(),
        _opt(n_valid), x.data_ptr(), v.data_ptr(), _raw_stream(page_table.device)))
    return x, v


def _plan_gather(cache, page_table, start, n, n_valid, x, v):
    _on_current_device(None, page_table=page_table, start=start, n_valid=n_valid, x=x, v=v,
                       cache=cache.k)
    B = page_table.shape[0]
    shape = (B, cache.heads, n, cache.d)
    _check_tables(B, page_table, start, n_valid, "start")
    return (ctypes.byref(_cache_rows(B, n, page_table.shape[1], False, _new_rows(shape, x, "x"),
                                     _new_rows(shape, v, "v"))), shape)


def lsh_cache_attend(cache: LshCache, x, page_table, seq_len, *, n_valid=None, out=None, lse=None,
                     ws=None, stream=None):
    """Shared-QK attention of the n newest tokens of every sequence over the cache, after
    lsh_cache_append has stored them: x [B, H, n, d] bf16, the rotated rows that it returned,
    with its page_table, seq_len (before those tokens) and n_valid. Returns out [B, H, n, d]
    bf16 and lse [B, H, n] fp32; rows past n_valid are zeros and -inf."""
    if stream is not None:
        _on_current_device(stream, x=x, page_table=page_table, seq_len=seq_len, n_valid=n_valid,
                           out=out, lse=lse, ws=ws, cache=cache.k)
        return _on_stream(stream, lambda: lsh_cache_attend(cache, x, page_table, seq_len,
                                                           n_valid=n_valid, out=out, lse=lse,
                                                           ws=ws),
                          x, page_table, seq_len, n_valid, out, lse, ws, *cache.tensors.values())
    key = ("attend", torch.cuda.current_device(), cache.kind,
           _seen(x, page_table, seq_len, n_valid, out, lse, ws))
    rows, need = _plans.get(key) or _keep(key, _plan_attend(cache, x, page_table, seq_len, n_valid,
                                                            out, lse, ws))
    device = x.device
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    if lse is None:
        lse = torch.empty(x.shape[:3], dtype=torch.float32, device=device)
    stream = _raw_stream(device)
    if ws is None and torch.cuda.is_current_stream_capturing():
        # a graph keeps its own workspace: the cached one may grow and go away
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    elif ws is None:
        ws = _ws_cache.get((device.index, stream))
        if ws is None or ws.numel() < need:
            ws = _scratch(device, None, need)
    _check((_lib or load()).lsh_cache_attend(
        cache.desc_ref, cache.memory_ref, rows, x.data_ptr(), page_table.data_ptr(),
        seq_len.data_ptr(), _opt(n_valid), out.data_ptr(), lse.data_ptr(), ws.data_ptr(),
        ws.numel() * ws.element_size(), stream))
    return out, lse


def _plan_attend(cache, x, page_table, seq_len, n_valid, out, lse, ws):
    _on_current_device(None, x=x, page_table=page_table, seq_len=seq_len, n_valid=n_valid, out=out,
                       lse=lse, ws=ws, cache=cache.k)
    B, H, n, d = shape = tuple(x.shape)
    if (H, d) != (cache.heads, cache.d):
        raise ValueError(f"x has {H} heads of {d}, the cache {cache.heads} of {cache.d}")
    xs = _rows_strides(x, "x", torch.bfloat16, shape)
    _check_tables(B, page_table, seq_len, n_valid)
    if lse is not None:
        _require(lse, "lse", torch.float32, (B, H, n))
    if ws is not None:
        _require(ws, "ws", None, None)
    rows = _cache_rows(B, n, page_table.shape[1], False, xs, (0, 0, 0), _new_rows(shape, out, "out"))
    need = ctypes.c_size_t(0)
    _check(load().lsh_cache_attend_workspace_size(cache.desc_ref, ctypes.byref(rows),
                                                  ctypes.byref(need)))
    return ctypes.byref(rows), need.value


def _scratch(device, stream, need: int) -> torch.Tensor:
    """The cached workspace of (device, stream), grown to `need` bytes."""
    dev = torch.device(device)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    key = (dev.index, s.cuda_stream)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < need:
        _ws_cache.pop(key, None)
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        _ws_cache[key] = ws
    return ws


def lsh_attn_sort_noalloc(buckets, n_buckets: int, perm=None, stream=None):
    """perm [B, H, rounds, n] of the stable bucket sort without any workspace:
    the library's fixed device scratch is used (see lsh_attn.h)."""
    _on_current_device(stream, buckets=buckets, perm=perm)
    B, H, rounds, n = buckets.shape
    _require(buckets, "buckets", torch.int32, None)
    desc = make_desc(B, H, n, 64, n_buckets, 1, rounds, False, torch.bfloat16)
    if perm is None:
        perm = torch.empty((B, H, rounds, n), dtype=torch.int32, device=buckets.device)
    _require(perm, "perm", torch.int32, (B, H, rounds, n))
    _check(load().lsh_attn_sort_noalloc(ctypes.byref(desc), _ptr(buckets), _ptr(perm),
                                        _stream(stream)))
    return perm


def lsh_attn_get_diag(ws, stream=None) -> dict:
    _on_current_device(stream, ws=ws)
    d = LshAttnDiag()
    _check(load().lsh_attn_get_diag(_ptr(ws), _stream(stream), ctypes.byref(d)))
    return {"status": d.status, "hash_refined": d.hash_refined,
            "bad_bucket_ids": d.bad_bucket_ids}


def lsh_attn_get_device_status(ws, stream=None) -> int:
    _on_current_device(stream, ws=ws)
    return load().lsh_attn_get_device_status(_ptr(ws), _stream(stream))


def lsh_attn_selftest_wait_timeout(ws, limit_us: int, stream=None) -> None:
    """Launch the bounded-wait self-test on `ws` (a uint8 CUDA tensor of at
    least 256 bytes): a wait that nothing completes gives up after
    `limit_us` and records LSH_ERR_TIMEOUT (read it with
    lsh_attn_get_device_status)."""
    _on_current_device(stream, ws=ws)
    _check(load().lsh_attn_selftest_wait_timeout(_ptr(ws), ws.numel() * ws.element_size(),
                                                 int(limit_us), _stream(stream)))
