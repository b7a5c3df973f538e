"""MI355X (gfx950) dynamic short convolution: Python binding of libdynconv.

Thin ctypes binding of the C ABI in ``include/dynconv.h``, with the same
names (``dynconv_fwd``, ``dynconv_bwd``, ``dynconv_decode``, ``dynconv_workspace_bytes``,
``dynconv_gen_cache_bytes``, ``dynconv_status_str``, ``dynconv_abi_version``).
It only marshals arguments: torch provides device memory (outputs and
workspace are ``torch.empty``) and the current HIP stream; every step of the
layer runs in the library's HIP kernels.  There is no CPU fallback: if the
library is not built this module raises on import of the binding.

The layer ("Dynamic Short Convolutions Improve Transformers", gist.science
Technical Summary, Methodology -> Dynamic Short Convolutions) is
``y = x + sum_j w_t[:, j] * x_{t-j}`` with the per-token filter ``w_t``
generated from the hidden state ``h_t`` head-wise (``W``) or low-rank
(``A``, ``U``), plus a static bias ``w0``.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch
from torch import _C
from torch.autograd.function import once_differentiable

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdynconv.so")

DYNCONV_FP32, DYNCONV_BF16 = 0, 1
DYNCONV_HEADWISE, DYNCONV_LOWRANK, DYNCONV_STATIC = 0, 1, 2
ABI_VERSION = 3
DYNCONV_WS_CACHED = 2  # or-ed into dynconv_workspace_bytes' pass when the call gets gen_cache


class DynConvError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {dynconv_status_str(status)} (status {status})")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("d_model", ctypes.c_int64),
                ("D", ctypes.c_int64), ("k", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("cu_seqlens", ctypes.c_void_p), ("n_seqs", ctypes.c_int64)]


class Gen(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("W", ctypes.c_void_p), ("A", ctypes.c_void_p),
                ("U", ctypes.c_void_p), ("w0", ctypes.c_void_p)]


class GenGrad(ctypes.Structure):
    _fields_ = [("dW", ctypes.c_void_p), ("dA", ctypes.c_void_p), ("dU", ctypes.c_void_p),
                ("dw0", ctypes.c_void_p)]


class View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class Attn(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int64)]


class Rotary(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("factor", ctypes.c_float), ("freqs", ctypes.c_void_p)]


# names the C header declares; the CPU tests check each is exported
EXPORTS = ("dynconv_fwd", "dynconv_fwd_proj", "dynconv_fwd_noalloc", "dynconv_bwd", "dynconv_decode", "dynconv_workspace_bytes",
           "dynconv_gen_cache_bytes", "dynconv_status_str", "dynconv_abi_version", "dynconv_trace_next",
           "dynconv_rope_freqs", "dynconv_rope", "dynconv_attn_fwd", "dynconv_attn_bwd_workspace_bytes",
           "dynconv_attn_bwd", "dynconv_attn_decode_workspace_bytes", "dynconv_attn_decode")
DYNCONV_E_SCRATCH = -10
NOALLOC_SCRATCH_BYTES = 16 << 20  # the static scratch of dynconv_fwd_noalloc

# kernel ids for dynconv_trace_next
DYNCONV_K_GEN_PROJ, DYNCONV_K_FWD_CONV, DYNCONV_K_BWD_CONV, DYNCONV_K_GEN_BWD, DYNCONV_K_FINALIZE = 1, 2, 3, 4, 5

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libdynconv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m input_dependent_depthwise_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        PP, PG, PGG = ctypes.POINTER(Problem), ctypes.POINTER(Gen), ctypes.POINTER(GenGrad)
        L.dynconv_fwd.argtypes = [PP, PG, P, P, P, P, P, ctypes.c_size_t, P]
        L.dynconv_fwd.restype = ctypes.c_int
        L.dynconv_fwd_proj.argtypes = [PP, PG, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.dynconv_fwd_proj.restype = ctypes.c_int
        L.dynconv_fwd_noalloc.argtypes = [PP, PG, P, P, P, P, P]
        L.dynconv_fwd_noalloc.restype = ctypes.c_int
        L.dynconv_bwd.argtypes = [PP, PG, P, P, P, P, P, P, PGG, P, ctypes.c_size_t, P]
        L.dynconv_bwd.restype = ctypes.c_int
        L.dynconv_decode.argtypes = [PP, PG, P, P, P, P, P]
        L.dynconv_decode.restype = ctypes.c_int
        L.dynconv_workspace_bytes.argtypes = [PP, PG, ctypes.c_int]
        L.dynconv_workspace_bytes.restype = ctypes.c_size_t
        L.dynconv_gen_cache_bytes.argtypes = [PP, PG]
        L.dynconv_gen_cache_bytes.restype = ctypes.c_size_t
        L.dynconv_status_str.argtypes = [ctypes.c_int]
        L.dynconv_status_str.restype = ctypes.c_char_p
        L.dynconv_abi_version.restype = ctypes.c_int
        L.dynconv_trace_next.argtypes = [ctypes.c_int, P, P]
        L.dynconv_trace_next.restype = ctypes.c_int
        PA = PR = PV = P  # Attn, Rotary and View, by reference or as packed bytes
        D, SZ, I64 = ctypes.c_double, ctypes.c_size_t, ctypes.c_int64
        L.dynconv_rope_freqs.argtypes = [ctypes.c_int, D, D, D, D, D, P]
        L.dynconv_rope.argtypes = [PA, PR, PV, P, PV, P]
        L.dynconv_attn_fwd.argtypes = [PA, PV, PV, PV, PV, P, P]
        L.dynconv_attn_bwd_workspace_bytes.argtypes = [PA]
        L.dynconv_attn_bwd_workspace_bytes.restype = SZ
        L.dynconv_attn_bwd.argtypes = [PA, PV, PV, PV, PV, P, PV, PV, PV, PV, P, SZ, P]
        L.dynconv_attn_decode_workspace_bytes.argtypes = [PA, I64]
        L.dynconv_attn_decode_workspace_bytes.restype = SZ
        L.dynconv_attn_decode.argtypes = [PA, PR, PV, PV, PV, PV, PV, I64, P, PV, P, SZ, P]
        _lib = L
    return _lib


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _dtype_code(dt) -> int:
    if dt == torch.float32:
        return DYNCONV_FP32
    if dt == torch.bfloat16:
        return DYNCONV_BF16
    raise TypeError(f"unsupported I/O dtype {dt}")


def make_problem(x: torch.Tensor, h, k: int, cu_seqlens=None) -> Problem:
    """Problem struct from x[B,T,D], h[B,T,d_model] and the filter width k.

    h may be None for the static filter (d_model 0).  cu_seqlens: None, or
    packed documents (B must be 1): an int32 device tensor of n_seqs + 1
    offsets rising from 0 to T."""
    if x.dim() != 3 or (h is not None and (h.dim() != 3 or h.shape[:2] != x.shape[:2])):
        raise ValueError(f"expected h[B,T,d] and x[B,T,D], got {None if h is None else tuple(h.shape)} "
                         f"and {tuple(x.shape)}")
    B, T, D = x.shape
    d = 0 if h is None else h.shape[2]
    if cu_seqlens is None:
        return Problem(B, T, d, D, int(k), _dtype_code(x.dtype), None, 0)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
        raise TypeError("cu_seqlens must be a contiguous 1-d int32 tensor")
    return Problem(B, T, d, D, int(k), _dtype_code(x.dtype), cu_seqlens.data_ptr(), cu_seqlens.numel() - 1)


def make_gen(W=None, A=None, U=None, w0=None, n_heads: int = 0) -> Gen:
    """Generator struct: head-wise when W is given, low-rank when A and U
    are, the static filter (w0 alone) when none of them is."""
    if W is None and A is None and U is None:
        if w0 is None:
            raise ValueError("the static filter needs w0")
        return Gen(DYNCONV_STATIC, 0, 0, 0, None, None, None, _ptr(w0))
    if W is not None:
        if n_heads <= 0:
            raise ValueError("head-wise generator needs n_heads")
        return Gen(DYNCONV_HEADWISE, int(n_heads), 0, 0, _ptr(W), None, None, _ptr(w0))
    if A is None or U is None:
        raise ValueError("pass W (head-wise) or both A and U (low-rank)")
    return Gen(DYNCONV_LOWRANK, 0, int(A.shape[1]), 0, None, _ptr(A), _ptr(U), _ptr(w0))


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, where: str):
    if rc != 0:
        raise DynConvError(rc, where)


def dynconv_status_str(status: int) -> str:
    return lib().dynconv_status_str(int(status)).decode()


def dynconv_abi_version() -> int:
    return int(lib().dynconv_abi_version())


def dynconv_trace_next(kernel: int, start, stop) -> None:
    """Arm a one-shot event pair around the next launch of ``kernel`` on this
    thread (torch.cuda.Event objects, or None to disarm)."""
    a = None if start is None else start.cuda_event
    b = None if stop is None else stop.cuda_event
    _check(lib().dynconv_trace_next(int(kernel), a, b), "dynconv_trace_next")


def dynconv_workspace_bytes(prob: Problem, gen: Gen, pass_: int) -> int:
    return int(lib().dynconv_workspace_bytes(ctypes.byref(prob), ctypes.byref(gen), int(pass_)))


def dynconv_gen_cache_bytes(prob: Problem, gen: Gen) -> int:
    return int(lib().dynconv_gen_cache_bytes(ctypes.byref(prob), ctypes.byref(gen)))


def _workspace(nbytes: int, device, workspace):
    if workspace is not None:
        if workspace.device != device or not workspace.is_contiguous():
            raise TypeError(f"workspace must be a contiguous tensor on {device}, got one on {workspace.device}")
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def dynconv_fwd(h, x, *, k, W=None, A=None, U=None, w0=None, n_heads=0, y=None, gen_cache=None,
                want_cache=False, workspace=None, stream=None, cu_seqlens=None):
    """Forward: returns y (and the fp32 generator cache when want_cache).
    cu_seqlens: packed documents in a single row (see make_problem)."""
    prob = make_problem(x, h, k, cu_seqlens)
    gen = make_gen(W, A, U, w0, n_heads)
    if y is None:
        y = torch.empty_like(x)
    if gen_cache is None and want_cache and gen.kind != DYNCONV_STATIC:
        n = gen.n_heads * k if gen.kind == DYNCONV_HEADWISE else gen.rank
        gen_cache = torch.empty(x.shape[0] * x.shape[1], n, dtype=torch.float32, device=x.device)
    nbytes = dynconv_workspace_bytes(prob, gen, 0 | (DYNCONV_WS_CACHED if gen_cache is not None else 0))
    ws = _workspace(nbytes, x.device, workspace)
    rc = lib().dynconv_fwd(ctypes.byref(prob), ctypes.byref(gen), _ptr(h), _ptr(x), _ptr(y),
                           _ptr(gen_cache), _ptr(ws), ws.numel() * ws.element_size(),
                           _stream(stream))
    _check(rc, "dynconv_fwd")
    return (y, gen_cache) if want_cache else y


def dynconv_fwd_proj(h, Wp, *, k, W=None, A=None, U=None, w0=None, n_heads=0, x=None, y=None, gen_cache=None,
                     want_cache=False, workspace=None, stream=None, cu_seqlens=None):
    """Forward with the producing projection fused in: x = h Wp, then
    y = x + dynconv(x).  Returns (x, y) (and the generator cache when
    want_cache)."""
    B, T = h.shape[0], h.shape[1]
    if x is None:
        x = torch.empty(B, T, Wp.shape[1], dtype=h.dtype, device=h.device)
    prob = make_problem(x, h, k, cu_seqlens)
    gen = make_gen(W, A, U, w0, n_heads)
    if y is None:
        y = torch.empty_like(x)
    if gen_cache is None and want_cache and gen.kind != DYNCONV_STATIC:
        n = gen.n_heads * k if gen.kind == DYNCONV_HEADWISE else gen.rank
        gen_cache = torch.empty(B * T, n, dtype=torch.float32, device=h.device)
    nbytes = dynconv_workspace_bytes(prob, gen, 0 | (DYNCONV_WS_CACHED if gen_cache is not None else 0))
    ws = _workspace(nbytes, h.device, workspace)
    rc = lib().dynconv_fwd_proj(ctypes.byref(prob), ctypes.byref(gen), _ptr(h), _ptr(Wp), _ptr(x), _ptr(y),
                                _ptr(gen_cache), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "dynconv_fwd_proj")
    return (x, y, gen_cache) if want_cache else (x, y)


def dynconv_fwd_noalloc(h, x, *, k, W=None, A=None, U=None, w0=None, n_heads=0, y=None, gen_cache=None,
                        stream=None, cu_seqlens=None):
    """Forward whose workspace is the library's static scratch (no workspace
    argument).  y and gen_cache, when not given, are allocated here by torch,
    outside the library call; pass them for a call that allocates nothing."""
    prob = make_problem(x, h, k, cu_seqlens)
    gen = make_gen(W, A, U, w0, n_heads)
    if y is None:
        y = torch.empty_like(x)
    rc = lib().dynconv_fwd_noalloc(ctypes.byref(prob), ctypes.byref(gen), _ptr(h), _ptr(x), _ptr(y),
                                   _ptr(gen_cache), _stream(stream))
    _check(rc, "dynconv_fwd_noalloc")
    return y


def dynconv_bwd(h, x, dy, *, k, W=None, A=None, U=None, w0=None, n_heads=0, gen_cache=None,
                need_dh=True, need_dw0=True, out=None, workspace=None, stream=None, cu_seqlens=None):
    """Backward of sum(dy * y).  Returns dict(dx, dh, dw0, dW | dA, dU).
    cu_seqlens: packed documents, as given to the forward."""
    prob = make_problem(x, h, k, cu_seqlens)
    gen = make_gen(W, A, U, w0, n_heads)
    dev = x.device
    f32 = dict(dtype=torch.float32, device=dev)
    o = dict(out or {})
    o.setdefault("dx", torch.empty_like(x))
    if need_dh and h is not None:
        o.setdefault("dh", torch.empty_like(h))
    if need_dw0:
        o.setdefault("dw0", torch.empty(prob.D, k, **f32))
    if gen.kind == DYNCONV_STATIC:
        pass
    elif gen.kind == DYNCONV_HEADWISE:
        o.setdefault("dW", torch.empty(prob.d_model, gen.n_heads * k, **f32))
    else:
        o.setdefault("dA", torch.empty(prob.d_model, gen.rank, **f32))
        o.setdefault("dU", torch.empty(gen.rank, prob.D * k, **f32))
    gg = GenGrad(_ptr(o.get("dW")), _ptr(o.get("dA")), _ptr(o.get("dU")), _ptr(o.get("dw0")))
    nbytes = dynconv_workspace_bytes(prob, gen, 1 | (DYNCONV_WS_CACHED if gen_cache is not None else 0))
    ws = _workspace(nbytes, dev, workspace)
    rc = lib().dynconv_bwd(ctypes.byref(prob), ctypes.byref(gen), _ptr(h), _ptr(x), _ptr(dy),
                           _ptr(gen_cache), _ptr(o["dx"]), _ptr(o.get("dh")), ctypes.byref(gg),
                           _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "dynconv_bwd")
    return o


def dynconv_decode(h, x, state, *, k, W=None, A=None, U=None, w0=None, n_heads=0, y=None, stream=None):
    """One decoding step: h [B, d_model], x [B, D], state [B, k-1, D] (updated
    in place; None when k == 1).  Returns y [B, D]."""
    B, D = x.shape
    prob = Problem(B, 1, 0 if h is None else h.shape[-1], D, k, _dtype_code(x.dtype), None, 0)
    gen = make_gen(W, A, U, w0, n_heads)
    if y is None:
        y = torch.empty_like(x)
    rc = lib().dynconv_decode(ctypes.byref(prob), ctypes.byref(gen), _ptr(h), _ptr(x), _ptr(state), _ptr(y),
                              _stream(stream))
    _check(rc, "dynconv_decode")
    return y


class DynConvFn(torch.autograd.Function):
    """autograd wrapper: y = DynConvFn.apply(h, x, W, A, U, w0, k, n_heads[, cu_seqlens]).

    Pass W (head-wise, with n_heads) or A and U (low-rank), or none of them
    for the static filter (w0 alone; h may then be None); unused weights are
    None; cu_seqlens packs documents into one row.  The forward keeps the
    fp32 generator cache for the backward.  First derivatives only.
    """

    @staticmethod
    def forward(ctx, h, x, W, A, U, w0, k, n_heads, cu_seqlens=None):
        y, cache = dynconv_fwd(h, x, k=k, W=W, A=A, U=U, w0=w0, n_heads=n_heads, want_cache=True,
                               cu_seqlens=cu_seqlens)
        ctx.save_for_backward(h, x, W, A, U, w0, cache, cu_seqlens)
        ctx.k, ctx.n_heads = k, n_heads
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        h, x, W, A, U, w0, cache, cu_seqlens = ctx.saved_tensors
        g = dynconv_bwd(h, x, dy.contiguous(), k=ctx.k, W=W, A=A, U=U, w0=w0, n_heads=ctx.n_heads,
                        gen_cache=cache, need_dh=ctx.needs_input_grad[0],
                        need_dw0=w0 is not None, cu_seqlens=cu_seqlens)
        cast = lambda t, ref: None if t is None or ref is None else t.to(ref.dtype)
        return (g.get("dh"), g["dx"], cast(g.get("dW"), W), cast(g.get("dA"), A),
                cast(g.get("dU"), U), cast(g.get("dw0"), w0), None, None, None)


# --- the Q/K/V path behind the convolution ------------------------------------------------------
#
# These calls are made once a token and layer in serving, so what they cost on the host
# counts: the structs are packed directly (as View, Attn and Rotary lay them out) and the
# raw stream is asked for, 12 us a rotary call -> 8.

_VIEW, _ATTN, _ROTARY = struct.Struct("Pqqq").pack, struct.Struct("qqiiiifiPq").pack, struct.Struct("iiifP").pack


def _pack_view(t: torch.Tensor, what: str, shape, dtype, dev: int) -> bytes:
    """The View of a [B, T, heads, head_dim] (or [B, heads, head_dim]) tensor of the given shape and dtype on GPU dev."""
    if t.shape != shape:
        raise ValueError(f"{what}: expected the shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{what}: expected a {dtype} tensor on the GPU, got {t.dtype} on {t.device}")
    if t.get_device() != dev:
        _other_device(t, what, dev)
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1 and t.numel():
        raise ValueError(f"{what}: the last axis must be contiguous, got strides {s}")
    return _VIEW(t.data_ptr(), s[0], s[1], s[2]) if len(s) == 4 else _VIEW(t.data_ptr(), s[0], 0, s[1])


def _other_device(t, what: str, dev: int):
    raise ValueError(f"{what}: expected a tensor on cuda:{dev}, got one on {t.device}")


def _dims(t: torch.Tensor, what: str, n: int):
    if t.dim() != n:
        raise ValueError(f"{what}: expected {n} axes, got the shape {tuple(t.shape)}")
    return t.shape


def _int32(t, what: str, dev: int, shape=None) -> int:
    """Address of a contiguous int32 tensor on GPU dev, 0 for None."""
    if t is None:
        return 0
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or (shape is not None and t.shape != shape):
        raise TypeError(f"{what} must be a contiguous int32 tensor on the GPU"
                        + (f" of shape {tuple(shape)}" if shape is not None else ""))
    if t.get_device() != dev:
        _other_device(t, what, dev)
    return t.data_ptr()


def _scale(scale) -> float:
    """The factor on q.k as the struct has it, where 0 stands for the default."""
    if scale is None:
        return 0.0
    if 0.0 <= scale < 2.0 ** -120:
        raise ValueError(f"scale must be positive and no less than 2^-120, got {scale}")
    return scale


def _pack_attn(B, T, H, G, hd, dtype, dev, scale, cu_seqlens) -> bytes:
    if cu_seqlens is None:
        return _ATTN(B, T, H, G, hd, _dtype_code(dtype), _scale(scale), 0, 0, 0)
    if cu_seqlens.dim() != 1:
        raise TypeError("cu_seqlens must be a contiguous 1-d int32 tensor")
    return _ATTN(B, T, H, G, hd, _dtype_code(dtype), _scale(scale), 0, _int32(cu_seqlens, "cu_seqlens", dev),
                 cu_seqlens.shape[0] - 1)


def _pack_rotary(freqs: torch.Tensor, interleaved, inverse, factor, dev) -> bytes:
    if freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous() or not freqs.is_cuda:
        raise TypeError("freqs must be a contiguous 1-d float64 tensor on the GPU (radians per position, one per pair)")
    if freqs.get_device() != dev:
        _other_device(freqs, "freqs", dev)
    return _ROTARY(2 * freqs.shape[0], 1 if interleaved else 0, 1 if inverse else 0, factor, freqs.data_ptr())


def _launch(dev: int, where: str, call, *args) -> None:
    """call(*args, stream) on the current stream of GPU dev, which is made the current device for it: that is where
    a launch goes."""
    if dev == _C._cuda_getDevice():
        rc = call(*args, _C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            rc = call(*args, _C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, where)


def _on(stream, call, t, *args, **kw):
    """call(t, ...) with `stream` (a torch stream or a raw one of t's GPU) current, so that what it allocates belongs
    to that stream too and is not handed out again while the stream still uses it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=t.device)
    if stream.device != t.device:
        raise ValueError(f"stream: expected one of {t.device}, got one of {stream.device}")
    with torch.cuda.stream(stream):
        return call(t, *args, **kw)


def _lse(lse, shape, dev) -> int:
    if lse.dtype != torch.float32 or lse.shape != shape or not lse.is_contiguous() or not lse.is_cuda:
        raise TypeError(f"lse must be a contiguous float32 tensor {list(shape)} on the GPU")
    if lse.get_device() != dev:
        _other_device(lse, "lse", dev)
    return lse.data_ptr()


def _new(like: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(like, memory_format=torch.contiguous_format)


def _out(t, like: torch.Tensor, what: str, shape, dev: int):
    """An output and its View: the caller's, or a new contiguous one of like's shape."""
    if t is not None:
        return t, _pack_view(t, what, shape, like.dtype, dev)
    t = _new(like)
    row = shape[-2] * shape[-1]
    return t, _VIEW(t.data_ptr(), shape[1] * row if len(shape) == 4 else row, row, shape[-1])


def dynconv_rope_freqs(rot_dim: int, base: float = 10000.0, *, stretch: float = 1.0, trained_len: float = 0.0,
                       slow_turns: float = 1.0, fast_turns: float = 32.0, device="cuda") -> torch.Tensor:
    """The frequencies of a rotary plan, float64 [rot_dim/2] on ``device``.

    ``base ** (-2m / rot_dim)``; with ``stretch`` > 1 divided by it, for all
    pairs, or with ``trained_len`` > 0 by wavelength: pairs that make
    ``fast_turns`` or more turns over the trained length keep their frequency,
    those of ``slow_turns`` or fewer are divided, linear in between."""
    out = torch.empty(max(int(rot_dim), 0) // 2, dtype=torch.float64)
    _check(lib().dynconv_rope_freqs(int(rot_dim), base, stretch, trained_len, slow_turns, fast_turns,
                                    out.data_ptr() or None), "dynconv_rope_freqs")
    return out.to(device)


def dynconv_rope(x, freqs, *, positions=None, cu_seqlens=None, interleaved=False, factor=1.0, inverse=False, out=None,
                 stream=None):
    """Rotary positions: x [B, T, heads, head_dim] (any strides with a contiguous
    last axis) with its first 2 * len(freqs) elements turned, as a new tensor or
    into ``out`` (x itself: in place).  positions: int32 [B, T], or the token's
    index in its row or, with cu_seqlens, in its document.  inverse: the backward."""
    if stream is not None:
        return _on(stream, dynconv_rope, x, freqs, positions=positions, cu_seqlens=cu_seqlens, interleaved=interleaved,
                   factor=factor, inverse=inverse, out=out)
    B, T, H, hd = shape = _dims(x, "x", 4)
    dt, dev = x.dtype, x.get_device()
    vx = _pack_view(x, "x", shape, dt, dev)
    a = _pack_attn(B, T, H, 1, hd, dt, dev, None, cu_seqlens)
    r = _pack_rotary(freqs, interleaved, inverse, factor, dev)
    out, vy = _out(out, x, "out", shape, dev)
    _launch(dev, "dynconv_rope", lib().dynconv_rope, a, r, vx, _int32(positions, "positions", dev, (B, T)), vy)
    return out


def dynconv_attn_fwd(q, k, v, *, scale=None, cu_seqlens=None, o=None, lse=None, want_lse=False, stream=None):
    """Causal attention over whole sequences: q [B, T, n_heads, head_dim], k and
    v [B, T, n_kv_heads, head_dim] (any strides with a contiguous last axis).
    Returns o (and lse, fp32 [B, n_heads, T], when want_lse).  scale: default
    1 / sqrt(head_dim).  cu_seqlens: packed documents (B must be 1)."""
    if stream is not None:
        return _on(stream, dynconv_attn_fwd, q, k, v, scale=scale, cu_seqlens=cu_seqlens, o=o, lse=lse, want_lse=want_lse)
    B, T, H, hd = shape = _dims(q, "q", 4)
    G, dt, dev = _dims(k, "k", 4)[2], q.dtype, q.get_device()
    kv = (B, T, G, hd)
    vq, a = _pack_view(q, "q", shape, dt, dev), _pack_attn(B, T, H, G, hd, dt, dev, scale, cu_seqlens)
    o, vo = _out(o, q, "o", shape, dev)
    if lse is not None:
        pl = _lse(lse, (B, H, T), dev)
    elif want_lse:
        lse = q.new_empty((B, H, T), dtype=torch.float32)
        pl = lse.data_ptr()
    else:
        pl = None
    _launch(dev, "dynconv_attn_fwd", lib().dynconv_attn_fwd, a, vq, _pack_view(k, "k", kv, dt, dev),
            _pack_view(v, "v", kv, dt, dev), vo, pl)
    return (o, lse) if want_lse else o


def dynconv_attn_bwd(q, k, v, o, lse, d_o, *, scale=None, cu_seqlens=None, out=None, workspace=None, stream=None):
    """Backward of dynconv_attn_fwd from its inputs, o, lse and d_o.  Returns
    dict(dq, dk, dv); ``out`` may hold any of them (views of one gradient row,
    for instance)."""
    if stream is not None:
        return _on(stream, dynconv_attn_bwd, q, k, v, o, lse, d_o, scale=scale, cu_seqlens=cu_seqlens, out=out,
                   workspace=workspace)
    B, T, H, hd = shape = _dims(q, "q", 4)
    G, dt, dev = _dims(k, "k", 4)[2], q.dtype, q.get_device()
    kv = (B, T, G, hd)
    ins = (_pack_view(q, "q", shape, dt, dev), _pack_view(k, "k", kv, dt, dev), _pack_view(v, "v", kv, dt, dev),
           _pack_view(o, "o", shape, dt, dev), _lse(lse, (B, H, T), dev), _pack_view(d_o, "d_o", shape, dt, dev))
    a = _pack_attn(B, T, H, G, hd, dt, dev, scale, cu_seqlens)
    out = out or {}
    dq, vdq = _out(out.get("dq"), q, "dq", shape, dev)
    dk, vdk = _out(out.get("dk"), k, "dk", kv, dev)
    dv, vdv = _out(out.get("dv"), v, "dv", kv, dev)
    L = lib()
    ws = _workspace(L.dynconv_attn_bwd_workspace_bytes(a), q.device, workspace)
    _launch(dev, "dynconv_attn_bwd", L.dynconv_attn_bwd, a, *ins, vdq, vdk, vdv, ws.data_ptr(), ws.nbytes)
    return {"dq": dq, "dk": dk, "dv": dv}


def dynconv_attn_decode(q, k, v, k_cache, v_cache, lengths, *, scale=None, freqs=None, interleaved=False, factor=1.0,
                        o=None, workspace=None, stream=None):
    """One token per sequence: q [B, n_heads, head_dim], k and v [B, n_kv_heads,
    head_dim], caches [B, capacity, n_kv_heads, head_dim], lengths int32 [B] (the
    tokens in each cache; the new one's position).  q and k are turned by the
    rotary plan (freqs None: not), k and v stored in the caches' rows lengths[b],
    and o [B, n_heads, head_dim] returned.  A slot with lengths[b] < 0 (or a full
    one) is idle: its o is zero."""
    if stream is not None:
        return _on(stream, dynconv_attn_decode, q, k, v, k_cache, v_cache, lengths, scale=scale, freqs=freqs,
                   interleaved=interleaved, factor=factor, o=o, workspace=workspace)
    B, H, hd = shape = _dims(q, "q", 3)
    G, cap = _dims(k, "k", 3)[1], _dims(k_cache, "k_cache", 4)[1]
    dt, dev = q.dtype, q.get_device()
    kv, rows = (B, G, hd), (B, cap, G, hd)
    vq = _pack_view(q, "q", shape, dt, dev)
    a = _pack_attn(B, 1, H, G, hd, dt, dev, scale, None)
    o, vo = _out(o, q, "o", shape, dev)
    L = lib()
    nbytes = L.dynconv_attn_decode_workspace_bytes(a, cap)
    ws = _workspace(nbytes, q.device, workspace) if nbytes or workspace is not None else None
    _launch(dev, "dynconv_attn_decode", L.dynconv_attn_decode, a,
            None if freqs is None else _pack_rotary(freqs, interleaved, False, factor, dev), vq,
            _pack_view(k, "k", kv, dt, dev), _pack_view(v, "v", kv, dt, dev),
            _pack_view(k_cache, "k_cache", rows, dt, dev), _pack_view(v_cache, "v_cache", rows, dt, dev), cap,
            _int32(lengths, "lengths", dev, (B,)), vo, _ptr(ws), 0 if ws is None else ws.nbytes)
    return o


class QKVAttnFn(torch.autograd.Function):
    """autograd wrapper of what follows the convolution on the Q/K/V path:
    o = QKVAttnFn.apply(row, n_heads, n_kv_heads, freqs[, interleaved, factor, scale, cu_seqlens]).

    row [B, T, (n_heads + 2 n_kv_heads) head_dim] (query, key and value heads
    side by side, as DynConvFn returns it) -> rotary positions on its query and
    key heads (freqs None: none) -> causal attention -> o [B, T, n_heads, head_dim].
    The backward writes one gradient row, turned back in place.  First derivatives only.
    """

    @staticmethod
    def forward(ctx, row, n_heads, n_kv_heads, freqs, interleaved=False, factor=1.0, scale=None, cu_seqlens=None):
        H, G = n_heads, n_kv_heads
        heads = row.view(row.shape[0], row.shape[1], H + 2 * G, row.shape[2] // (H + 2 * G))
        qk, v = heads[:, :, :H + G], heads[:, :, H + G:]
        if freqs is not None:
            qk = dynconv_rope(qk, freqs, cu_seqlens=cu_seqlens, interleaved=interleaved, factor=factor)
        o, lse = dynconv_attn_fwd(qk[:, :, :H], qk[:, :, H:], v, scale=scale, cu_seqlens=cu_seqlens, want_lse=True)
        ctx.save_for_backward(qk, v, o, lse, freqs, cu_seqlens)
        ctx.args = H, interleaved, factor, scale
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o):
        qk, v, o, lse, freqs, cu_seqlens = ctx.saved_tensors
        H, interleaved, factor, scale = ctx.args
        both = qk.shape[2]
        B, T, heads, hd = qk.shape[0], qk.shape[1], both + v.shape[2], qk.shape[3]
        row = torch.empty((B, T, heads, hd), dtype=qk.dtype, device=qk.device)
        dynconv_attn_bwd(qk[:, :, :H], qk[:, :, H:], v, o, lse, d_o.contiguous(), scale=scale, cu_seqlens=cu_seqlens,
                         out={"dq": row[:, :, :H], "dk": row[:, :, H:both], "dv": row[:, :, both:]})
        if freqs is not None:
            dynconv_rope(row[:, :, :both], freqs, cu_seqlens=cu_seqlens, interleaved=interleaved, factor=factor,
                         inverse=True, out=row[:, :, :both])
        return (row.view(B, T, heads * hd),) + (None,) * 7
