"""ctypes binding of libla2 (include/la2.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libla2.so.  PyTorch supplies device memory (outputs, scratch
workspace) and the current CUDA stream.  There is no fallback: if the
library is missing or a call fails, an exception is raised.

A call launches on the current stream, or on the one given as `stream`.  The
caller orders a stream that it names behind what made the inputs, and what uses
the results behind it; inputs, results and scratch may be dropped at any time.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import json
import math
import os
import struct
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libla2.so")

LA2_OK, LA2_ERR_INVALID, LA2_ERR_UNSUPPORTED, LA2_ERR_CUDA, LA2_ERR_TIMEOUT = range(5)
LA2_F32, LA2_BF16 = 0, 1
LA2_OP_FORWARD, LA2_OP_BACKWARD, LA2_OP_SHARD_STATE, LA2_OP_DLAMBDA = 0, 1, 2, 3
LA2_OP_GATED_NORM_BACKWARD, LA2_OP_RESIDUAL_NORM_BACKWARD = 4, 5
LA2_OPT_SPLIT, LA2_OPT_PATH, LA2_OPT_INJECT_TIMEOUT, LA2_OPT_VARIANT, LA2_OPT_TRACE = 0, 1, 2, 3, 4
LA2_OPT_VARLEN_ORDER, LA2_OPT_DECODE_BLOCK_TOKENS, LA2_OPT_BWD_FORM = 5, 6, 7

_lock = threading.Lock()
_lib = None


class LA2Error(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)}")


def library():
    """Load libla2.so (built in-tree by ``build.py``); raise if it is absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libla2.so is not built ({LIB_PATH}); run "
                "`python -c 'import __graft_entry__ as g; g.build()'` or "
                "`python causal_linear_attention_fwd_b200/build.py`")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        lib.la2_workspace_size.argtypes = [I, I, I, I64, I, I, I]
        lib.la2_workspace_size.restype = SZ
        lib.la2_forward.argtypes = [P, P, P, P, P, P, P, I, I, I64, I, I, I, P, SZ, P]
        lib.la2_forward.restype = I
        lib.la2_forward_noalloc.argtypes = [P, P, P, P, P, P, P, I, I, I64, I, I, I, P]
        lib.la2_forward_noalloc.restype = I
        lib.la2_backward.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I64, I, I, I,
                                     P, SZ, P]
        lib.la2_backward.restype = I
        lib.la2_backward_ex.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I64, I, I, I,
                                        P, SZ, ctypes.c_uint, P]
        lib.la2_backward_ex.restype = I
        lib.la2_forward_varlen.argtypes = [P, P, P, P, P, P, P, P, I, I, I64, I, I, I, P]
        lib.la2_forward_varlen.restype = I
        lib.la2_backward_varlen.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I64, I, I,
                                            I, P]
        lib.la2_backward_varlen.restype = I
        lib.la2_forward_pool.argtypes = [P, P, P, P, P, P, I, P, ctypes.c_uint, I, I, I64, I,
                                         I, I, P, SZ, P]
        lib.la2_forward_pool.restype = I
        lib.la2_decode_tokens.argtypes = [P, P, P, P, P, P, I, P, I, I, I, I, I, I, P]
        lib.la2_decode_tokens.restype = I
        lib.la2_shard_state.argtypes = [P, P, P, P, I, I, I64, I, I, I, I, P, SZ, P]
        lib.la2_shard_state.restype = I
        lib.la2_state_prefix.argtypes = [P, P, P, P, I, I, I, I64, I, I, I, P]
        lib.la2_state_prefix.restype = I
        lib.la2_backward_shard.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I64, I, I, I,
                                           P, SZ, ctypes.c_uint, P]
        lib.la2_backward_shard.restype = I
        lib.la2_backward_dlambda.argtypes = [P, P, P, P, P, P, P, I, I, I64, I, I, I, P]
        lib.la2_backward_dlambda.restype = I
        lib.la2_backward_dlambda_ex.argtypes = [P, P, P, P, P, P, P, I, I, I64, I, I, I, P, SZ, P]
        lib.la2_backward_dlambda_ex.restype = I
        lib.la2_decode_step.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P]
        lib.la2_decode_step.restype = I
        lib.la2_feature_map.argtypes = [P, P, P, P, I64, I, P]
        lib.la2_feature_map.restype = I
        lib.la2_feature_map_backward.argtypes = [P, P, P, P, P, P, I64, I, P]
        lib.la2_feature_map_backward.restype = I
        F, U = ctypes.c_float, ctypes.c_uint
        lib.la2_rotary.argtypes = [P, P, P, P, P, I, P, P, P, F, U, I, I, I, I64, I, I, I, I, P]
        lib.la2_rotary.restype = I
        lib.la2_rotary_backward.argtypes = [P, P, P, P, P, I, P, P, P, F, U, I, I, I, I64, I, I,
                                            I, I, P]
        lib.la2_rotary_backward.restype = I
        lib.la2_gated_norm.argtypes = [P, P, I64, I64, P, P, F, U, I, I, I64, I, I, P]
        lib.la2_gated_norm.restype = I
        lib.la2_gated_norm_backward.argtypes = [P, P, P, I64, I64, P, P, P, I64, I64, P, F, U, I, I,
                                                I64, I, I, P, SZ, P]
        lib.la2_gated_norm_backward.restype = I
        lib.la2_residual_norm.argtypes = [P, I, P, P, P, P, P, F, F, F, U, I64, I, I, P]
        lib.la2_residual_norm.restype = I
        lib.la2_residual_norm_backward.argtypes = [P, P, P, I, P, P, P, P, P, P, P, F, F, F, U, I64,
                                                   I, I, P, SZ, P]
        lib.la2_residual_norm_backward.restype = I
        lib.la2_pool_copy.argtypes = [P, I, P, I, P, P, I, I, I, I, I, P]
        lib.la2_pool_copy.restype = I
        lib.la2_last_device_error.argtypes = [P]
        lib.la2_last_device_error.restype = I
        lib.la2_status_string.argtypes = [I]
        lib.la2_status_string.restype = ctypes.c_char_p
        lib.la2_set_option.argtypes = [I, I]
        lib.la2_set_option.restype = I
        lib.la2_profile_enable.argtypes = [I]
        lib.la2_profile_enable.restype = None
        lib.la2_profile_report.argtypes = [ctypes.c_char_p, SZ]
        lib.la2_profile_report.restype = SZ
        lib.la2_trace_read.argtypes = [P, SZ]
        lib.la2_trace_read.restype = SZ
        lib.la2_version.argtypes = []
        lib.la2_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def status_string(code: int) -> str:
    try:
        return library().la2_status_string(int(code)).decode()
    except Exception:  # library missing: still give a name
        return {0: "LA2_OK", 1: "LA2_ERR_INVALID", 2: "LA2_ERR_UNSUPPORTED",
                3: "LA2_ERR_CUDA", 4: "LA2_ERR_TIMEOUT"}.get(int(code), str(code))


def _check(code: int, what: str):
    if code != LA2_OK:
        raise LA2Error(code, what)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LA2_F32
    if t.dtype == torch.bfloat16:
        return LA2_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _devices(*named):
    """Check (name, tensor) pairs -- None tensors skipped -- as _dev does and
    that all of them live on one device; return that device.  The library
    launches on the CURRENT device, so a call with tensors elsewhere would
    run its kernels and tensor maps over another GPU's memory."""
    dev = None
    for name, t in named:
        if t is None:
            continue
        _dev(t, name)
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, other arguments on {dev}")
    if dev is None:
        raise ValueError("no tensor arguments")
    return dev


def _stream(stream, device=None):
    if stream is None:
        s = torch.cuda.current_stream(device)
    else:
        s = stream
        if device is not None and s.device != device:
            raise ValueError(f"stream is on {s.device}, the tensors on {device}")
    return ctypes.c_void_p(s.cuda_stream)


_no_guard = contextlib.nullcontext()  # a device that is current is not made current again


@contextlib.contextmanager
def _named_stream(dev, stream):
    caller = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        yield caller


def _guard(dev, stream=None):
    """What a call runs under: its device current and, where it names a stream
    that is not, that stream as well: its scratch and results then come from
    memory that this stream's earlier work is done with, and scratch goes back
    behind the call's own work.  Gives the caller's stream then, else None."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
        if stream.cuda_stream != torch._C._cuda_getCurrentRawStream(dev.index):
            return _named_stream(dev, stream)
    return _no_guard if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _used_on(streams, *tensors):
    """Marks tensors (or None) as used on these streams: memory that is given
    back before such a use has run is not handed out until it has."""
    for t in tensors:
        if t is not None:
            for s in streams:
                t.record_stream(s)


def _out(t, name, shape, dtype, device):
    """A caller-provided output buffer: contiguous, on `device`, of this
    shape and dtype."""
    _dev(t, name)
    if t.device != device or tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)} on {device}")
    return t


def set_option(option: int, value: int) -> int:
    return int(library().la2_set_option(int(option), int(value)))


def version() -> str:
    return library().la2_version().decode()


def workspace_size(op: int, B: int, H: int, L: int, d: int, e: int, dtype) -> int:
    dt = LA2_F32 if dtype == torch.float32 else LA2_BF16
    return int(library().la2_workspace_size(op, B, H, L, d, e, dt))


def _workspace(nbytes: int, device):
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def forward(q, k, v, lam, kv0=None, *, want_state: bool = False, out=None,
            workspace=None, stream=None):
    """o = (Q K^T (.) M) V (+ the kv0 term); optionally the final state."""
    lib = library()
    dev = _devices(("q", q), ("k", k), ("v", v), ("lam", lam), ("kv0", kv0),
                   ("workspace", workspace))
    B, H, L, d = q.shape
    e = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (B, H, L):
        raise ValueError("shape mismatch among q, k, v")
    if lam.dtype != torch.float32 or lam.numel() != H:
        raise ValueError("lam must be float32 [H]")
    if kv0 is not None and (kv0.dtype != torch.float32 or kv0.shape != (B, H, d, e)):
        raise ValueError("kv0 must be float32 [B,H,d,e]")
    with _guard(dev, stream) as caller:
        o = (_out(out, "out", (B, H, L, e), q.dtype, dev) if out is not None
             else torch.empty((B, H, L, e), dtype=q.dtype, device=dev))
        st = torch.empty((B, H, d, e), dtype=torch.float32, device=dev) if want_state else None
        ws = workspace
        if ws is None:
            ws = _workspace(workspace_size(LA2_OP_FORWARD, B, H, L, d, e, q.dtype), dev)
        code = lib.la2_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(kv0), _ptr(o),
                               _ptr(st), B, H, L, d, e, _dt(q), _ptr(ws),
                               0 if ws is None else ws.numel() * ws.element_size(),
                               _stream(stream, dev))
    _check(code, "la2_forward")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, kv0, ws, o, st)
    return (o, st) if want_state else o


def forward_noalloc(q, k, v, lam, kv0=None, *, want_state: bool = False, out=None,
                    state_out=None, stream=None):
    """forward() for callers that cannot allocate device scratch: the library
    keeps the chunk-boundary states in its own fixed 32 MiB device array
    (see la2_forward_noalloc in include/la2.h).  Outputs are allocated here
    unless the caller passes them: `out` (o) and, with want_state,
    `state_out` (the final state)."""
    lib = library()
    dev = _devices(("q", q), ("k", k), ("v", v), ("lam", lam), ("kv0", kv0))
    B, H, L, d = q.shape
    e = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (B, H, L):
        raise ValueError("shape mismatch among q, k, v")
    if lam.dtype != torch.float32 or lam.numel() != H:
        raise ValueError("lam must be float32 [H]")
    if kv0 is not None and (kv0.dtype != torch.float32 or kv0.shape != (B, H, d, e)):
        raise ValueError("kv0 must be float32 [B,H,d,e]")
    if state_out is not None and not want_state:
        raise ValueError("state_out is given but want_state is False")
    with _guard(dev, stream) as caller:
        o = (_out(out, "out", (B, H, L, e), q.dtype, dev) if out is not None
             else torch.empty((B, H, L, e), dtype=q.dtype, device=dev))
        st = None
        if want_state:
            st = (_out(state_out, "state_out", (B, H, d, e), torch.float32, dev)
                  if state_out is not None
                  else torch.empty((B, H, d, e), dtype=torch.float32, device=dev))
        code = lib.la2_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(kv0), _ptr(o),
                                       _ptr(st), B, H, L, d, e, _dt(q), _stream(stream, dev))
    _check(code, "la2_forward_noalloc")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, kv0, o, st)
    return (o, st) if want_state else o


def backward(q, k, v, lam, dO, kv0=None, *, want_dkv0: bool = False, outs=None,
             workspace=None, reuse_forward_states: bool = False, stream=None):
    """Gradients (dq, dk, dv[, dkv0]) of sum(o * dO).

    reuse_forward_states: `workspace` (sized for the backward) was passed to
    forward() with the same inputs and still holds the chunk states it wrote,
    so the backward does not recompute them."""
    if reuse_forward_states and workspace is None:
        raise ValueError("reuse_forward_states needs the forward's workspace")
    lib = library()
    dev = _devices(("q", q), ("k", k), ("v", v), ("lam", lam), ("dO", dO), ("kv0", kv0),
                   ("workspace", workspace))
    B, H, L, d = q.shape
    e = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (B, H, L) or dO.shape != v.shape:
        raise ValueError("shape mismatch among q, k, v, dO")
    if lam.dtype != torch.float32 or lam.numel() != H:
        raise ValueError("lam must be float32 [H]")
    if kv0 is not None and (kv0.dtype != torch.float32 or kv0.shape != (B, H, d, e)):
        raise ValueError("kv0 must be float32 [B,H,d,e]")
    with _guard(dev, stream) as caller:
        if outs is not None:
            dq, dk, dv = outs
            _out(dq, "dq", q.shape, q.dtype, dev)
            _out(dk, "dk", k.shape, q.dtype, dev)
            _out(dv, "dv", v.shape, q.dtype, dev)
        else:
            dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dkv0 = torch.empty((B, H, d, e), dtype=torch.float32, device=dev) if want_dkv0 else None
        ws = workspace
        if ws is None:
            ws = _workspace(workspace_size(LA2_OP_BACKWARD, B, H, L, d, e, q.dtype), dev)
        code = lib.la2_backward_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(kv0), _ptr(dO),
                                   _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dkv0), B, H, L, d, e,
                                   _dt(q), _ptr(ws),
                                   0 if ws is None else ws.numel() * ws.element_size(),
                                   1 if reuse_forward_states else 0, _stream(stream, dev))
    _check(code, "la2_backward")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, dO, kv0, ws, dq, dk, dv, dkv0)
    return (dq, dk, dv, dkv0) if want_dkv0 else (dq, dk, dv)


def _varlen_args(q, k, v, lam, cu_seqlens, kv0, *extra):
    dev = _devices(("q", q), ("k", k), ("v", v), ("lam", lam), ("cu_seqlens", cu_seqlens),
                   ("kv0", kv0), *extra)
    H, T, d = q.shape
    e = v.shape[-1]
    if k.shape != q.shape or v.shape[:2] != (H, T):
        raise ValueError("q, k must be [H, T, d] and v [H, T, e]")
    if lam.dtype != torch.float32 or lam.numel() != H:
        raise ValueError("lam must be float32 [H]")
    if cu_seqlens.dtype != torch.int64 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be int64 [N+1]")
    N = cu_seqlens.numel() - 1
    if kv0 is not None and (kv0.dtype != torch.float32 or kv0.shape != (N, H, d, e)):
        raise ValueError("kv0 must be float32 [N,H,d,e]")
    return dev, N, H, T, d, e


def forward_varlen(q, k, v, lam, cu_seqlens, kv0=None, *, want_state: bool = False,
                   out=None, stream=None):
    """Packed variable-length forward: q, k [H,T,d], v [H,T,e], sequence n on
    rows cu_seqlens[n]..cu_seqlens[n+1] of every head; per-sequence states
    [N,H,d,e].  Returns o [H,T,e] (and the final states)."""
    lib = library()
    dev, N, H, T, d, e = _varlen_args(q, k, v, lam, cu_seqlens, kv0)
    with _guard(dev, stream) as caller:
        o = (_out(out, "out", (H, T, e), q.dtype, dev) if out is not None
             else torch.empty((H, T, e), dtype=q.dtype, device=dev))
        st = torch.empty((N, H, d, e), dtype=torch.float32, device=dev) if want_state else None
        code = lib.la2_forward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(cu_seqlens),
                                      _ptr(kv0), _ptr(o), _ptr(st), N, H, T, d, e, _dt(q),
                                      _stream(stream, dev))
    _check(code, "la2_forward_varlen")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, cu_seqlens, kv0, o, st)
    return (o, st) if want_state else o


def backward_varlen(q, k, v, lam, cu_seqlens, dO, kv0=None, *, want_dkv0: bool = False,
                    outs=None, stream=None):
    """Gradients (dq, dk, dv[, dkv0]) of sum(o * dO) for forward_varlen."""
    lib = library()
    dev, N, H, T, d, e = _varlen_args(q, k, v, lam, cu_seqlens, kv0, ("dO", dO))
    if dO.shape != v.shape:
        raise ValueError("dO must match v")
    with _guard(dev, stream) as caller:
        if outs is not None:
            dq, dk, dv = outs
            _out(dq, "dq", q.shape, q.dtype, dev)
            _out(dk, "dk", k.shape, q.dtype, dev)
            _out(dv, "dv", v.shape, q.dtype, dev)
        else:
            dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dkv0 = torch.empty((N, H, d, e), dtype=torch.float32, device=dev) if want_dkv0 else None
        code = lib.la2_backward_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(cu_seqlens),
                                       _ptr(kv0), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv),
                                       _ptr(dkv0), N, H, T, d, e, _dt(q), _stream(stream, dev))
    _check(code, "la2_backward_varlen")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, cu_seqlens, dO, kv0, dq, dk, dv, dkv0)
    return (dq, dk, dv, dkv0) if want_dkv0 else (dq, dk, dv)


LA2_POOL_CONTINUE = 1


def _slots(slots, B):
    if slots is None:
        return None
    if slots.dtype != torch.int32 or slots.shape != (B,):
        raise ValueError("slots must be int32 [B]")
    return slots


def forward_pool(q, k, v, lam, pool, slots, *, continue_state: bool = False, out=None,
                 workspace=None, stream=None):
    """Prefill into a state pool [P,H,d,e]: request b starts from zero (or,
    with continue_state, from pool[slots[b]]) and leaves its final state in
    pool[slots[b]].  Returns o [B,H,L,e]."""
    lib = library()
    if slots is None:
        raise ValueError("forward_pool needs a slot table")
    dev = _devices(("q", q), ("k", k), ("v", v), ("lam", lam), ("pool", pool),
                   ("slots", slots), ("workspace", workspace))
    B, H, L, d = q.shape
    e = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (B, H, L):
        raise ValueError("shape mismatch among q, k, v")
    if pool.dtype != torch.float32 or pool.dim() != 4 or pool.shape[1:] != (H, d, e):
        raise ValueError("pool must be float32 [P,H,d,e]")
    slots = _slots(slots, B)
    with _guard(dev, stream) as caller:
        o = (_out(out, "out", (B, H, L, e), q.dtype, dev) if out is not None
             else torch.empty((B, H, L, e), dtype=q.dtype, device=dev))
        ws = workspace
        if ws is None:
            ws = _workspace(workspace_size(LA2_OP_FORWARD, B, H, L, d, e, q.dtype), dev)
        code = lib.la2_forward_pool(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(pool),
                                    _ptr(slots), pool.shape[0], _ptr(o),
                                    LA2_POOL_CONTINUE if continue_state else 0, B, H, L, d, e,
                                    _dt(q), _ptr(ws),
                                    0 if ws is None else ws.numel() * ws.element_size(),
                                    _stream(stream, dev))
    _check(code, "la2_forward_pool")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, pool, slots, ws, o)
    return o


def decode_tokens(q, k, v, lam, pool, slots=None, *, out=None, stream=None):
    """T tokens per request at once: q, k [B,H,T,d], v [B,H,T,e]; the state
    of request b is pool[slots[b]] (pool[b] without a slot table), updated
    in place; returns o [B,H,T,e]."""
    lib = library()
    dev = _devices(("q", q), ("k", k), ("v", v), ("lam", lam), ("pool", pool),
                   ("slots", slots))
    B, H, T, d = q.shape
    e = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (B, H, T):
        raise ValueError("shape mismatch among q, k, v")
    if pool.dtype != torch.float32 or pool.dim() != 4 or pool.shape[1:] != (H, d, e):
        raise ValueError("pool must be float32 [P,H,d,e]")
    slots = _slots(slots, B)
    with _guard(dev, stream) as caller:
        o = (_out(out, "out", (B, H, T, e), q.dtype, dev) if out is not None
             else torch.empty((B, H, T, e), dtype=q.dtype, device=dev))
        code = lib.la2_decode_tokens(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(pool),
                                     _ptr(slots), pool.shape[0], _ptr(o), B, H, T, d, e, _dt(q),
                                     _stream(stream, dev))
    _check(code, "la2_decode_tokens")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, pool, slots, o)
    return o


def shard_state(a, b, lam, *, reverse: bool = False, workspace=None, stream=None):
    """One shard's d x e summary: forward (a = k, b = v) sum_t
    lam^(L-1-t) k_t^T v_t, reverse (a = q, b = dO) sum_t lam^t q_t^T dO_t;
    fp32 [B,H,d,e]."""
    lib = library()
    dev = _devices(("a", a), ("b", b), ("lam", lam), ("workspace", workspace))
    B, H, L, d = a.shape
    e = b.shape[-1]
    if b.shape[:3] != (B, H, L):
        raise ValueError("shape mismatch between a and b")
    with _guard(dev, stream) as caller:
        out = torch.empty((B, H, d, e), dtype=torch.float32, device=dev)
        ws = workspace
        if ws is None:
            ws = _workspace(workspace_size(LA2_OP_SHARD_STATE, B, H, L, d, e, a.dtype), dev)
        code = lib.la2_shard_state(_ptr(a), _ptr(b), _ptr(lam), _ptr(out), B, H, L, d, e,
                                   _dt(a), 1 if reverse else 0, _ptr(ws),
                                   0 if ws is None else ws.numel() * ws.element_size(),
                                   _stream(stream, dev))
    _check(code, "la2_shard_state")
    if caller is not None:
        _used_on((caller, stream), a, b, lam, ws, out)
    return out


def state_prefix(delta, lam, L_shard: int, kv0=None, *, reverse: bool = False, stream=None):
    """Every shard's boundary state from the R shards' deltas [R,B,H,d,e]:
    forward, the state entering shard r (from kv0); reverse, the reverse
    state flowing into shard r from the rows after it."""
    lib = library()
    dev = _devices(("delta", delta), ("lam", lam), ("kv0", kv0))
    if delta.dtype != torch.float32 or delta.dim() != 5:
        raise ValueError("delta must be float32 [R,B,H,d,e]")
    R, B, H, d, e = delta.shape
    if kv0 is not None and (kv0.dtype != torch.float32 or kv0.shape != (B, H, d, e)):
        raise ValueError("kv0 must be float32 [B,H,d,e]")
    with _guard(dev, stream) as caller:
        out = torch.empty_like(delta)
        code = lib.la2_state_prefix(_ptr(delta), _ptr(kv0), _ptr(lam), _ptr(out), R, B, H,
                                    int(L_shard), d, e, 1 if reverse else 0,
                                    _stream(stream, dev))
    _check(code, "la2_state_prefix")
    if caller is not None:
        _used_on((caller, stream), delta, lam, kv0, out)
    return out


def backward_shard(q, k, v, lam, dO, kv0=None, dstate_end=None, *, want_dkv0: bool = False,
                   outs=None, workspace=None, stream=None):
    """backward() of one shard of a longer sequence: kv0 its entry state,
    dstate_end the reverse state flowing in from the rows after it."""
    lib = library()
    dev = _devices(("q", q), ("k", k), ("v", v), ("lam", lam), ("dO", dO), ("kv0", kv0),
                   ("dstate_end", dstate_end), ("workspace", workspace))
    B, H, L, d = q.shape
    e = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (B, H, L) or dO.shape != v.shape:
        raise ValueError("shape mismatch among q, k, v, dO")
    for name, t in (("kv0", kv0), ("dstate_end", dstate_end)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (B, H, d, e)):
            raise ValueError(f"{name} must be float32 [B,H,d,e]")
    with _guard(dev, stream) as caller:
        if outs is not None:
            dq, dk, dv = outs
            _out(dq, "dq", q.shape, q.dtype, dev)
            _out(dk, "dk", k.shape, q.dtype, dev)
            _out(dv, "dv", v.shape, q.dtype, dev)
        else:
            dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dkv0 = torch.empty((B, H, d, e), dtype=torch.float32, device=dev) if want_dkv0 else None
        ws = workspace
        if ws is None:
            ws = _workspace(workspace_size(LA2_OP_BACKWARD, B, H, L, d, e, q.dtype), dev)
        code = lib.la2_backward_shard(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(kv0), _ptr(dO),
                                      _ptr(dstate_end), _ptr(dq), _ptr(dk), _ptr(dv),
                                      _ptr(dkv0), B, H, L, d, e, _dt(q), _ptr(ws),
                                      0 if ws is None else ws.numel() * ws.element_size(), 0,
                                      _stream(stream, dev))
    _check(code, "la2_backward_shard")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, dO, kv0, dstate_end, ws, dq, dk, dv, dkv0)
    return (dq, dk, dv, dkv0) if want_dkv0 else (dq, dk, dv)


def dlambda(q, k, v, lam, dO, kv0=None, *, workspace=None, chunked: bool = True, stream=None):
    """Gradient of sum(o * dO) with respect to lam [H] (float32 [H], summed
    over the batch).  chunked: split the sequences over several CTAs
    (la2_backward_dlambda_ex with `workspace`, allocated here when None);
    False: one CTA per (b,h), no workspace (la2_backward_dlambda)."""
    lib = library()
    dev = _devices(("q", q), ("k", k), ("v", v), ("lam", lam), ("dO", dO), ("kv0", kv0),
                   ("workspace", workspace))
    B, H, L, d = q.shape
    e = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != (B, H, L) or dO.shape != v.shape:
        raise ValueError("shape mismatch among q, k, v, dO")
    if lam.dtype != torch.float32 or lam.numel() != H:
        raise ValueError("lam must be float32 [H]")
    if kv0 is not None and (kv0.dtype != torch.float32 or kv0.shape != (B, H, d, e)):
        raise ValueError("kv0 must be float32 [B,H,d,e]")
    with _guard(dev, stream) as caller:
        out = torch.empty(H, dtype=torch.float32, device=dev)
        if not chunked:
            code = lib.la2_backward_dlambda(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(kv0),
                                            _ptr(dO), _ptr(out), B, H, L, d, e, _dt(q),
                                            _stream(stream, dev))
        else:
            if workspace is None:
                workspace = _workspace(workspace_size(LA2_OP_DLAMBDA, B, H, L, d, e, q.dtype), dev)
            code = lib.la2_backward_dlambda_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(kv0),
                                               _ptr(dO), _ptr(out), B, H, L, d, e, _dt(q),
                                               _ptr(workspace), _nbytes(workspace),
                                               _stream(stream, dev))
    _check(code, "la2_backward_dlambda_ex" if chunked else "la2_backward_dlambda")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, dO, kv0, workspace, out)
    return out


def _fmap_args(q, k, extra):
    dev = _devices(("q", q), ("k", k), *extra)
    if k is not None and (k.shape != q.shape or k.dtype != q.dtype):
        raise ValueError("q and k must have the same shape and dtype")
    for name, t in extra:
        if t is not None and (t.shape != q.shape or t.dtype != q.dtype):
            raise ValueError(f"{name} must match q's shape and dtype")
    return dev


def feature_map(q, k=None, *, out=None, stream=None):
    """phi(x) = elu(x) + 1 applied to q (and k): returns phi_q (and phi_k).
    out: (phi_q, phi_k) buffers, which may be q and k themselves (in place)."""
    lib = library()
    dev = _fmap_args(q, k, ())
    with _guard(dev, stream) as caller:
        phi_q, phi_k = out if out is not None else (
            torch.empty_like(q), None if k is None else torch.empty_like(k))
        _fmap_args(q, k, (("phi_q", phi_q), ("phi_k", phi_k)))
        code = lib.la2_feature_map(_ptr(q), _ptr(k), _ptr(phi_q), _ptr(phi_k), q.numel(),
                                   _dt(q), _stream(stream, dev))
    _check(code, "la2_feature_map")
    if caller is not None:
        _used_on((caller, stream), q, k, phi_q, phi_k)
    return phi_q if k is None else (phi_q, phi_k)


def feature_map_backward(q, k, dphi_q, dphi_k=None, *, out=None, stream=None):
    """Chain rule through the feature map: dq = dphi_q * phi'(q) (and dk
    likewise), q, k the unmapped inputs, dphi_* the attention's gradients
    with respect to phi(q), phi(k).  out may be (dphi_q, dphi_k) (in place).
    k and dphi_k are both None to map q alone."""
    lib = library()
    if (k is None) != (dphi_k is None):
        raise ValueError("k and dphi_k are both given or both None")
    dev = _fmap_args(q, k, (("dphi_q", dphi_q), ("dphi_k", dphi_k)))
    with _guard(dev, stream) as caller:
        dq, dk = out if out is not None else (
            torch.empty_like(q), None if k is None else torch.empty_like(k))
        _fmap_args(q, k, (("dphi_q", dphi_q), ("dphi_k", dphi_k), ("dq", dq), ("dk", dk)))
        code = lib.la2_feature_map_backward(_ptr(q), _ptr(k), _ptr(dphi_q), _ptr(dphi_k),
                                            _ptr(dq), _ptr(dk), q.numel(), _dt(q),
                                            _stream(stream, dev))
    _check(code, "la2_feature_map_backward")
    if caller is not None:
        _used_on((caller, stream), q, k, dphi_q, dphi_k, dq, dk)
    return dq if k is None else (dq, dk)


LA2_ROTARY_INTERLEAVED = 1
LA2_POSITIONS_ROW, LA2_POSITIONS_START, LA2_POSITIONS_TABLE = 0, 1, 2
LA2_NORM_SILU, LA2_NORM_ROW, LA2_NORM_SHARED_WEIGHT, LA2_NORM_POST = 1, 2, 4, 8


# The calls below are also made for single tokens, where the host's part of a
# call is what it costs: their checks read each property of a tensor once, and
# a device that is already current is not made current again.
def _cuda(name, t):
    """The device of a call's first tensor."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _on(dev, name, t, dense=True):
    """A tensor (or None) on `dev`, contiguous unless not dense."""
    if t is None:
        return
    if t.device != dev:
        _cuda(name, t)
        raise ValueError(f"{name} is on {t.device}, other arguments on {dev}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _raw_stream(stream, dev):
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _at(t):
    return None if t is None else t.data_ptr()


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


@functools.lru_cache(maxsize=256)
def _norm_floats(op, B, H, L, d, e, dt, device_index):
    """Size of a norm backward's workspace: it depends on these alone."""
    return int(library().la2_workspace_size(op, B, H, L, d, e, dt)) // 4


def _row_strides(name, t):
    """A [B,L,columns] tensor's strides of batch and row."""
    st = t.stride()
    if st[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    return st[0], st[1]


_pack_heads = struct.Struct("=qqqq").pack  # la2_heads


def _heads(name, t):
    """la2_heads of a [B,heads,L,width] tensor: its first value and strides."""
    st = t.stride()
    if st[3] != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    return _pack_heads(t.data_ptr(), st[0], st[1], st[2])


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, factor: float = 1.0,
                       scaling: str = "none", original_length: int = 8192, fast: float = 32.0,
                       slow: float = 1.0, device="cuda"):
    """(inv_freq, scale) for rotary(): inv_freq float64 [rotary_dim / 2], pair
    i's angle per position, base^(-2i / rotary_dim), and the number that q and
    k are multiplied by.  For contexts `factor` times as long as the
    `original_length` a model was trained on, scaling is
      "none"      as trained;
      "linear"    every position divided by factor;
      "base"      the base raised so that the slowest pair turns 1 / factor as
                  fast and the fastest keeps its pace;
      "by_parts"  pairs that turn more than `fast` times over original_length
                  kept, those that turn less than `slow` times slowed down by
                  factor, a linear blend between, and scale = 1 + 0.1 ln
                  factor."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling not in ("none", "linear", "base", "by_parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    n = rotary_dim // 2
    if scaling == "base" and n > 1:
        base *= factor ** (rotary_dim / (rotary_dim - 2))
    f = [base ** (-2.0 * i / rotary_dim) for i in range(n)]
    scale = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "by_parts":
        if not fast > slow > 0.0 or original_length < 1:
            raise ValueError("fast must be above slow, slow above 0 and original_length at least 1")
        for i, x in enumerate(f):
            turns = original_length * x / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            f[i] = x * (keep + (1.0 - keep) / factor)
        scale = 1.0 + 0.1 * math.log(factor)
    return torch.tensor(f, dtype=torch.float64, device=device), scale


def _rotary_args(inv_freq, positions, B, L, dev):
    """(columns that turn, the kind of positions)"""
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be float64 [rotary_dim / 2]")
    _on(dev, "inv_freq", inv_freq)
    r = 2 * inv_freq.shape[0]
    if positions is None:
        return r, LA2_POSITIONS_ROW
    if positions.dtype != torch.int64 or tuple(positions.shape) not in ((B,), (B, L)):
        raise ValueError("positions must be int64 [B] or [B,L]")
    _on(dev, "positions", positions)
    return r, LA2_POSITIONS_START if positions.dim() == 1 else LA2_POSITIONS_TABLE


def rotary(q, k, inv_freq, positions=None, *, v=None, interleaved: bool = False,
           scale: float = 1.0, out=None, stream=None):
    """Rotary positions on q and k on their way from a projection to the
    attention.  q [B,H,L,d], k [B,Hk,L,d] and v [B,Hk,L,e] may be strided views
    (of a fused token-major projection, say) with contiguous columns; the
    results are contiguous [B,H,L,.] as forward() and decode_tokens() take them,
    k and v heads shared by H / Hk q heads repeated.  The first 2 *
    len(inv_freq) columns of every head turn (halves paired, or neighbours when
    interleaved) and are multiplied by scale; see rotary_frequencies().
    positions: None (row t is position t), int64 [B] (row t of request b is
    positions[b] + t) or int64 [B,L].  Returns (rq, rk), or with v (rq, rk, rv);
    out: buffers for them."""
    lib = _lib or library()
    dev = _cuda("q", q)
    _on(dev, "k", k, False)
    _on(dev, "v", v, False)
    B, H, L, d = shape = q.shape
    kshape, dtype = k.shape, q.dtype
    Hk = kshape[1]
    e = d if v is None else v.shape[-1]
    if kshape != (B, Hk, L, d) or (v is not None and v.shape != (B, Hk, L, e)):
        raise ValueError("q must be [B,H,L,d], k [B,Hk,L,d] and v [B,Hk,L,e]")
    if H != Hk and (Hk == 0 or H % Hk):
        raise ValueError("H must be a multiple of Hk")
    if k.dtype != dtype or (v is not None and v.dtype != dtype):
        raise ValueError("q, k and v must have one dtype")
    r, kind = _rotary_args(inv_freq, positions, B, L, dev)
    with _guard(dev, stream) as caller:
        if out is None:
            rq = q.new_empty(shape)
            rk = torch.empty_like(rq)
            rv = None if v is None else torch.empty_like(rq) if e == d else q.new_empty((B, H, L, e))
        else:
            if len(out) != (2 if v is None else 3):
                raise ValueError(f"out must be {2 if v is None else 3} buffers")
            rq, rk, rv = (*out, None)[:3]
            _out(rq, "out[0]", shape, dtype, dev)
            _out(rk, "out[1]", shape, dtype, dev)
            if v is not None:
                _out(rv, "out[2]", (B, H, L, e), dtype, dev)
        code = lib.la2_rotary(_heads("q", q), _heads("k", k), None if v is None else _heads("v", v),
                              inv_freq.data_ptr(), _at(positions), kind, rq.data_ptr(),
                              rk.data_ptr(), _at(rv), scale,
                              LA2_ROTARY_INTERLEAVED if interleaved else 0, B, H, Hk, L, d, e, r,
                              _dt(q), _raw_stream(stream, dev))
    _check(code, "la2_rotary")
    if caller is not None:
        _used_on((caller, stream), q, k, v, inv_freq, positions, rq, rk, rv)
    return (rq, rk) if v is None else (rq, rk, rv)


def rotary_backward(dq, dk, inv_freq, positions=None, *, dv=None, kv_heads=None,
                    interleaved: bool = False, scale: float = 1.0, out=None, stream=None):
    """Chain rule through rotary(): dq, dk [B,H,L,d] (and dv [B,H,L,e]) are
    the attention's gradients; returns the gradients (gq [B,H,L,d], gk
    [B,kv_heads,L,d][, gv [B,kv_heads,L,e]]) of its inputs, those of a shared
    head summed over its q heads.  kv_heads: H when None.  out: tensors of
    those shapes to write, strided views allowed (slices of a fused
    projection's gradient); by default views of token-major [B,L,heads,.]
    buffers."""
    lib = _lib or library()
    dev = _cuda("dq", dq)
    _on(dev, "dq", dq)
    _on(dev, "dk", dk)
    _on(dev, "dv", dv)
    B, H, L, d = shape = dq.shape
    dtype = dq.dtype
    Hk, e = H if kv_heads is None else int(kv_heads), (d if dv is None else dv.shape[-1])
    if dk.shape != shape or (dv is not None and dv.shape != (B, H, L, e)):
        raise ValueError("dq, dk must be [B,H,L,d] and dv [B,H,L,e]")
    if Hk < 0 or (H != Hk and (Hk == 0 or H % Hk)):
        raise ValueError("H must be a multiple of kv_heads")
    if dk.dtype != dtype or (dv is not None and dv.dtype != dtype):
        raise ValueError("dq, dk and dv must have one dtype")
    r, kind = _rotary_args(inv_freq, positions, B, L, dev)
    with _guard(dev, stream) as caller:
        shapes = ((B, H, L, d), (B, Hk, L, d), (B, Hk, L, e))[:2 if dv is None else 3]
        if out is None:
            outs = [dq.new_empty((b, n, h, w)).transpose(1, 2) for b, h, n, w in shapes]
        else:
            if len(out) != len(shapes):
                raise ValueError(f"out must be {len(shapes)} tensors")
            outs = list(out)
            for i, (x, s) in enumerate(zip(outs, shapes)):
                _on(dev, "out", x, False)
                if x.shape != s or x.dtype != dtype:
                    raise ValueError(f"out[{i}] must be {dtype} {s}")
        views = [_heads("out", x) for x in outs]
        code = lib.la2_rotary_backward(dq.data_ptr(), dk.data_ptr(), _at(dv), inv_freq.data_ptr(),
                                       _at(positions), kind, views[0], views[1],
                                       None if dv is None else views[2], scale,
                                       LA2_ROTARY_INTERLEAVED if interleaved else 0, B, H, Hk, L,
                                       d, e, r, _dt(dq), _raw_stream(stream, dev))
    _check(code, "la2_rotary_backward")
    if caller is not None:
        _used_on((caller, stream), dq, dk, dv, inv_freq, positions, *outs)
    return tuple(outs)


def _gated_args(o, gate, weight, activation, per_head, dev):
    B, H, L, e = o.shape
    if activation not in ("silu", "sigmoid"):
        raise ValueError(f"unknown activation {activation!r}")
    flags = (LA2_NORM_SILU if activation == "silu" else 0) | (0 if per_head else LA2_NORM_ROW)
    _on(dev, "o", o)
    if gate is not None:
        _on(dev, "gate", gate, False)
        if gate.shape != (B, L, H * e) or gate.dtype != o.dtype:
            raise ValueError("gate must be [B,L,H*e] of o's dtype")
    if weight is not None:
        _on(dev, "weight", weight)
        n = weight.numel()
        if weight.dtype != torch.float32 or weight.dim() != 1:
            raise ValueError("weight must be float32 [H*e] or [e]")
        if per_head and n == e:
            flags |= LA2_NORM_SHARED_WEIGHT
        elif n != H * e:
            raise ValueError("weight must be float32 [H*e], or [e] for a norm per head")
    return B, H, L, e, flags


def gated_norm(o, gate=None, weight=None, *, activation: str = "silu", per_head: bool = True,
               eps: float = 1e-6, out=None, stream=None):
    """The attention's output normed and gated for the output projection:
    u = o / sqrt(mean(o^2) + eps) * weight * a(gate), o [B,H,L,e] to u
    [B,L,H*e], the mean over each head's columns or (per_head False) over the
    token's whole row.  gate [B,L,H*e] may be a view with strided batches and
    rows (a slice of a fused projection); a is "silu" or "sigmoid".  weight
    float32 [H*e], or [e] for all heads alike (per head only), or None."""
    lib = _lib or library()
    dev = _cuda("o", o)
    B, H, L, e, flags = _gated_args(o, gate, weight, activation, per_head, dev)
    with _guard(dev, stream) as caller:
        u = (_out(out, "out", (B, L, H * e), o.dtype, dev) if out is not None
             else o.new_empty((B, L, H * e)))
        sb, sl = (0, 0) if gate is None else _row_strides("gate", gate)
        code = lib.la2_gated_norm(o.data_ptr(), _at(gate), sb, sl, _at(weight), u.data_ptr(), eps,
                                  flags, B, H, L, e, _dt(o), _raw_stream(stream, dev))
    _check(code, "la2_gated_norm")
    if caller is not None:
        _used_on((caller, stream), o, gate, weight, u)
    return u


def gated_norm_backward(du, o, gate=None, weight=None, *, activation: str = "silu",
                        per_head: bool = True, eps: float = 1e-6, out=None, workspace=None,
                        stream=None):
    """Gradients (do, dgate, dweight) of gated_norm's inputs from du
    [B,L,H*e]; dgate is None without a gate, dweight (float32, of weight's
    shape) None without a weight.  out: (do, dgate) to write; dgate may be a
    view with strided batches and rows."""
    lib = _lib or library()
    dev = _cuda("du", du)
    _on(dev, "du", du)
    _on(dev, "workspace", workspace)
    B, H, L, e, flags = _gated_args(o, gate, weight, activation, per_head, dev)
    dtype = o.dtype
    if du.shape != (B, L, H * e) or du.dtype != dtype:
        raise ValueError("du must be [B,L,H*e] of o's dtype")
    with _guard(dev, stream) as caller:
        if out is not None:
            do, dgate = out
            _out(do, "do", o.shape, dtype, dev)
            if (dgate is None) != (gate is None):
                raise ValueError("gate and dgate are both given or both None")
            if dgate is not None:
                _on(dev, "dgate", dgate, False)
                if dgate.shape != gate.shape or dgate.dtype != dtype:
                    raise ValueError("dgate must match gate's shape and dtype")
        else:
            do = torch.empty_like(o)
            dgate = None if gate is None else o.new_empty((B, L, H * e))
        dw = None if weight is None else torch.empty_like(weight)
        if workspace is None and dw is not None:
            workspace = dw.new_empty(_norm_floats(LA2_OP_GATED_NORM_BACKWARD, B, H, L, e, e,
                                                  _dt(o), dev.index))
        sb, sl = (0, 0) if gate is None else _row_strides("gate", gate)
        tb, tl = (0, 0) if gate is None else _row_strides("dgate", dgate)
        code = lib.la2_gated_norm_backward(du.data_ptr(), o.data_ptr(), _at(gate), sb, sl,
                                           _at(weight), do.data_ptr(), _at(dgate), tb, tl, _at(dw),
                                           eps, flags, B, H, L, e, _dt(o), _at(workspace),
                                           _nbytes(workspace), _raw_stream(stream, dev))
    _check(code, "la2_gated_norm_backward")
    if caller is not None:
        _used_on((caller, stream), du, o, gate, weight, workspace, do, dgate, dw)
    return do, dgate, dw


def _residual_args(x, weight, post_weight, post_norm, dev):
    """(rows, their width, flags)"""
    D = x.shape[-1]
    for name, w in (("weight", weight), ("post_weight", post_weight)):
        if w is not None:
            _on(dev, name, w)
            if w.dtype != torch.float32 or w.shape != (D,):
                raise ValueError(f"{name} must be float32 [D]")
    if post_weight is not None and not post_norm:
        raise ValueError("post_weight is given but post_norm is False")
    return x.numel() // D if D else 0, D, LA2_NORM_POST if post_norm else 0


def residual_norm(h, y=None, weight=None, *, post_norm: bool = False, post_weight=None,
                  alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6, dtype=None, out=None,
                  stream=None):
    """The residual sum after a block and the norm before the next:
    h_new = alpha h + beta p, n = h_new / sqrt(mean(h_new^2) + eps) * weight,
    with p = y or (post_norm) y / sqrt(mean(y^2) + eps) * post_weight; rows are
    the last axis.  y is of h's dtype, or bfloat16 with a float32 h; n is of
    y's.  Returns (h_new, n); without y the norm of h alone, (h, n), n of
    `dtype` (h's when None).  out: (h_new, n) to write, which may be h and y
    themselves; without y, n."""
    lib = _lib or library()
    dev = _cuda("h", h)
    _on(dev, "h", h)
    _on(dev, "y", y)
    N, D, flags = _residual_args(h, weight, post_weight, post_norm, dev)
    if y is None:
        if post_norm or alpha != 1.0:
            raise ValueError("post_norm and alpha need a block output y")
        h_new, n, dt = None, out, dtype or h.dtype
    else:
        dt = y.dtype
        if y.shape != h.shape or (dtype is not None and dtype != dt):
            raise ValueError("y must match h's shape, and dtype y's")
        h_new, n = (None, None) if out is None else out
    with _guard(dev, stream) as caller:
        if h_new is not None:
            _out(h_new, "h_new", h.shape, h.dtype, dev)
        elif y is not None:
            h_new = torch.empty_like(h)
        if n is not None:
            _out(n, "n", h.shape, dt, dev)
        else:
            n = torch.empty_like(h, dtype=dt) if y is None else torch.empty_like(y)
        code = lib.la2_residual_norm(h.data_ptr(), _dt(h), _at(y), _at(weight), _at(post_weight),
                                     _at(h_new), n.data_ptr(), alpha, beta, eps, flags, N, D,
                                     _dt(n), _raw_stream(stream, dev))
    _check(code, "la2_residual_norm")
    if caller is not None:
        _used_on((caller, stream), h, y, weight, post_weight, h_new, n)
    return (h if y is None else h_new), n


def residual_norm_backward(dn, h_new, y=None, weight=None, *, dh_new=None, post_norm: bool = False,
                           post_weight=None, alpha: float = 1.0, beta: float = 1.0,
                           eps: float = 1e-6, want_dy: bool = True, out=None, workspace=None,
                           stream=None):
    """Gradients (dh, dy, dweight, dpost_weight) of residual_norm's inputs
    from dn and dh_new (None: zero), the gradients of n and h_new; h_new is the
    stored sum and y (needed with post_norm only) the block's output.  dweight
    and dpost_weight are None without their weights, dy with want_dy False (a
    call that had no y).  out: (dh, dy) to write; dh may be dh_new itself."""
    lib = _lib or library()
    dev = _cuda("dn", dn)
    for name, x in (("dn", dn), ("h_new", h_new), ("y", y), ("dh_new", dh_new),
                    ("workspace", workspace)):
        _on(dev, name, x)
    N, D, flags = _residual_args(h_new, weight, post_weight, post_norm, dev)
    shape = h_new.shape
    if post_norm and y is None:
        raise ValueError("post_norm needs the block output y")
    if dn.shape != shape or (y is not None and (y.shape != shape or y.dtype != dn.dtype)):
        raise ValueError("dn and y must match h_new's shape and have one dtype")
    if dh_new is not None and (dh_new.shape != shape or dh_new.dtype != h_new.dtype):
        raise ValueError("dh_new must match h_new's shape and dtype")
    with _guard(dev, stream) as caller:
        dh, dy = (None, None) if out is None else out
        dh = (_out(dh, "dh", shape, h_new.dtype, dev) if dh is not None
              else torch.empty_like(h_new))
        if not want_dy:
            dy = None
        else:
            dy = _out(dy, "dy", shape, dn.dtype, dev) if dy is not None else torch.empty_like(dn)
        dw = None if weight is None else torch.empty_like(weight)
        dpw = None if post_weight is None else torch.empty_like(post_weight)
        if workspace is None and (dw is not None or dpw is not None):
            workspace = (dpw if dw is None else dw).new_empty(
                _norm_floats(LA2_OP_RESIDUAL_NORM_BACKWARD, 1, 1, N, D, D, _dt(dn), dev.index))
        code = lib.la2_residual_norm_backward(
            dn.data_ptr(), _at(dh_new), h_new.data_ptr(), _dt(h_new), _at(y), _at(weight),
            _at(post_weight), dh.data_ptr(), _at(dy), _at(dw), _at(dpw), alpha, beta, eps, flags,
            N, D, _dt(dn), _at(workspace), _nbytes(workspace), _raw_stream(stream, dev))
    _check(code, "la2_residual_norm_backward")
    if caller is not None:
        _used_on((caller, stream), dn, h_new, y, weight, dh_new, post_weight, workspace,
                 dh, dy, dw, dpw)
    return dh, dy, dw, dpw


def pool_copy(pool, src, dst, *, source=None, stream=None):
    """States moved between slots, all at once: pool[dst[n]] = pool[src[n]] as
    it was before the call (src[n] < 0: cleared; dst[n] < 0: no move), for
    forking, reordering, compacting and clearing requests.  pool float32
    [P,H,d,e], or [layers,P,H,d,e] with the same moves in every layer; src, dst
    int32 [N], the destinations distinct.  source: another pool to copy from
    (same layers, H, d, e; any number of slots).  Returns pool."""
    lib = _lib or library()
    dev = _cuda("pool", pool)
    origin = pool if source is None else source
    for name, x in (("pool", pool), ("source", source), ("src", src), ("dst", dst)):
        _on(dev, name, x)
    shape, from_shape = pool.shape, origin.shape
    dims = len(shape)
    if dims not in (4, 5) or pool.dtype != torch.float32 or origin.dtype != torch.float32:
        raise ValueError("pool and source must be float32 [P,H,d,e] or [layers,P,H,d,e]")
    layers = shape[0] if dims == 5 else 1
    H, d, e = shape[-3:]
    if source is not None and (len(from_shape) != dims or from_shape[-3:] != (H, d, e)
                               or (dims == 5 and from_shape[0] != layers)):
        raise ValueError("source must match pool but for its number of slots")
    if (src.dtype != torch.int32 or src.dim() != 1 or dst.dtype != torch.int32
            or dst.shape != src.shape):
        raise ValueError("src and dst must be int32 [N]")
    with _guard(dev, stream) as caller:
        code = lib.la2_pool_copy(origin.data_ptr(), from_shape[-4], pool.data_ptr(), shape[-4],
                                 src.data_ptr(), dst.data_ptr(), src.shape[0], layers, H, d, e,
                                 _raw_stream(stream, dev))
    _check(code, "la2_pool_copy")
    if caller is not None:
        _used_on((caller, stream), pool, source, src, dst)
    return pool


def decode_step(q, k, v, lam, kv, *, out=None, stream=None):
    """kv <- lam kv + k^T v (in place); returns o = q kv."""
    lib = library()
    dev = _devices(("q", q), ("k", k), ("v", v), ("lam", lam), ("kv", kv))
    B, H, d = q.shape
    e = v.shape[-1]
    if kv.dtype != torch.float32 or kv.shape != (B, H, d, e):
        raise ValueError("kv must be float32 [B,H,d,e]")
    with _guard(dev, stream) as caller:
        o = (_out(out, "out", (B, H, e), q.dtype, dev) if out is not None
             else torch.empty((B, H, e), dtype=q.dtype, device=dev))
        code = lib.la2_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(lam), _ptr(kv), _ptr(o),
                                   B, H, d, e, _dt(q), _stream(stream, dev))
    _check(code, "la2_decode_step")
    if caller is not None:
        _used_on((caller, stream), q, k, v, lam, kv, o)
    return o


def last_device_error(stream=None) -> int:
    return int(library().la2_last_device_error(_stream(stream)))


def trace_read():
    """Trace buffer as a [16 events, 512 blocks] int64 tensor (ns; 0 = unset)."""
    lib = library()
    n = int(lib.la2_trace_read(None, 0))
    buf = torch.zeros(n, dtype=torch.int64)
    lib.la2_trace_read(ctypes.c_void_p(buf.data_ptr()), n)
    return buf.view(16, -1)


def profile_enable(on: bool = True):
    library().la2_profile_enable(1 if on else 0)


def profile_report() -> dict:
    # one report clears the records, so size the buffer generously up front
    n = 1 << 16
    buf = ctypes.create_string_buffer(n)
    library().la2_profile_report(buf, n)
    return json.loads(buf.value.decode() or "{}")
