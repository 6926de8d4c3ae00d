"""The gated delta rule: binding of m3_delta_fwd, m3_delta_step and
m3_delta_bwd (include/m3scan.h).  Argument marshalling only, as in binding.py.

    S_t = a_t S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - (a_t S_{t-1})^T k_t),
    o_t = scale S_t^T q_t,           a_t = exp(g_t)

Layouts (contiguous):
    q, k [Bt, L, G, N]   v, o [Bt, L, H, P]   g, beta [Bt, L, H] float32
    h [Bt, H, N, P] float32: the state record
N is 32, 64 or 128, P is 32, 64, 96 or 128, H a multiple of G; float32 or
bfloat16 tokens.

Options: scale (default N ** -0.5); l2norm: rows of q and k divided by
sqrt(sum of squares + norm_eps); cu_seqlens (int32 [nseq + 1]) and max_seqlen:
sequences packed along the token axis of [1, T, ...] arrays; slots (int32, one
per row): row b's record is slot slots[b] of a pool h [slots, H, N, P], read
and written in place.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from .binding import M3Error, _check, _io_code, _ptr, load_library

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class DeltaArgs(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("nheads", _i64), ("ngroups", _i64),
                ("headdim", _i64), ("dstate", _i64), ("io_dtype", _i32), ("l2norm", _i32),
                ("scale", _f32), ("norm_eps", _f32),
                ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("h_in", _vp),
                ("o", _vp), ("h_out", _vp), ("cu_seqlens", _vp), ("max_seqlen", _i64),
                ("slots", _vp), ("nslots", _i64), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t)]


class DeltaStepArgs(ctypes.Structure):
    _fields_ = [("batch", _i64), ("nheads", _i64), ("ngroups", _i64), ("headdim", _i64),
                ("dstate", _i64), ("io_dtype", _i32), ("l2norm", _i32),
                ("scale", _f32), ("norm_eps", _f32),
                ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("h", _vp),
                ("o", _vp), ("slots", _vp), ("nslots", _i64)]


class DeltaBwdArgs(ctypes.Structure):
    _fields_ = [("in_", DeltaArgs), ("dout", _vp), ("dh_out", _vp), ("dq", _vp), ("dk", _vp),
                ("dv", _vp), ("dg", _vp), ("dbeta", _vp), ("dh_in", _vp)]


class DeltaGrads(NamedTuple):
    """Gradients from m3_delta_bwd (float32, shapes of the inputs)."""
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    dg: torch.Tensor
    dbeta: torch.Tensor
    dh_in: Optional[torch.Tensor]


@contextlib.contextmanager
def on_device_of(t: torch.Tensor, stream=None):
    """The tensor's device made current, and `stream` (None: that device's
    current stream) the stream that the call's own allocations belong to.
    Yields the stream's handle."""
    with torch.cuda.device(t.device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
        else:
            if stream.device != t.device:
                raise ValueError("stream belongs to %s, the tensors to %s" % (stream.device, t.device))
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def same_device(t: torch.Tensor, name: str, device):
    if t.device != device:
        raise ValueError("%s is on %s, q on %s" % (name, t.device, device))


def _shapes(q, k, v, g, beta, step):
    """(Bx, L, H, G, N, P) after the checks of the token arrays."""
    lead = 1 if step else 2
    if q.dim() != lead + 2 or v.dim() != lead + 2:
        raise ValueError("q and v: expected %d dimensions, got %d and %d" % (lead + 2, q.dim(), v.dim()))
    tok, (G, N), (H, P) = tuple(q.shape[:lead]), q.shape[lead:], v.shape[lead:]
    _io_code(q.dtype)
    for t, name, shape, dt in ((q, "q", tok + (G, N), q.dtype), (k, "k", tok + (G, N), q.dtype),
                               (v, "v", tok + (H, P), q.dtype), (g, "g", tok + (H,), torch.float32),
                               (beta, "beta", tok + (H,), torch.float32)):
        _check(t, name, shape, dt)
        same_device(t, name, q.device)
    if G < 1 or H % G != 0:
        raise ValueError("heads (%d) must be a multiple of q and k's groups (%d)" % (H, G))
    return tok[0], (1 if step else tok[1]), H, G, N, P


def _common(a, H, G, N, P, io, scale, l2norm, norm_eps):
    a.nheads, a.ngroups, a.headdim, a.dstate, a.io_dtype = H, G, P, N, io
    a.scale = float(N ** -0.5 if scale is None else scale)
    a.l2norm, a.norm_eps = int(bool(l2norm)), float(norm_eps)


def _rows(a, cu_seqlens, max_seqlen, Bx, L, device):
    """Batch rows or packed sequences of the call."""
    if cu_seqlens is None:
        a.batch, a.seqlen = Bx, L
        return Bx
    if Bx != 1:
        raise ValueError("packed sequences: token arrays must have a leading dimension of 1")
    if cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens: at least one offset is needed")
    _check(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32)
    same_device(cu_seqlens, "cu_seqlens", device)
    a.batch, a.seqlen = cu_seqlens.numel() - 1, L
    a.cu_seqlens = cu_seqlens.data_ptr()
    a.max_seqlen = int(L if max_seqlen is None else max_seqlen)
    return a.batch


def _take_slots(a, slots, rows, pool, device):
    _check(slots, "slots", (rows,), torch.int32)
    same_device(slots, "slots", device)
    if pool is None:
        raise ValueError("slots need a pool: h, or h_out for records that start from zero")
    a.slots, a.nslots = slots.data_ptr(), pool.shape[0]


def _workspace(need, given, device):
    if need == 0:
        return None
    if given is None or given.numel() * given.element_size() < need:
        return torch.empty(int(need), dtype=torch.uint8, device=device)
    _check(given, "workspace", given.shape, given.dtype)
    same_device(given, "workspace", device)
    return given


def m3_delta_supported(dstate: int, headdim: int, io_dtype: int) -> bool:
    return bool(load_library().m3_delta_supported(dstate, headdim, io_dtype))


def m3_delta_fwd(q, k, v, g, beta, h: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                 l2norm: bool = False, norm_eps: float = 1e-6, return_state: bool = True,
                 o: Optional[torch.Tensor] = None, h_out: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None, max_seqlen: Optional[int] = None,
                 slots: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None):
    """Prefill of the gated delta rule.  Returns (o, state after the last token
    or None).  ``h_out`` may be ``h`` (the record is updated in place); with
    ``slots`` that is the default.  Without ``return_state`` and ``h_out`` no
    state is written."""
    lib = load_library()
    Bx, L, H, G, N, P = _shapes(q, k, v, g, beta, False)
    a = DeltaArgs()
    _common(a, H, G, N, P, _io_code(q.dtype), scale, l2norm, norm_eps)
    rows = _rows(a, cu_seqlens, max_seqlen, Bx, L, q.device)
    with on_device_of(q, stream) as handle:
        if slots is not None:
            _take_slots(a, slots, rows, h if h is not None else h_out, q.device)
            if h_out is None and return_state:
                h_out = h
        elif h_out is None and return_state:
            h_out = torch.empty(rows, H, N, P, dtype=torch.float32, device=q.device)
        for t, name in ((h, "h"), (h_out, "h_out")):
            if t is not None:
                _check(t, name, (a.nslots if slots is not None else rows, H, N, P), torch.float32)
                same_device(t, name, q.device)
        if o is None:
            o = torch.empty_like(v)
        _check(o, "o", v.shape, v.dtype)
        same_device(o, "o", q.device)
        a.q, a.k, a.v, a.g, a.beta = (t.data_ptr() for t in (q, k, v, g, beta))
        a.h_in, a.o, a.h_out = _ptr(h), o.data_ptr(), _ptr(h_out)
        ws = _workspace(lib.m3_delta_workspace_bytes(ctypes.byref(a)), workspace, q.device)
        if ws is not None:
            a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
        st = lib.m3_delta_fwd(ctypes.byref(a), handle)
    if st != 0:
        raise M3Error(st, "m3_delta_fwd")
    return o, h_out


def m3_delta_workspace_bytes(q, v, *, cu_seqlens=None, max_seqlen=None) -> int:
    """Workspace bytes of m3_delta_fwd on token arrays like q and v."""
    Bx, L, G, N = q.shape
    a = DeltaArgs()
    _common(a, v.shape[2], G, N, v.shape[3], _io_code(q.dtype), None, False, 0.0)
    _rows(a, cu_seqlens, max_seqlen, Bx, L, q.device)
    return int(load_library().m3_delta_workspace_bytes(ctypes.byref(a)))


def m3_delta_step(q, k, v, g, beta, h: torch.Tensor, *, scale: Optional[float] = None,
                  l2norm: bool = False, norm_eps: float = 1e-6, o: Optional[torch.Tensor] = None,
                  slots: Optional[torch.Tensor] = None, stream=None):
    """One token for every row: q, k [Bt, G, N], v [Bt, H, P], g, beta [Bt, H];
    ``h`` is updated in place.  Returns o_t."""
    Bt, _, H, G, N, P = _shapes(q, k, v, g, beta, True)
    a = DeltaStepArgs(batch=Bt)
    _common(a, H, G, N, P, _io_code(q.dtype), scale, l2norm, norm_eps)
    if slots is not None:
        _take_slots(a, slots, Bt, h, q.device)
    _check(h, "h", (h.shape[0] if slots is not None else Bt, H, N, P), torch.float32)
    same_device(h, "h", q.device)
    with on_device_of(q, stream) as handle:
        if o is None:
            o = torch.empty_like(v)
        _check(o, "o", v.shape, v.dtype)
        same_device(o, "o", q.device)
        a.q, a.k, a.v, a.g, a.beta = (t.data_ptr() for t in (q, k, v, g, beta))
        a.h, a.o = h.data_ptr(), o.data_ptr()
        st = load_library().m3_delta_step(ctypes.byref(a), handle)
    if st != 0:
        raise M3Error(st, "m3_delta_step")
    return o


def m3_delta_bwd(q, k, v, g, beta, do, h: Optional[torch.Tensor] = None,
                 dh_out: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                 l2norm: bool = False, norm_eps: float = 1e-6, state_grad: bool = True,
                 cu_seqlens: Optional[torch.Tensor] = None, max_seqlen: Optional[int] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> DeltaGrads:
    """Gradients of sum(do * o) + sum(dh_out * h_L) of m3_delta_fwd with respect
    to every input as given; ``state_grad`` also returns that of the input
    state (a zero state when ``h`` is None)."""
    lib = load_library()
    Bx, L, H, G, N, P = _shapes(q, k, v, g, beta, False)
    b = DeltaBwdArgs()
    a = b.in_
    _common(a, H, G, N, P, _io_code(q.dtype), scale, l2norm, norm_eps)
    rows = _rows(a, cu_seqlens, max_seqlen, Bx, L, q.device)
    _check(do, "do", v.shape, v.dtype)
    same_device(do, "do", q.device)
    for t, name in ((h, "h"), (dh_out, "dh_out")):
        if t is not None:
            _check(t, name, (rows, H, N, P), torch.float32)
            same_device(t, name, q.device)
    with on_device_of(q, stream) as handle:
        f32 = dict(dtype=torch.float32, device=q.device)
        r = DeltaGrads(torch.empty(q.shape, **f32), torch.empty(k.shape, **f32),
                       torch.empty(v.shape, **f32), torch.empty(g.shape, **f32),
                       torch.empty(beta.shape, **f32),
                       torch.empty(rows, H, N, P, **f32) if state_grad else None)
        a.q, a.k, a.v, a.g, a.beta, a.h_in = (_ptr(t) for t in (q, k, v, g, beta, h))
        b.dout, b.dh_out = do.data_ptr(), _ptr(dh_out)
        b.dq, b.dk, b.dv, b.dg, b.dbeta, b.dh_in = (_ptr(t) for t in r)
        ws = _workspace(lib.m3_delta_bwd_workspace_bytes(ctypes.byref(b)), workspace, q.device)
        if ws is not None:
            a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
        st = lib.m3_delta_bwd(ctypes.byref(b), handle)
    if st != 0:
        raise M3Error(st, "m3_delta_bwd")
    return r
