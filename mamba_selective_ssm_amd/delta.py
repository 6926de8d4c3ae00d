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
sqrt(sum of squares + norm_eps); cu_seqlens (int32 [nseq + 1]) and max_seqlen
(a bound of the lengths, default T): sequences packed along the token axis of
[1, T, ...] arrays; slots (int32, one
per row): row b's record is slot slots[b] of a pool h [slots, H, N, P], read
and written in place.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import NamedTuple, Optional

import torch

from .binding import M3Error, _check, _io_code, load_library

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


def packer(cls):
    """A function from all of a structure's values, in their order, to its
    bytes: a call costs one of these instead of an attribute store per field."""
    codes = {_i64: "q", _i32: "i", _f32: "f", _vp: "P", ctypes.c_size_t: "N"}

    def fmt(c):
        return "".join(fmt(f) if isinstance(f, type) and issubclass(f, ctypes.Structure) else
                       codes[f._type_] * f._length_ if hasattr(f, "_length_") else codes[f] for _, f in c._fields_)

    s = struct.Struct("@" + fmt(cls))
    assert s.size == ctypes.sizeof(cls), cls
    return s.pack


_pack_fwd, _pack_step, _pack_bwd = packer(DeltaArgs), packer(DeltaStepArgs), packer(DeltaBwdArgs)


# The handle alone: building a Stream object around it takes 2.7 of a one-token
# step's 12 us.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def enter(device, stream):
    """The handle of the stream that a call on `device` runs on (None: the
    device's current stream), and the contexts that make that device and
    stream current, which the call's own allocations follow (None: they are)."""
    if stream is None and torch.cuda.current_device() == device.index:
        return _current_stream(device.index), None
    ctx = contextlib.ExitStack()
    ctx.enter_context(torch.cuda.device(device))
    if stream is None:
        return _current_stream(device.index), ctx
    if stream.device != device:
        ctx.close()
        raise ValueError("stream belongs to %s, the tensors to %s" % (stream.device, device))
    ctx.enter_context(torch.cuda.stream(stream))
    return stream.cuda_stream, ctx


def expect(t: torch.Tensor, name: str, shape, dtype, device):
    """_check, and the device that all of a call's tensors share."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _check(t, name, shape, dtype)
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))


def _shapes(q, k, v, g, beta, step):
    """(token dimensions, H, G, N, P, io code, device) after the checks of the token arrays."""
    lead = 1 if step else 2
    if q.dim() != lead + 2 or v.dim() != lead + 2:
        raise ValueError("q and v: expected %d dimensions, got %d and %d" % (lead + 2, q.dim(), v.dim()))
    sq, sv, dt, dev = tuple(q.shape), tuple(v.shape), q.dtype, q.device
    tok, (G, N), (H, P) = sq[:lead], sq[lead:], sv[lead:]
    io = _io_code(dt)
    if dev.type != "cuda":
        raise ValueError("q must be a device tensor")
    expect(q, "q", sq, dt, dev)
    expect(k, "k", sq, dt, dev)
    expect(v, "v", tok + (H, P), dt, dev)
    expect(g, "g", tok + (H,), torch.float32, dev)
    expect(beta, "beta", tok + (H,), torch.float32, dev)
    if G < 1 or H % G != 0:
        raise ValueError("heads (%d) must be a multiple of q and k's groups (%d)" % (H, G))
    return tok, H, G, N, P, io, dev


def _rows(cu_seqlens, max_seqlen, tok, dev):
    """(batch rows or packed sequences, offsets' address, longest) of a call."""
    if cu_seqlens is None:
        return tok[0], 0, 0
    if tok[0] != 1:
        raise ValueError("packed sequences: token arrays must have a leading dimension of 1")
    n = cu_seqlens.numel()
    if n < 1:
        raise ValueError("cu_seqlens: at least one offset is needed")
    expect(cu_seqlens, "cu_seqlens", (n,), torch.int32, dev)
    return n - 1, cu_seqlens.data_ptr(), int(tok[1] if max_seqlen is None else max_seqlen)


def workspace_of(need, given, dev):
    """(tensor to keep, address, bytes): `given` where it is large enough."""
    if need == 0:
        return None, 0, 0
    if given is None or given.numel() * given.element_size() < need:
        given = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        expect(given, "workspace", given.shape, given.dtype, dev)
    return given, given.data_ptr(), given.numel() * given.element_size()


def address(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


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
    tok, H, G, N, P, io, dev = _shapes(q, k, v, g, beta, False)
    rows, cu, longest = _rows(cu_seqlens, max_seqlen, tok, dev)
    handle, ctx = enter(dev, stream)
    try:
        nslots = at = 0
        if slots is not None:
            expect(slots, "slots", (rows,), torch.int32, dev)
            pool = h if h is not None else h_out
            if pool is None:
                raise ValueError("slots need a pool: h, or h_out for records that start from zero")
            nslots, at = pool.shape[0], slots.data_ptr()
            if h_out is None and return_state:
                h_out = h
        elif h_out is None and return_state:
            h_out = torch.empty((rows, H, N, P), dtype=torch.float32, device=dev)
        record = (nslots if slots is not None else rows, H, N, P)
        if h is not None:
            expect(h, "h", record, torch.float32, dev)
        if h_out is not None:
            expect(h_out, "h_out", record, torch.float32, dev)
        if o is None:
            o = torch.empty_like(v)
        else:
            expect(o, "o", v.shape, v.dtype, dev)
        sizes = (rows, tok[1], H, G, P, N, io, 1 if l2norm else 0, N ** -0.5 if scale is None else scale, norm_eps)
        need = lib.m3_delta_workspace_bytes(_pack_fwd(*sizes, 0, 0, 0, 0, 0, 0, 0, 0, cu, longest, 0, 0, 0, 0))
        ws, wp, wn = workspace_of(need, workspace, dev)
        st = lib.m3_delta_fwd(_pack_fwd(*sizes, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                                        address(h), o.data_ptr(), address(h_out), cu, longest, at, nslots, wp, wn), handle)
    finally:
        if ctx is not None:
            ctx.close()
    if st != 0:
        raise M3Error(st, "m3_delta_fwd")
    return o, h_out


def m3_delta_workspace_bytes(q, v, *, cu_seqlens=None, max_seqlen=None) -> int:
    """Workspace bytes of m3_delta_fwd on token arrays like q and v."""
    tok, (G, N), (H, P) = tuple(q.shape[:2]), q.shape[2:], v.shape[2:]
    rows, cu, longest = _rows(cu_seqlens, max_seqlen, tok, q.device)
    return load_library().m3_delta_workspace_bytes(
        _pack_fwd(rows, tok[1], H, G, P, N, _io_code(q.dtype), 0, 1.0, 0.0, 0, 0, 0, 0, 0, 0, 0, 0, cu, longest, 0, 0, 0, 0))


def m3_delta_step(q, k, v, g, beta, h: torch.Tensor, *, scale: Optional[float] = None,
                  l2norm: bool = False, norm_eps: float = 1e-6, o: Optional[torch.Tensor] = None,
                  slots: Optional[torch.Tensor] = None, stream=None):
    """One token for every row: q, k [Bt, G, N], v [Bt, H, P], g, beta [Bt, H];
    ``h`` is updated in place.  Returns o_t."""
    (Bt,), H, G, N, P, io, dev = _shapes(q, k, v, g, beta, True)
    nslots = at = 0
    if slots is not None:
        expect(slots, "slots", (Bt,), torch.int32, dev)
        nslots, at = h.shape[0], slots.data_ptr()
    expect(h, "h", (nslots if slots is not None else Bt, H, N, P), torch.float32, dev)
    handle, ctx = enter(dev, stream)
    try:
        if o is None:
            o = torch.empty_like(v)
        else:
            expect(o, "o", v.shape, v.dtype, dev)
        st = load_library().m3_delta_step(
            _pack_step(Bt, H, G, P, N, io, 1 if l2norm else 0, N ** -0.5 if scale is None else scale, norm_eps, q.data_ptr(),
                       k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), h.data_ptr(), o.data_ptr(), at, nslots), handle)
    finally:
        if ctx is not None:
            ctx.close()
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
    tok, H, G, N, P, io, dev = _shapes(q, k, v, g, beta, False)
    rows, cu, longest = _rows(cu_seqlens, max_seqlen, tok, dev)
    expect(do, "do", v.shape, v.dtype, dev)
    for t, name in ((h, "h"), (dh_out, "dh_out")):
        if t is not None:
            expect(t, name, (rows, H, N, P), torch.float32, dev)
    handle, ctx = enter(dev, stream)
    try:
        f32 = dict(dtype=torch.float32, device=dev)
        r = DeltaGrads(torch.empty(q.shape, **f32), torch.empty(k.shape, **f32),
                       torch.empty(v.shape, **f32), torch.empty(g.shape, **f32),
                       torch.empty(beta.shape, **f32),
                       torch.empty((rows, H, N, P), **f32) if state_grad else None)

        def args(wp, wn):
            return _pack_bwd(rows, tok[1], H, G, P, N, io, 1 if l2norm else 0, N ** -0.5 if scale is None else scale, norm_eps,
                             q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), address(h), 0, 0, cu,
                             longest, 0, 0, wp, wn, do.data_ptr(), address(dh_out), *(address(t) for t in r))

        ws, wp, wn = workspace_of(lib.m3_delta_bwd_workspace_bytes(args(0, 0)), workspace, dev)
        st = lib.m3_delta_bwd(args(wp, wn), handle)
    finally:
        if ctx is not None:
            ctx.close()
    if st != 0:
        raise M3Error(st, "m3_delta_bwd")
    return r
