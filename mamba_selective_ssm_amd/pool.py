"""Pools of state records: binding of m3_pool_copy, m3_pool_fork,
m3_pool_compact and m3_pool_free (include/m3scan.h).

A pool is a sequence of up to 8 contiguous device tensors with one record per
slot along their leading axis: a State (h, B_prev, x_prev) of the Mamba-3
mixer, (h,) of the delta rule, or any other.  ``live`` is an int32 tensor of
one value per slot, 0 where the slot is free.  Every decision is taken on the
device; no call waits for it.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import torch

from .binding import M3Error, load_library
from .delta import address, enter, expect, packer, workspace_of

MAX_ARRAYS = 8
_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class PoolDesc(ctypes.Structure):
    _fields_ = [("slots", _i64), ("narrays", _i32), ("reserved", _i32),
                ("data", _vp * MAX_ARRAYS), ("row_bytes", _i64 * MAX_ARRAYS)]


class PoolCopyArgs(ctypes.Structure):
    _fields_ = [("src", PoolDesc), ("dst", PoolDesc), ("src_slot", _vp), ("dst_slot", _vp),
                ("count", _i64), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class PoolForkArgs(ctypes.Structure):
    _fields_ = [("pool", PoolDesc), ("live", _vp), ("live_out", _vp), ("parents", _vp),
                ("children", _vp), ("count", _i64), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t)]


class PoolCompactArgs(ctypes.Structure):
    _fields_ = [("pool", PoolDesc), ("live", _vp), ("live_out", _vp), ("new_slot", _vp),
                ("count", _vp), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


_pack_copy, _pack_fork, _pack_compact = packer(PoolCopyArgs), packer(PoolForkArgs), packer(PoolCompactArgs)


def _desc(pool: Sequence[torch.Tensor], name: str):
    """(slots, device, the values of an m3_pool)."""
    arrays = (pool,) if isinstance(pool, torch.Tensor) else tuple(pool)
    n = len(arrays)
    if not 1 <= n <= MAX_ARRAYS:
        raise ValueError("%s: 1 to %d arrays, got %d" % (name, MAX_ARRAYS, n))
    dev, slots = arrays[0].device, None
    at, rows = [0] * MAX_ARRAYS, [0] * MAX_ARRAYS
    if dev.type != "cuda":
        raise ValueError("%s[0] must be a device tensor" % name)
    for i, t in enumerate(arrays):
        shape = tuple(t.shape)
        if not shape:
            raise ValueError("%s[%d] has no slot axis" % (name, i))
        slots = shape[0] if slots is None else slots
        expect(t, "%s[%d]" % (name, i), (slots,) + shape[1:], t.dtype, dev)
        at[i], rows[i] = t.data_ptr(), t.element_size() * math.prod(shape[1:])
    return slots, dev, (slots, n, 0, *at, *rows)


def m3_pool_copy(src, dst, src_slot: torch.Tensor, dst_slot: torch.Tensor, *,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Record src_slot[i] of ``src`` to slot dst_slot[i] of ``dst`` (which may be
    ``src``), as if every source were read first; the last pair that names a
    slot wins; src_slot[i] < 0 clears the slot; pairs outside are left out."""
    lib = load_library()
    _, dev, s = _desc(src, "src")
    _, dd, d = _desc(dst, "dst")
    if dd != dev:
        raise ValueError("src is on %s, dst on %s" % (dev, dd))
    n = src_slot.numel()
    expect(src_slot, "src_slot", (n,), torch.int32, dev)
    expect(dst_slot, "dst_slot", (n,), torch.int32, dev)
    handle, ctx = enter(dev, stream)
    try:
        head = (*s, *d, src_slot.data_ptr(), dst_slot.data_ptr(), n)
        ws, wp, wn = workspace_of(lib.m3_pool_copy_workspace_bytes(_pack_copy(*head, 0, 0)), workspace, dev)
        st = lib.m3_pool_copy(_pack_copy(*head, wp, wn), handle)
    finally:
        if ctx is not None:
            ctx.close()
    if st != 0:
        raise M3Error(st, "m3_pool_copy")


def m3_pool_fork(pool, live: torch.Tensor, parents: torch.Tensor, *,
                 children: Optional[torch.Tensor] = None, live_out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """For each parents[i] the lowest free slot, a copy of that record (< 0: a
    cleared one) in it, marked in ``live_out`` (default: ``live`` itself).
    Returns the slots, -1 where none was left or the parent was not live before
    the call."""
    slots, dev, d = _desc(pool, "pool")
    n = parents.numel()
    live_out = live if live_out is None else live_out
    expect(live, "live", (slots,), torch.int32, dev)
    expect(live_out, "live_out", (slots,), torch.int32, dev)
    expect(parents, "parents", (n,), torch.int32, dev)
    handle, ctx = enter(dev, stream)
    try:
        if children is None:
            children = torch.empty_like(parents)
        else:
            expect(children, "children", (n,), torch.int32, dev)
        ws, wp, wn = workspace_of(4 * n, workspace, dev)
        st = load_library().m3_pool_fork(_pack_fork(*d, live.data_ptr(), live_out.data_ptr(), parents.data_ptr(),
                                                    children.data_ptr(), n, wp, wn), handle)
    finally:
        if ctx is not None:
            ctx.close()
    if st != 0:
        raise M3Error(st, "m3_pool_fork")
    return children


def m3_pool_compact(pool, live: torch.Tensor, *, new_slot: Optional[torch.Tensor] = None,
                    count: Optional[torch.Tensor] = None, live_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the live records past the front into the front's free slots.
    Returns new_slot: where each slot's record is now (-1: free).  ``count``
    (int32 [1]) receives the number of live records; ``live_out`` (may be
    ``live``) the new marks."""
    slots, dev, d = _desc(pool, "pool")
    expect(live, "live", (slots,), torch.int32, dev)
    handle, ctx = enter(dev, stream)
    try:
        if new_slot is None:
            new_slot = torch.empty_like(live)
        for t, name, n in ((new_slot, "new_slot", slots), (count, "count", 1), (live_out, "live_out", slots)):
            if t is not None:
                expect(t, name, (n,), torch.int32, dev)
        ws, wp, wn = workspace_of(4 * (slots + 1), workspace, dev)
        st = load_library().m3_pool_compact(_pack_compact(*d, live.data_ptr(), address(live_out), new_slot.data_ptr(),
                                                          address(count), wp, wn), handle)
    finally:
        if ctx is not None:
            ctx.close()
    if st != 0:
        raise M3Error(st, "m3_pool_compact")
    return new_slot


def m3_pool_free(live: torch.Tensor, slots: torch.Tensor, *, stream=None) -> None:
    """Marks the slots as free; entries outside the pool are left out."""
    if live.device.type != "cuda":
        raise ValueError("live must be a device tensor")
    expect(live, "live", (live.numel(),), torch.int32, live.device)
    expect(slots, "slots", (slots.numel(),), torch.int32, live.device)
    handle, ctx = enter(live.device, stream)
    try:
        st = load_library().m3_pool_free(live.data_ptr(), live.numel(), slots.data_ptr(), slots.numel(), handle)
    finally:
        if ctx is not None:
            ctx.close()
    if st != 0:
        raise M3Error(st, "m3_pool_free")
