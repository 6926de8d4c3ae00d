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
from typing import Optional, Sequence

import torch

from .binding import M3Error, _check, _ptr, load_library
from .delta import on_device_of

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


def _desc(pool: Sequence[torch.Tensor], name: str) -> PoolDesc:
    arrays = (pool,) if isinstance(pool, torch.Tensor) else tuple(pool)
    if not 1 <= len(arrays) <= MAX_ARRAYS:
        raise ValueError("%s: 1 to %d arrays, got %d" % (name, MAX_ARRAYS, len(arrays)))
    d = PoolDesc(narrays=len(arrays))
    for i, t in enumerate(arrays):
        if t.dim() < 1:
            raise ValueError("%s[%d] has no slot axis" % (name, i))
        _check(t, "%s[%d]" % (name, i), (arrays[0].shape[0],) + tuple(t.shape[1:]), t.dtype)
        if t.device != arrays[0].device:
            raise ValueError("%s[%d] is on %s, the first array on %s" % (name, i, t.device, arrays[0].device))
        d.data[i] = t.data_ptr()
        row = t.element_size()
        for n in t.shape[1:]:
            row *= n
        d.row_bytes[i] = row
    d.slots = arrays[0].shape[0]
    return d


def _first(pool):
    return pool if isinstance(pool, torch.Tensor) else pool[0]


def _index(t, name, n, device):
    _check(t, name, (n,), torch.int32)
    if t.device != device:
        raise ValueError("%s is on %s, the pool on %s" % (name, t.device, device))


def _bytes(need, given, device):
    if need == 0:
        return None
    if given is None or given.numel() * given.element_size() < need:
        return torch.empty(int(need), dtype=torch.uint8, device=device)
    _check(given, "workspace", given.shape, given.dtype)
    if given.device != device:
        raise ValueError("workspace is on %s, the pool on %s" % (given.device, device))
    return given


def _run(fn, a, need, workspace, device, handle, what):
    ws = _bytes(need, workspace, device)
    if ws is not None:
        a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    st = fn(ctypes.byref(a), handle)
    if st != 0:
        raise M3Error(st, what)


def m3_pool_copy(src, dst, src_slot: torch.Tensor, dst_slot: torch.Tensor, *,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Record src_slot[i] of ``src`` to slot dst_slot[i] of ``dst`` (which may be
    ``src``), as if every source were read first; the last pair that names a
    slot wins; src_slot[i] < 0 clears the slot; pairs outside are left out."""
    lib = load_library()
    a = PoolCopyArgs(src=_desc(src, "src"), dst=_desc(dst, "dst"), count=src_slot.numel())
    dev = _first(dst).device
    if _first(src).device != dev:
        raise ValueError("src is on %s, dst on %s" % (_first(src).device, dev))
    _index(src_slot, "src_slot", a.count, dev)
    _index(dst_slot, "dst_slot", a.count, dev)
    a.src_slot, a.dst_slot = src_slot.data_ptr(), dst_slot.data_ptr()
    with on_device_of(_first(dst), stream) as handle:
        need = lib.m3_pool_copy_workspace_bytes(ctypes.byref(a))
        _run(lib.m3_pool_copy, a, need, workspace, dev, handle, "m3_pool_copy")


def m3_pool_fork(pool, live: torch.Tensor, parents: torch.Tensor, *,
                 children: Optional[torch.Tensor] = None, live_out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """For each parents[i] the lowest free slot, a copy of that record (< 0: a
    cleared one) in it, marked in ``live_out`` (default: ``live`` itself).
    Returns the slots, -1 where none was left or the parent is not live."""
    lib = load_library()
    dev = _first(pool).device
    a = PoolForkArgs(pool=_desc(pool, "pool"), count=parents.numel())
    _index(live, "live", a.pool.slots, dev)
    _index(parents, "parents", a.count, dev)
    live_out = live if live_out is None else live_out
    _index(live_out, "live_out", a.pool.slots, dev)
    with on_device_of(_first(pool), stream) as handle:
        if children is None:
            children = torch.empty_like(parents)
        _index(children, "children", a.count, dev)
        a.live, a.live_out, a.parents, a.children = (t.data_ptr() for t in (live, live_out, parents, children))
        _run(lib.m3_pool_fork, a, 4 * a.count, workspace, dev, handle, "m3_pool_fork")
    return children


def m3_pool_compact(pool, live: torch.Tensor, *, new_slot: Optional[torch.Tensor] = None,
                    count: Optional[torch.Tensor] = None, live_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the live records past the front into the front's free slots.
    Returns new_slot: where each slot's record is now (-1: free).  ``count``
    (int32 [1]) receives the number of live records; ``live_out`` (may be
    ``live``) the new marks."""
    lib = load_library()
    dev = _first(pool).device
    a = PoolCompactArgs(pool=_desc(pool, "pool"))
    _index(live, "live", a.pool.slots, dev)
    with on_device_of(_first(pool), stream) as handle:
        if new_slot is None:
            new_slot = torch.empty_like(live)
        for t, name, n in ((new_slot, "new_slot", a.pool.slots), (count, "count", 1),
                           (live_out, "live_out", a.pool.slots)):
            if t is not None:
                _index(t, name, n, dev)
        a.live, a.new_slot = live.data_ptr(), new_slot.data_ptr()
        a.live_out, a.count = _ptr(live_out), _ptr(count)
        _run(lib.m3_pool_compact, a, 4 * (a.pool.slots + 1), workspace, dev, handle, "m3_pool_compact")
    return new_slot


def m3_pool_free(live: torch.Tensor, slots: torch.Tensor, *, stream=None) -> None:
    """Marks the slots as free; entries outside the pool are left out."""
    _index(live, "live", live.numel(), live.device)
    _index(slots, "slots", slots.numel(), live.device)
    with on_device_of(live, stream) as handle:
        st = load_library().m3_pool_free(live.data_ptr(), live.numel(), slots.data_ptr(), slots.numel(), handle)
    if st != 0:
        raise M3Error(st, "m3_pool_free")
