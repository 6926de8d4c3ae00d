"""The gated delta rule's and the record pools' C ABI without a GPU: structure
layouts, the workspace sizes, and every refusal, given before any HIP call (the
pointers are never dereferenced)."""
import ctypes
import os
import subprocess

import pytest
import torch

from mamba_selective_ssm_amd import binding, delta, m3_delta_fwd, m3_delta_step, m3_pool_copy, m3_pool_free, pool

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000
GIB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def test_struct_layouts_match_header(tmp_path):
    structs = [("m3_delta_args", delta.DeltaArgs, {}), ("m3_delta_step_args", delta.DeltaStepArgs, {}),
               ("m3_delta_bwd_args", delta.DeltaBwdArgs, {"in_": "in"}), ("m3_pool", pool.PoolDesc, {}),
               ("m3_pool_copy_args", pool.PoolCopyArgs, {}), ("m3_pool_fork_args", pool.PoolForkArgs, {}),
               ("m3_pool_compact_args", pool.PoolCompactArgs, {})]
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "m3scan.h"', "int main(void){"]
    want = []
    for name, cls, other in structs:
        src.append('printf("%%zu\\n", sizeof(%s));' % name)
        want.append(ctypes.sizeof(cls))
        for f in cls._fields_:
            src.append('printf("%%zu\\n", offsetof(%s, %s));' % (name, other.get(f[0], f[0])))
            want.append(getattr(cls, f[0]).offset)
    src.append("return 0;}")
    c = tmp_path / "layout.c"
    c.write_text("\n".join(src))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(c)], check=True)
    out = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True, check=True).stdout
    assert [int(v) for v in out.split()] == want


def at(i):
    return FAKE + i * 4 * GIB


def fwd_args(**kw):
    a = delta.DeltaArgs(batch=2, seqlen=100, nheads=4, ngroups=2, headdim=64, dstate=64, io_dtype=1, l2norm=1,
                        scale=0.125, norm_eps=1e-6)
    for i, n in enumerate(("q", "k", "v", "g", "beta", "h_in", "o", "h_out")):
        setattr(a, n, at(i))
    a.workspace, a.workspace_bytes = at(20), 1 << 40
    for k, v in kw.items():
        setattr(a, k, v)
    return a


SIZES = [
    (dict(batch=-1), -2), (dict(seqlen=-1), -2), (dict(nheads=-4), -2), (dict(headdim=0), -2), (dict(dstate=0), -2),
    (dict(io_dtype=2), -4), (dict(io_dtype=-1), -4),
    (dict(dstate=16), -3), (dict(dstate=48), -3), (dict(dstate=256), -3), (dict(headdim=48), -3), (dict(headdim=160), -3),
    (dict(ngroups=3), -9), (dict(ngroups=-1), -9), (dict(l2norm=2), -9), (dict(l2norm=-1), -9),
    (dict(norm_eps=-1.0), -9), (dict(norm_eps=float("nan")), -9), (dict(norm_eps=float("inf")), -9),
    (dict(scale=float("nan")), -9), (dict(scale=float("inf")), -9),
    (dict(nheads=1 << 15, ngroups=0), -3), (dict(batch=1 << 25), -3), (dict(batch=1 << 14, nheads=1 << 14, ngroups=0), -3),
    (dict(seqlen=1 << 31), -3), (dict(batch=1 << 12, seqlen=1 << 16, nheads=16), -3),
]
POINTERS = [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(g=None), -1), (dict(beta=None), -1),
    (dict(q=at(0) + 8), -5), (dict(beta=at(4) + 4), -5), (dict(h_in=at(5) + 8), -5), (dict(cu_seqlens=at(9) + 2), -5),
    (dict(workspace=None), -6), (dict(workspace_bytes=1000), -6), (dict(workspace=at(20) + 16), -5),
    (dict(cu_seqlens=at(9), max_seqlen=101), -9), (dict(cu_seqlens=at(9), max_seqlen=-1), -9),
]


@pytest.mark.parametrize("kw,code", SIZES + POINTERS + [
    (dict(o=None), -1), (dict(o=at(6) + 2), -5), (dict(h_out=at(7) + 4), -5),
    (dict(o=at(2)), -7), (dict(o=at(0) + 64), -7), (dict(h_out=at(5) + 1024), -7), (dict(h_out=at(6)), -7),
    (dict(workspace=at(6)), -7), (dict(workspace=at(5)), -7),
    (dict(slots=at(9), nslots=-1), -9), (dict(slots=at(9) + 1, nslots=8), -5), (dict(slots=at(7) + 64, nslots=8), -7),
])
def test_prefill_refusals(lib, kw, code):
    assert lib.m3_delta_fwd(ctypes.byref(fwd_args(**kw)), None) == code


def test_null_arguments(lib):
    for fn in ("m3_delta_fwd", "m3_delta_step", "m3_delta_bwd", "m3_pool_copy", "m3_pool_fork", "m3_pool_compact"):
        assert getattr(lib, fn)(None, None) == -1
    for fn in ("m3_delta_workspace_bytes", "m3_delta_bwd_workspace_bytes", "m3_pool_copy_workspace_bytes"):
        assert getattr(lib, fn)(None) == 0


def test_nothing_to_do(lib):
    assert lib.m3_delta_fwd(ctypes.byref(delta.DeltaArgs(nheads=4, headdim=64, dstate=64, io_dtype=1)), None) == 0
    assert lib.m3_delta_step(ctypes.byref(delta.DeltaStepArgs(nheads=4, headdim=64, dstate=64, io_dtype=1)), None) == 0
    b = delta.DeltaBwdArgs()
    b.in_.nheads, b.in_.headdim, b.in_.dstate, b.in_.io_dtype = 4, 64, 64, 1
    assert lib.m3_delta_bwd(ctypes.byref(b), None) == 0


def test_workspace_sizes(lib):
    a = fwd_args()
    w = lib.m3_delta_workspace_bytes(ctypes.byref(a))
    assert w > 0 and w % 256 == 0
    assert lib.m3_delta_fwd(ctypes.byref(fwd_args(workspace_bytes=w - 1)), None) == -6
    assert lib.m3_delta_workspace_bytes(ctypes.byref(fwd_args(seqlen=200))) > w
    assert lib.m3_delta_workspace_bytes(ctypes.byref(fwd_args(dstate=48))) == 0
    assert lib.m3_delta_workspace_bytes(ctypes.byref(fwd_args(seqlen=0))) == 0
    # packed: grows with the tokens, not with sequences times the longest
    p1 = lib.m3_delta_workspace_bytes(ctypes.byref(fwd_args(batch=100, seqlen=6400, cu_seqlens=at(9), max_seqlen=64)))
    p2 = lib.m3_delta_workspace_bytes(ctypes.byref(fwd_args(batch=100, seqlen=6400, cu_seqlens=at(9), max_seqlen=6400)))
    assert p1 == p2 > 0


@pytest.mark.parametrize("kw,code", [(k, c) for k, c in SIZES if "seqlen" not in k] + [
    (dict(q=None), -1), (dict(h=None), -1), (dict(o=None), -1), (dict(k=at(1) + 8), -5), (dict(h=at(5) + 8), -5),
    (dict(o=at(2)), -7), (dict(o=at(5)), -7), (dict(h=at(0)), -7),
    (dict(slots=at(9), nslots=-1), -9), (dict(slots=at(5) + 64, nslots=8), -7), (dict(slots=at(9) + 2, nslots=8), -5)])
def test_step_refusals(lib, kw, code):
    a = delta.DeltaStepArgs(batch=2, nheads=4, ngroups=2, headdim=64, dstate=64, io_dtype=1, l2norm=1, scale=0.125, norm_eps=1e-6)
    for i, n in enumerate(("q", "k", "v", "g", "beta", "h", "o")):
        setattr(a, n, at(i))
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.m3_delta_step(ctypes.byref(a), None) == code


@pytest.mark.parametrize("kw,code", SIZES + POINTERS + [
    (dict(slots=at(9), nslots=8), -3), (dict(o=at(6)), -3), (dict(h_out=at(7)), -3),
    (dict(dout=None), -1), (dict(dq=None), -1), (dict(dbeta=None), -1), (dict(dv=at(25) + 8), -5), (dict(dh_in=at(29) + 8), -5),
    (dict(dq=at(0)), -7), (dict(dk=at(23) + 4096), -7), (dict(dh_in=at(5)), -7), (dict(workspace=at(25)), -7), (dict(dg=at(10)), -7)])
def test_gradient_refusals(lib, kw, code):
    b = delta.DeltaBwdArgs()
    for f in delta.DeltaArgs._fields_:
        setattr(b.in_, f[0], getattr(fwd_args(o=None, h_out=None), f[0]))
    for n, i in (("dout", 10), ("dh_out", 11), ("dq", 23), ("dk", 24), ("dv", 25), ("dg", 26), ("dbeta", 27), ("dh_in", 29)):
        setattr(b, n, at(i))
    for k, v in kw.items():
        setattr(b if hasattr(b, k) else b.in_, k, v)
    assert lib.m3_delta_bwd(ctypes.byref(b), None) == code


def desc(base, slots=8, rows=(1024, 512), **kw):
    d = pool.PoolDesc(slots=slots, narrays=len(rows))
    for i, r in enumerate(rows):
        d.data[i], d.row_bytes[i] = at(base + i), r
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def copy_args(src=None, dst=None, **kw):
    a = pool.PoolCopyArgs(src=src or desc(0), dst=dst or desc(2), src_slot=at(10), dst_slot=at(11), count=3)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def shifted(base, by):
    d = desc(base)
    d.data[0] = at(base) + by
    return d


@pytest.mark.parametrize("a,code", [
    (lambda: copy_args(src=desc(0, narrays=0)), -2), (lambda: copy_args(dst=desc(2, narrays=9)), -2),
    (lambda: copy_args(src=desc(0, slots=-1)), -2), (lambda: copy_args(count=-1), -2),
    (lambda: copy_args(src=desc(0, rows=(1024,))), -2), (lambda: copy_args(dst=desc(2, rows=(1024, 256))), -2),
    (lambda: copy_args(dst=desc(2, rows=(1024, 0))), -2),
    (lambda: copy_args(src=desc(0, slots=1 << 31)), -3), (lambda: copy_args(count=1 << 25), -3),
    (lambda: copy_args(src_slot=None), -1), (lambda: copy_args(dst_slot=None), -1),
    (lambda: copy_args(src_slot=at(10) + 2), -5), (lambda: copy_args(src=shifted(0, 8)), -5),
    (lambda: copy_args(dst=shifted(0, 4096)), -7),                            # overlaps src, but is not src
    (lambda: copy_args(src=desc(0), dst=desc(0, slots=4)), -7),               # the same arrays, another number of slots
    (lambda: copy_args(src=desc(0), dst=desc(0)), -6),                        # in place: needs a workspace
    (lambda: copy_args(src=desc(0), dst=desc(0), workspace=at(12), workspace_bytes=3 * 1536 - 1), -6),
    (lambda: copy_args(src=desc(0), dst=desc(0), workspace=at(12) + 8, workspace_bytes=1 << 20), -5),
    (lambda: copy_args(src=desc(0), dst=desc(0), workspace=at(0), workspace_bytes=1 << 20), -7),
    (lambda: copy_args(dst_slot=at(2) + 64), -7),
])
def test_copy_refusals(lib, a, code):
    assert lib.m3_pool_copy(ctypes.byref(a()), None) == code


def test_copy_workspace(lib):
    assert lib.m3_pool_copy_workspace_bytes(ctypes.byref(copy_args())) == 0
    assert lib.m3_pool_copy_workspace_bytes(ctypes.byref(copy_args(dst=desc(0)))) == 3 * 1536
    odd = desc(0, rows=(5, 18))
    assert lib.m3_pool_copy_workspace_bytes(ctypes.byref(copy_args(src=odd, dst=odd))) == 3 * (16 + 32)
    assert lib.m3_pool_copy(ctypes.byref(copy_args(count=0)), None) == 0


def fork_args(**kw):
    a = pool.PoolForkArgs(pool=desc(0), live=at(10), live_out=at(10), parents=at(11), children=at(12), count=3,
                          workspace=at(13), workspace_bytes=12)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(live=None), -1), (dict(live_out=None), -1), (dict(parents=None), -1), (dict(children=None), -1),
    (dict(count=-1), -2), (dict(count=1 << 25), -3), (dict(workspace=None), -6), (dict(workspace_bytes=11), -6),
    (dict(parents=at(11) + 1), -5), (dict(children=at(11)), -7), (dict(children=at(10)), -7), (dict(live_out=at(10) + 4), -7),
    (dict(live=at(0), live_out=at(0)), -7), (dict(workspace=at(12)), -7), (dict(parents=at(10)), -7)])
def test_fork_refusals(lib, kw, code):
    assert lib.m3_pool_fork(ctypes.byref(fork_args(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(live=None), -1), (dict(new_slot=None), -1), (dict(workspace=None), -6), (dict(workspace_bytes=35), -6),
    (dict(new_slot=at(10)), -7), (dict(count=at(12)), -7), (dict(live_out=at(10) + 4), -7), (dict(new_slot=at(1)), -7),
    (dict(count=at(14) + 2), -5), (dict(pool=desc(0, narrays=0)), -2)])
def test_compact_refusals(lib, kw, code):
    a = pool.PoolCompactArgs(pool=desc(0), live=at(10), live_out=at(10), new_slot=at(12), count=at(14), workspace=at(13),
                             workspace_bytes=36)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.m3_pool_compact(ctypes.byref(a), None) == code


def test_free_refusals(lib):
    assert lib.m3_pool_free(at(0), -1, at(1), 1, None) == -2
    assert lib.m3_pool_free(at(0), 4, at(1), -1, None) == -2
    assert lib.m3_pool_free(None, 4, at(1), 1, None) == -1
    assert lib.m3_pool_free(at(0), 4, None, 1, None) == -1
    assert lib.m3_pool_free(at(0), 4, at(0) + 4, 2, None) == -7
    assert lib.m3_pool_free(at(0), 4, at(1), 0, None) == 0


def test_binding_refusals():
    q = torch.zeros(1, 4, 2, 64)
    v = torch.zeros(1, 4, 3, 64)
    gb = torch.zeros(1, 4, 3)
    with pytest.raises(ValueError):
        m3_delta_fwd(q, q, v, gb, gb)                  # not on a device
    with pytest.raises(TypeError):
        m3_delta_fwd(q.half(), q.half(), v.half(), gb, gb)
    with pytest.raises(ValueError):
        m3_delta_fwd(q[0], q[0], v, gb, gb)
    with pytest.raises(ValueError):
        m3_delta_step(q, q, v, gb, gb, torch.zeros(1, 3, 64, 64))
    with pytest.raises(ValueError):
        m3_pool_copy((q,), (q,), torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        m3_pool_copy((), (), torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        m3_pool_free(torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_workspace_of_long_packed_calls(lib):
    """One that a call with a long max_seqlen takes is what one with a short max_seqlen asks for."""
    kw = dict(batch=1, nheads=2, ngroups=2, seqlen=1 << 15, cu_seqlens=at(9))
    for f in (lambda a: lib.m3_delta_workspace_bytes(ctypes.byref(a)),
              lambda a: lib.m3_delta_bwd_workspace_bytes(ctypes.byref(delta.DeltaBwdArgs(in_=a)))):
        need = [f(fwd_args(max_seqlen=n, **kw)) for n in (0, 1, 64, 16383, 16385, 1 << 15)]
        assert min(need) == max(need) > 0


LAUNCH = [   # launches count their threads in 32 bits: the first size that does not fit, and the last that does
    ("fwd", dict(nheads=1 << 10, ngroups=0, headdim=128), "batch", (((1 << 32) - 1) // 448 // 8) // (1 << 10) + 1),
    ("bwd", dict(nheads=1 << 10, ngroups=0, headdim=128), "batch", (((1 << 32) - 1) // 640 // 8) // (1 << 10) + 1),
    ("bwd", dict(nheads=1, ngroups=0, dstate=32, cu_seqlens=at(9), max_seqlen=64), "seqlen", (1 << 29) - 31),
    ("fwd", dict(cu_seqlens=at(9), max_seqlen=64), "seqlen", (1 << 38) + 1),
]


@pytest.mark.parametrize("what,kw,name,first", LAUNCH)
def test_sizes_beyond_a_launch(lib, what, kw, name, first):
    def need(n):
        a = fwd_args(**{**kw, name: n})
        if what == "fwd":
            return lib.m3_delta_workspace_bytes(ctypes.byref(a)), lib.m3_delta_fwd(ctypes.byref(a), None)
        b = delta.DeltaBwdArgs()
        a.o = a.h_out = None
        b.in_ = a
        return lib.m3_delta_bwd_workspace_bytes(ctypes.byref(b)), lib.m3_delta_bwd(ctypes.byref(b), None)

    assert need(first) == (0, -3)
    b, st = need(first - 1)
    assert b > 0 and st != -3


def test_step_beyond_a_launch(lib):
    a = delta.DeltaStepArgs(batch=1 << 12, nheads=1 << 12, headdim=128, dstate=32, io_dtype=1, scale=1.0)
    assert lib.m3_delta_step(ctypes.byref(a), None) == -3
    a.batch -= 1
    assert lib.m3_delta_step(ctypes.byref(a), None) == -1   # fits: its null pointers are next


def test_pools_beyond_address_arithmetic(lib):
    """slots x row bytes of one array is bounded, so that no product of the checks wraps."""
    d = desc(0, slots=1 << 30, rows=(1 << 33, 512))
    a = copy_args(src=d, dst=desc(2, slots=1 << 30, rows=(1 << 33, 512)))
    assert lib.m3_pool_copy(ctypes.byref(a), None) == -3
    assert lib.m3_pool_free(at(0), 4, at(8), (1 << 32) - 255, None) == -3
