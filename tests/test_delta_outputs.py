"""Every output of the gated delta rule's gradient is written: outputs that
hold NaN before the call, in calls without heads."""
import ctypes

import pytest
import torch

from mamba_selective_ssm_amd import binding, delta, m3_delta_bwd

FAKE = 0x7F0000000000
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh_in")


def call(x, do, h=None, dh=None, cu=None, max_seqlen=0, scale=0.2, rows=None):
    """m3_delta_bwd into outputs full of NaN.  Returns them by name."""
    lib = binding.load_library()
    (B, L, G, N), (H, P) = x[0].shape, x[2].shape[2:]
    rows = B if cu is None else cu.numel() - 1
    out = {n: torch.full(t.shape, float("nan"), device="cuda") for n, t in zip(NAMES, x)}
    out["dh_in"] = torch.full((rows, H, N, P), float("nan"), device="cuda")
    a = delta.DeltaArgs(batch=rows, seqlen=L, nheads=H, ngroups=G, headdim=P, dstate=N, io_dtype=1 if x[0].dtype == torch.bfloat16 else 0,
                        l2norm=1, scale=scale, norm_eps=1e-6, max_seqlen=max_seqlen)
    for n, t in zip(("q", "k", "v", "g", "beta", "h_in", "cu_seqlens"), x + [h, cu]):
        setattr(a, n, 0 if t is None else t.data_ptr())
    b = delta.DeltaBwdArgs(in_=a, dout=do.data_ptr(), dh_out=0 if dh is None else dh.data_ptr())
    for n, t in out.items():
        setattr(b, n, t.data_ptr())
    need = lib.m3_delta_bwd_workspace_bytes(ctypes.byref(b))
    ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")   # NaN as float32 too
    b.in_.workspace, b.in_.workspace_bytes = ws.data_ptr(), need
    assert lib.m3_delta_bwd(ctypes.byref(b), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("io", [torch.bfloat16, torch.float32])
def test_groups_without_heads(packed, io):
    """No head reads q and k: their gradients are zero."""
    G, N, P, T = 2, 64, 32, 70
    q = torch.randn(1, T, G, N, device="cuda").to(io)
    v, gb = torch.empty(1, T, 0, P, dtype=io, device="cuda"), torch.empty(1, T, 0, device="cuda")
    cu = torch.tensor([0, 30, 60], dtype=torch.int32, device="cuda") if packed else None
    got = call([q, q.clone(), v, gb, gb.clone()], v.clone(), cu=cu, max_seqlen=30)
    assert bool((got["dq"] == 0).all()) and bool((got["dk"] == 0).all())
    r = m3_delta_bwd(q, q.clone(), v, gb, gb.clone(), v.clone(), cu_seqlens=cu)
    assert bool((r.dq == 0).all()) and bool((r.dk == 0).all()) and r.dq.shape == q.shape


def test_groups_without_heads_need_their_outputs():
    """Refusals on the CPU: dq and dk of such a call are outputs like any other."""
    lib = binding.load_library()
    a = delta.DeltaArgs(batch=1, seqlen=70, nheads=0, ngroups=2, headdim=32, dstate=64, io_dtype=1, l2norm=1, scale=1.0, norm_eps=1e-6,
                        q=FAKE, k=FAKE + (1 << 30))
    full = dict(dq=FAKE + (2 << 30), dk=FAKE + (3 << 30))
    for kw, code in ((dict(dq=0), -1), (dict(dk=0), -1), (dict(dq=FAKE + (2 << 30) + 8), -5), (dict(dq=FAKE), -7),
                     (dict(dk=full["dq"] + 64), -7)):
        b = delta.DeltaBwdArgs(in_=a, **{**full, **kw})
        assert lib.m3_delta_bwd(ctypes.byref(b), None) == code
    # sums that a launch cannot count, groups whose sizes would not fit
    a.ngroups = 1 << 60
    assert lib.m3_delta_bwd(ctypes.byref(delta.DeltaBwdArgs(in_=a, **full)), None) == -3
    a.ngroups = 2
    a.seqlen = 1 << 30
    a.batch = 1 << 8
    assert lib.m3_delta_bwd(ctypes.byref(delta.DeltaBwdArgs(in_=a, **full)), None) == -3
