"""Every output of the gated delta rule's gradient is written: outputs that
hold NaN before the call, tokens outside every sequence, rows longer than
max_seqlen, and calls without heads."""
import ctypes

import pytest
import torch

import delta_reference as ref
from helpers import say
from mamba_selective_ssm_amd import binding, delta, m3_delta_bwd

FAKE = 0x7F0000000000
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh_in")
TOL = 2e-5   # as in test_delta_bwd_gpu.py


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
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N,P,H,G", [(64, 64, 4, 4), (64, 64, 4, 2), (32, 96, 3, 1), (128, 32, 2, 2)])
def test_tokens_outside_every_sequence(io, N, P, H, G):
    """Gaps before the first sequence and behind the last, an empty sequence, one longer than max_seqlen: exact zeros there, the
    gradients of the rest as if each sequence ended at max_seqlen."""
    say("case outside", io, N, P, H, G)
    at, T, longest = [13, 18, 18, 82, 200, 263], 280, 100   # lengths 5, 0, 64, 118 (100 of them taken), 63
    x = ref.inputs(1, T, H, G, N, P, torch.bfloat16 if io == "bf16" else torch.float32, 321)
    gen = torch.Generator().manual_seed(322)
    do = torch.randn(1, T, H, P, generator=gen).to(x[0].dtype).cuda()
    h, dh = (torch.randn(5, H, N, P, generator=gen).cuda() for _ in range(2))
    got = call(x, do, h, dh, torch.tensor(at, dtype=torch.int32).cuda(), longest)
    rest = torch.ones(T, dtype=torch.bool)
    for i in range(5):
        part = slice(at[i], min(at[i + 1], at[i] + longest))
        rest[part] = False
        want = ref.backward(*(t[:, part] for t in x), do[:, part], h[i:i + 1], dh[i:i + 1], scale=0.2, l2norm=True)
        for n in NAMES:
            g = got[n][i:i + 1] if n == "dh_in" else got[n][:, part]
            assert bool(g.isfinite().all()), (n, i)
            assert ref.rel2(g, want[n]) <= TOL, (n, i)
    for n in NAMES[:5]:
        assert bool((got[n][:, rest.cuda()] == 0).all()), n


@pytest.mark.gpu
@pytest.mark.parametrize("G", [1, 3])
def test_dense_outputs_and_no_sequences(G):
    H, N, P = 3, 64, 32
    x = ref.inputs(2, 70, H, G, N, P, torch.bfloat16, 331)
    do = torch.randn(2, 70, H, P, generator=torch.Generator().manual_seed(332)).to(torch.bfloat16).cuda()
    got = call(x, do)
    want = ref.backward(*x, do, scale=0.2, l2norm=True)
    for n in NAMES:
        assert ref.rel2(got[n], want[n]) <= TOL, n
    # one offset: no sequence at all
    y = [t[:1].contiguous() for t in x]
    got = call(y, do[:1].contiguous(), cu=torch.zeros(1, dtype=torch.int32, device="cuda"), max_seqlen=70)
    for n in NAMES[:5]:
        assert bool((got[n] == 0).all()), n


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
