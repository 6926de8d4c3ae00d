"""Packed calls of the gated delta rule whose max_seqlen is far above every
length, as the default one (all tokens) is: they are taken, and their results
are those of the tight bound."""
import ctypes

import pytest
import torch

import delta_reference as ref
from helpers import say
from mamba_selective_ssm_amd import binding, delta, m3_delta_bwd, m3_delta_fwd
from test_delta_gpu import check_h, check_o

FAKE = 0x7F0000000000


@pytest.mark.parametrize("train", [False, True])
def test_many_rows_are_not_refused(train):
    """1024 sequences, 65536 tokens, 32 heads: as chunks of 65536 tokens each they would be 2^25 workgroups."""
    lib = binding.load_library()

    def need(longest, seqlen=65536, batch=1024, heads=32):
        a = delta.DeltaArgs(batch=batch, seqlen=seqlen, nheads=heads, headdim=64, dstate=64, io_dtype=1, l2norm=1, scale=1.0,
                            norm_eps=1e-6, cu_seqlens=FAKE, max_seqlen=longest)
        if train:
            return lib.m3_delta_bwd_workspace_bytes(ctypes.byref(delta.DeltaBwdArgs(in_=a)))
        return lib.m3_delta_workspace_bytes(ctypes.byref(a))

    assert need(65536) == need(64) > 0
    # the bound that is left: (seqlen / 64 + batch + 1) * heads < 2^24
    if not train:   # (the gradient has one of its own: tokens * ngroups * dstate)
        assert need(1 << 24, (1 << 25) - 64 * 2, 1, 32) > 0
    assert need(1 << 25, 1 << 25, 1024, 32) == 0


def rows(lens, gap=0):
    return torch.tensor([gap] + lens).cumsum(0).to(torch.int32).cuda()


CASES = [
    # lengths, H, G, N, P, io: rows a slot apart and many slots apart, empty ones at the ends and in a row
    ([3, 0, 64, 0, 0, 65, 1, 200, 128, 0], 4, 2, 64, 64, "bf16"),
    ([0, 0, 130, 5, 0], 3, 3, 128, 32, "f32"),
    ([63, 1] * 20, 2, 1, 32, 96, "bf16"),
    ([40, 0, 25] * 30 + [700], 30, 10, 64, 64, "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,G,N,P,io", CASES)
def test_results_do_not_depend_on_the_bound(lens, H, G, N, P, io):
    say("case bounds", len(lens), sum(lens), H, G, N, P, io)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    gap = 70                       # tokens before the first sequence and behind the last
    T = gap + sum(lens) + 30
    cu = rows(lens, gap)
    # more chunks by the default bound than twice the slots
    assert len(lens) * ((T + 63) // 64) > 2 * (T // 64 + len(lens) + 1)
    x = ref.inputs(1, T, H, G, N, P, dt, 401)
    gen = torch.Generator().manual_seed(402)
    h, dh = (torch.randn(len(lens), H, N, P, generator=gen).cuda() for _ in range(2))
    do = torch.randn(1, T, H, P, generator=gen).to(dt).cuda()
    outs = []
    for longest in (None, T, max(lens)):
        o = torch.full((1, T, H, P), 7.0, dtype=dt, device="cuda")
        o, hl = m3_delta_fwd(*x, h, l2norm=True, scale=0.3, cu_seqlens=cu, max_seqlen=longest, o=o)
        outs.append((o, hl, *m3_delta_bwd(*x, do, h, dh, l2norm=True, scale=0.3, cu_seqlens=cu, max_seqlen=longest)))
    for other in outs[:2]:
        for a, b in zip(other, outs[2]):
            assert torch.equal(a, b)
    part = [t[:, gap:gap + sum(lens)] for t in x]
    want = ref.packed(ref.forward, lens, part, [h], scale=0.3, l2norm=True)
    check_o(outs[0][0][:, gap:gap + sum(lens)], torch.cat([w[0] for w in want], 1), io, "default bound")
    check_h(outs[0][1], torch.cat([w[1] for w in want]), "default bound")
    assert bool((outs[0][0][:, :gap] == 7.0).all()) and bool((outs[0][0][:, gap + sum(lens):] == 7.0).all())


@pytest.mark.gpu
def test_many_rows_with_the_default_bound():
    """More rows and heads than a launch over rows times chunks could have, rows of 0 to 64 tokens, into a pool's slots."""
    n, H, N, P = 1200, 32, 32, 32
    gen = torch.Generator().manual_seed(411)
    lens = torch.randint(0, 65, (n,), generator=gen)
    T = int(lens.sum())
    assert n * H * ((T + 63) // 64) > 1 << 24
    cu = rows(lens.tolist())
    x = ref.inputs(1, T, H, 1, N, P, torch.bfloat16, 412)
    pool = torch.randn(n + 3, H, N, P, generator=gen).cuda()
    slots = torch.randperm(n + 3, generator=gen)[:n].to(torch.int32)
    got, tight = pool.clone(), pool.clone()
    o, _ = m3_delta_fwd(*x, got, l2norm=True, cu_seqlens=cu, slots=slots.cuda())
    want, _ = m3_delta_fwd(*x, tight, l2norm=True, cu_seqlens=cu, max_seqlen=64, slots=slots.cuda())
    assert torch.equal(o, want) and torch.equal(got, tight)
    at = cu.tolist()
    for i in (0, 1, 2, n // 2, n - 2, n - 1):
        part = slice(at[i], at[i + 1])
        s = int(slots[i])
        if at[i] == at[i + 1]:
            assert torch.equal(got[s], pool[s])
            continue
        wo, wh = ref.forward(*(t[:, part] for t in x), pool[s:s + 1], scale=N ** -0.5, l2norm=True)
        check_o(o[:, part], wo, "bf16", "row %d" % i)
        check_h(got[s:s + 1], wh, "row %d" % i)
