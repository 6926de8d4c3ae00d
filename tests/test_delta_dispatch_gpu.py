"""The gated delta rule's prefill on both sides of each choice of its walk.

A slice is 16 columns of one row and head.  bf16 calls with at most 256 slices
take one slice to a workgroup; with more, 32 columns; above 512 slices 64
columns where headdim is a multiple of 64.  Tolerances: test_delta_gpu.py's.
"""
import pytest
import torch

import delta_reference as ref
from helpers import say
from mamba_selective_ssm_amd import m3_delta_fwd
from test_delta_gpu import check_h, check_o

pytestmark = pytest.mark.gpu

# (N, P, heads of one row): slices = heads * P / 16
SIZES = [(N, P, s * 16 // P) for N in (32, 64, 128) for P, slices in (
    (32, (256, 258, 512, 514)), (64, (256, 260, 512, 516)), (96, (252, 258, 510, 516)), (128, (256, 264, 512, 520)))
    for s in slices]


@pytest.mark.parametrize("N,P,H", SIZES)
def test_dense(N, P, H):
    """Two chunks, the second ragged, from a given state."""
    say("case dispatch", N, P, H, "slices", H * P // 16)
    x = ref.inputs(1, 75, H, H if H % 2 else H // 2, N, P, torch.bfloat16, 301)
    h = torch.randn(1, H, N, P, generator=torch.Generator().manual_seed(302)).cuda()
    wo, wh = ref.forward(*x, h, scale=0.2, l2norm=True)
    o, hL = m3_delta_fwd(*x, h, l2norm=True, scale=0.2)
    check_o(o, wo, "bf16", "dense")
    check_h(hL, wh, "dense")


@pytest.mark.parametrize("N,P,H", [(32, 64, 20), (64, 64, 20), (64, 128, 11), (64, 96, 13), (128, 32, 40), (128, 64, 20), (128, 96, 13),
                                   (128, 128, 10)])
def test_packed_into_slots_with_32_columns(N, P, H):
    """257 to 512 slices in packed rows of unlike lengths, an empty one and one without a record among them, the pool's other
    slots and the tokens behind the last row as they were."""
    lens, slots = [130, 1, 64, 0, 191], [3, 0, -1, 5, 1]
    say("case packed", N, P, H, "slices", len(lens) * H * P // 16)
    assert 256 < len(lens) * H * P // 16 <= 512
    T = sum(lens) + 5
    x = ref.inputs(1, T, H, H, N, P, torch.bfloat16, 311)
    pool = torch.randn(6, H, N, P, generator=torch.Generator().manual_seed(312)).cuda()
    before = pool.clone()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    o = torch.full((1, T, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    m3_delta_fwd(*x, pool, l2norm=True, scale=0.2, cu_seqlens=cu, max_seqlen=191, o=o,
                 slots=torch.tensor(slots, dtype=torch.int32).cuda())
    at = 0
    for i, (n, s) in enumerate(zip(lens, slots)):
        part = slice(at, at + n)
        wo, wh = ref.forward(*(t[:, part] for t in x), before[s:s + 1] if s >= 0 else None, scale=0.2, l2norm=True)
        if n:
            check_o(o[:, part], wo, "bf16", "row %d" % i)
        if s >= 0:
            check_h(pool[s:s + 1], wh, "row %d" % i)
        at += n
    assert bool((o[:, at:] == 7.0).all())
    for s in (2, 4):
        assert torch.equal(pool[s], before[s])
