"""The gated delta rule on the GPU: prefill and one-token step against the
float64 recurrence, over types, sizes, lengths, packed sequences, pool slots
and the values where it can go wrong.

Tolerances.  Operands are held to 24 bits (three bf16 planes, or float32) and
sums to float32, so a state differs from the exact one by the roundings of its
sums: at most N + 3 * 64 <= 320 terms in a chunk's three products, each 2^-24
of the sum so far, 1.9e-5 together if all fell the same way; what earlier
chunks left decays with the state.  Outputs in bf16 carry two planes (2^-16 a
value) on their own path, below that, and one rounding of at most 2^-8 of the
value.
"""
import pytest
import torch

import delta_reference as ref
from helpers import say
from mamba_selective_ssm_amd import (M3Error, m3_delta_fwd, m3_delta_step, m3_delta_supported)

pytestmark = pytest.mark.gpu
F32_TOL = 320 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def check_o(o, want, io, label):
    e = ref.rel2(o, want)
    if io == "f32":
        say("   %s: o %.2e" % (label, e))
        assert e <= F32_TOL
        return
    off = (o.double().cpu() - want).abs()
    rms = float(want.pow(2).mean().sqrt())
    # one rounding, plus the path's own error against the size of its terms
    room = 2.0 ** -8 * want.abs() + 2.0 ** -12 * rms
    say("   %s: o %.2e, worst %.2f of the room" % (label, e, float((off / room).max()) if off.numel() else 0))
    assert bool((off <= room).all())


def check_h(h, want, label):
    e = ref.rel2(h, want)
    say("   %s: h %.2e" % (label, e))
    assert e <= F32_TOL


CASES = [
    # B, L, H, G, N, P, io, l2norm
    (1, 1, 1, 1, 64, 64, "bf16", True),
    (1, 1, 2, 1, 32, 32, "f32", True),
    (2, 15, 3, 3, 64, 32, "bf16", True),
    (1, 16, 2, 2, 128, 64, "bf16", False),
    (1, 17, 2, 2, 128, 96, "f32", True),
    (1, 63, 2, 1, 64, 64, "bf16", True),
    (2, 64, 4, 2, 64, 64, "f32", False),
    (1, 65, 9, 3, 32, 96, "bf16", True),
    (1, 127, 2, 2, 128, 128, "bf16", True),
    (1, 200, 1, 1, 128, 128, "f32", True),
    (3, 321, 5, 1, 64, 64, "bf16", False),
    (1, 1000, 2, 2, 64, 64, "bf16", True),
    (1, 700, 2, 1, 32, 64, "f32", True),
]


@pytest.mark.parametrize("B,L,H,G,N,P,io,l2", CASES)
def test_prefill(B, L, H, G, N, P, io, l2):
    say("case prefill", B, L, H, G, N, P, io, l2)
    x = ref.inputs(B, L, H, G, N, P, DT[io], 11, raw=not l2)
    h = torch.randn(B, H, N, P, generator=torch.Generator().manual_seed(12)).cuda()
    for h0 in (None, h):
        o, hL = m3_delta_fwd(*x, h0, l2norm=l2, scale=0.25)
        wo, wh = ref.forward(*x, h0, scale=0.25, l2norm=l2)
        check_o(o, wo, io, "zero state" if h0 is None else "given state")
        check_h(hL, wh, "zero state" if h0 is None else "given state")


@pytest.mark.parametrize("N,P", [(32, 32), (32, 64), (64, 96), (64, 64), (128, 64), (128, 128)])
def test_many_heads(N, P):
    """More (row, head, 16 columns) than CUs; packed sequences of all lengths
    around a chunk's, in a pool, some without a record, one slot named twice."""
    H = 4600 // P
    lens = [1, 130, 64, 0, 63, 200, 17, 65]
    x = ref.inputs(1, sum(lens), H, H, N, P, torch.bfloat16, 15)
    pool = torch.randn(9, H, N, P, generator=torch.Generator().manual_seed(16)).cuda()
    before = pool.clone()
    sl = torch.tensor([8, 0, 3, 5, -1, 2, 0, 6], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    assert len(lens) * H * P // 16 > 256
    o, _ = m3_delta_fwd(*x, pool, l2norm=True, scale=0.2, cu_seqlens=cu, max_seqlen=200, slots=sl)
    start = torch.stack([before[s] if s >= 0 else torch.zeros_like(before[0]) for s in sl.tolist()])
    want = ref.packed(ref.forward, lens, x, [start], scale=0.2, l2norm=True)
    at = 0
    for i, n in enumerate(lens):
        if i == 6:
            assert bool(o[:, at:at + n].isnan().all())
        elif n:
            check_o(o[:, at:at + n], want[i][0], "bf16", "row %d" % i)
        if i not in (4, 6):
            check_h(pool[sl[i].item()][None], want[i][1], "row %d" % i)
        at += n
    for s in (1, 4, 7):
        assert torch.equal(pool[s], before[s])
    # a dense batch without a state, one row longer than the others would be
    y = ref.inputs(8, 70, H, 1, N, P, torch.bfloat16, 17)
    o, h = m3_delta_fwd(*y, l2norm=True, scale=0.2)
    wo, wh = ref.forward(*y, scale=0.2, l2norm=True)
    check_o(o, wo, "bf16", "dense")
    check_h(h, wh, "dense")


def test_default_scale_and_no_state():
    x = ref.inputs(1, 70, 2, 2, 64, 32, torch.bfloat16, 21)
    o, h = m3_delta_fwd(*x, l2norm=True, return_state=False)
    assert h is None
    wo, _ = ref.forward(*x, scale=64 ** -0.5, l2norm=True)
    check_o(o, wo, "bf16", "default scale")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_split_into_calls_and_steps(io):
    """Prefill, prefill in place, then single tokens: one sequence."""
    B, L, H, G, N, P = 2, 150, 4, 2, 64, 64
    x = ref.inputs(B, L, H, G, N, P, DT[io], 31)
    wo, wh = ref.forward(*x, scale=0.125, l2norm=True)
    cut = [t[:, :77].contiguous() for t in x], [t[:, 77:147].contiguous() for t in x]
    o1, h = m3_delta_fwd(*cut[0], l2norm=True, scale=0.125)
    o2, h2 = m3_delta_fwd(*cut[1], h, l2norm=True, scale=0.125, h_out=h)
    assert h2 is h
    steps = [m3_delta_step(*[t[:, i].contiguous() for t in x], h, l2norm=True, scale=0.125) for i in range(147, 150)]
    check_o(torch.cat([o1, o2, torch.stack(steps, 1)], 1), wo, io, "split")
    check_h(h, wh, "split")


@pytest.mark.parametrize("io,N,P,H,G", [("bf16", 64, 64, 4, 4), ("f32", 32, 96, 6, 2), ("bf16", 128, 128, 3, 1)])
def test_packed_sequences(io, N, P, H, G):
    """Ragged lengths, empty sequences among them; tokens behind the last are left as they were."""
    lens = [5, 0, 64, 1, 130, 0, 63, 65]
    T = sum(lens) + 9
    x = ref.inputs(1, T, H, G, N, P, DT[io], 41)
    h = torch.randn(len(lens), H, N, P, generator=torch.Generator().manual_seed(42)).cuda()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    o = torch.full((1, T, H, P), 7.0, dtype=DT[io], device="cuda")
    o, hL = m3_delta_fwd(*x, h, l2norm=True, scale=0.2, cu_seqlens=cu, max_seqlen=130, o=o)
    want = ref.packed(ref.forward, lens, x, [h], scale=0.2, l2norm=True)
    check_o(o[:, :sum(lens)], torch.cat([w[0] for w in want], 1), io, "packed")
    check_h(hL, torch.cat([w[1] for w in want]), "packed")
    assert bool((o[:, sum(lens):] == 7.0).all())
    for i, n in enumerate(lens):
        if n == 0:
            assert torch.equal(hL[i], h[i])
    # the longest length as an upper bound only
    o2, h2 = m3_delta_fwd(*x, h, l2norm=True, scale=0.2, cu_seqlens=cu)
    assert torch.equal(o2[:, :sum(lens)], o[:, :sum(lens)]) and torch.equal(h2, hL)


def test_slots_of_a_pool():
    """Records read from and written to a pool's slots; a slot outside it (no
    record) and one named twice (the first row has it)."""
    H, N, P, slots = 3, 64, 64, 9
    lens = [40, 70, 3, 20, 11]
    x = ref.inputs(1, sum(lens), H, H, N, P, torch.bfloat16, 51)
    pool = torch.randn(slots, H, N, P, generator=torch.Generator().manual_seed(52)).cuda()
    before = pool.clone()
    sl = torch.tensor([4, 0, -1, 7, 0], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    o, h = m3_delta_fwd(*x, pool, l2norm=True, scale=0.2, cu_seqlens=cu, slots=sl)
    assert h is pool
    start = torch.stack([before[4], before[0], torch.zeros_like(before[0]), before[7], before[0]])
    want = ref.packed(ref.forward, lens, x, [start], scale=0.2, l2norm=True)
    at = 0
    for i, n in enumerate(lens):
        if i == 4:
            assert bool(o[:, at:at + n].isnan().all())
        else:
            check_o(o[:, at:at + n], want[i][0], "bf16", "row %d" % i)
        at += n
    for i, s in ((0, 4), (1, 0), (3, 7)):
        check_h(pool[s:s + 1], want[i][1], "slot %d" % s)
    for s in (1, 2, 3, 5, 6, 8):
        assert torch.equal(pool[s], before[s])


@pytest.mark.parametrize("B,H,G,N,P,io,l2", [(1, 1, 1, 64, 64, "bf16", True), (3, 6, 2, 32, 32, "f32", True),
                                             (5, 4, 4, 128, 96, "bf16", False), (70, 3, 1, 128, 128, "f32", False),
                                             (33, 8, 2, 64, 128, "bf16", True)])
def test_step(B, H, G, N, P, io, l2):
    say("case step", B, H, G, N, P, io, l2)
    x = ref.inputs(B, 1, H, G, N, P, DT[io], 61, step=True, raw=not l2)
    h = torch.randn(B, H, N, P, generator=torch.Generator().manual_seed(62)).cuda()
    wo, wh = ref.forward(*[t[:, None] for t in x], h, scale=0.3, l2norm=l2)
    o = m3_delta_step(*x, h, l2norm=l2, scale=0.3)
    check_o(o, wo[:, 0], io, "step")
    check_h(h, wh, "step")


def test_step_slots():
    B, H, N, P, slots = 6, 2, 64, 64, 8
    x = ref.inputs(B, 1, H, H, N, P, torch.bfloat16, 71, step=True)
    pool = torch.randn(slots, H, N, P, generator=torch.Generator().manual_seed(72)).cuda()
    before = pool.clone()
    sl = torch.tensor([3, -1, 5, 3, 0, 8], dtype=torch.int32, device="cuda")
    o = m3_delta_step(*x, pool, l2norm=True, scale=0.3, slots=sl)
    zero = torch.zeros_like(before[0])
    start = torch.stack([before[3], zero, before[5], zero, before[0], zero])
    wo, wh = ref.forward(*[t[:, None] for t in x], start, scale=0.3, l2norm=True)
    real = [0, 1, 2, 4, 5]
    check_o(o[real], wo[real, 0], "bf16", "rows")
    assert bool(o[3].isnan().all())
    for i, s in ((0, 3), (2, 5), (4, 0)):
        check_h(pool[s], wh[i], "slot %d" % s)
    for s in (1, 2, 4, 6, 7):
        assert torch.equal(pool[s], before[s])


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decays_that_forget(io):
    """Log decays of -inf, of -1e30 and of hundreds of runs between them: what
    comes after a reset keeps its accuracy."""
    x = ref.inputs(1, 190, 2, 2, 64, 32, DT[io], 81)
    g = x[3]
    g[:, 10] = -float("inf")
    g[:, 50:60] = -300.0
    g[:, 64] = -1e30
    g[:, 100:128:2] = -1000.0
    g[:, 150] = 0.0
    h = torch.randn(1, 2, 64, 32, generator=torch.Generator().manual_seed(82)).cuda()
    o, hL = m3_delta_fwd(*x, h, l2norm=True, scale=1.0)
    wo, wh = ref.forward(*x, h, scale=1.0, l2norm=True)
    check_o(o, wo, io, "resets")
    check_h(hL, wh, "resets")


def test_repeated_keys():
    """One key in every token, write strength 1, no decay: the inverse of a
    triangle full of ones."""
    x = ref.inputs(1, 150, 1, 1, 64, 32, torch.float32, 91)
    x[1][:] = x[1][:, :1].clone()
    x[3].zero_()
    x[4].fill_(1.0)
    o, h = m3_delta_fwd(*x, l2norm=True, scale=1.0)
    wo, wh = ref.forward(*x, scale=1.0, l2norm=True)
    check_o(o, wo, "f32", "repeated keys")
    check_h(h, wh, "repeated keys")


def test_zero_rows_and_no_writes():
    """Rows of zeros (their norm is eps alone) and write strength 0."""
    x = ref.inputs(1, 100, 2, 1, 64, 64, torch.bfloat16, 101)
    x[0][:, 7] = 0
    x[1][:, 9:30] = 0
    x[4][:, 40:80] = 0
    o, h = m3_delta_fwd(*x, l2norm=True, scale=1.0)
    wo, wh = ref.forward(*x, scale=1.0, l2norm=True)
    check_o(o, wo, "bf16", "zero rows")
    check_h(h, wh, "zero rows")


def test_nan_stays_in_its_row_and_head():
    x = ref.inputs(2, 130, 3, 3, 64, 64, torch.bfloat16, 111)
    clean, _ = m3_delta_fwd(*x, l2norm=True)
    x[2][1, 70, 1, 5] = float("nan")
    o, h = m3_delta_fwd(*x, l2norm=True)
    bad = o.isnan()
    assert bool(bad[1, 70:, 1].any()) and bool(h[1, 1].isnan().any())
    assert torch.equal(o[0], clean[0]) and torch.equal(o[1, :, [0, 2]], clean[1, :, [0, 2]])
    assert torch.equal(o[1, :64, 1], clean[1, :64, 1])


def test_large_and_small_values():
    """States far from 1: nothing on the way has a narrower range than float32."""
    for size in (1e12, 1e-12):
        x = ref.inputs(1, 150, 2, 2, 64, 64, torch.float32, 121)
        x[2] *= size
        o, h = m3_delta_fwd(*x, l2norm=True, scale=1.0)
        wo, wh = ref.forward(*x, scale=1.0, l2norm=True)
        check_o(o, wo, "f32", "size %g" % size)
        check_h(h, wh, "size %g" % size)


def test_empty_calls():
    x = ref.inputs(2, 0, 3, 3, 64, 64, torch.bfloat16, 131)
    h = torch.randn(2, 3, 64, 64, device="cuda")
    o, hL = m3_delta_fwd(*x, h)
    assert o.shape == (2, 0, 3, 64) and torch.equal(hL, h)
    _, hL = m3_delta_fwd(*x)
    assert bool((hL == 0).all())
    x = ref.inputs(0, 5, 3, 3, 64, 64, torch.bfloat16, 132)
    o, hL = m3_delta_fwd(*x)
    assert o.shape[0] == 0 and hL.shape[0] == 0


def test_same_results_every_time_and_other_streams():
    x = ref.inputs(2, 500, 4, 2, 64, 64, torch.bfloat16, 141)
    first = m3_delta_fwd(*x, l2norm=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [m3_delta_fwd(*x, l2norm=True, stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for o, h in got:
        assert torch.equal(o, first[0]) and torch.equal(h, first[1])


def test_captured_and_replayed():
    """Prefill into a pool and steps on it, captured; replayed on other inputs."""
    B, L, H, N, P = 2, 100, 4, 64, 64
    x = ref.inputs(B, L, H, H, N, P, torch.bfloat16, 151)
    y = ref.inputs(B, 1, H, H, N, P, torch.bfloat16, 152, step=True)
    sl = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    pool = torch.zeros(4, H, N, P, device="cuda")
    run = lambda: (m3_delta_fwd(*x, pool, l2norm=True, slots=sl)[0], m3_delta_step(*y, pool, l2norm=True, slots=sl))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for seed in (153, 154, 155):
        for dst, src in zip(x + y, ref.inputs(B, L, H, H, N, P, torch.bfloat16, seed)
                            + ref.inputs(B, 1, H, H, N, P, torch.bfloat16, seed + 50, step=True)):
            dst.copy_(src)
        start = torch.randn(4, H, N, P, generator=torch.Generator().manual_seed(seed)).cuda()
        pool.copy_(start)
        want = [t.clone() for t in run()]
        end = pool.clone()
        pool.copy_(start)
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool, end)
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_long_offsets():
    """A pool whose last record starts past 2^31 bytes and 2^31 / 4 values."""
    H, N, P = 32, 128, 128
    slots = 1100   # 2 MiB a record
    pool = torch.empty(slots, H, N, P, device="cuda")
    pool[slots - 1].normal_()
    start = pool[slots - 1].clone()
    x = ref.inputs(1, 1, H, 1, N, P, torch.bfloat16, 161, step=True)
    sl = torch.tensor([slots - 1], dtype=torch.int32, device="cuda")
    o = m3_delta_step(*x, pool, l2norm=True, scale=1.0, slots=sl)
    wo, wh = ref.forward(*[t[:, None] for t in x], start[None], scale=1.0, l2norm=True)
    check_o(o, wo[:, 0], "bf16", "far slot")
    check_h(pool[slots - 1], wh[0], "far slot")


def test_supported_set_runs():
    for io, code in (("f32", 0), ("bf16", 1)):
        for N in (32, 64, 128):
            for P in (32, 64, 96, 128):
                assert m3_delta_supported(N, P, code)
                x = ref.inputs(1, 66, 1, 1, N, P, DT[io], 171)
                o, h = m3_delta_fwd(*x, l2norm=True, scale=1.0)
                wo, wh = ref.forward(*x, scale=1.0, l2norm=True)
                check_o(o, wo, io, "%s N %d P %d" % (io, N, P))
                check_h(h, wh, "%s N %d P %d" % (io, N, P))


def test_refused_sizes():
    x = ref.inputs(1, 10, 2, 2, 48, 64, torch.bfloat16, 181)
    with pytest.raises(M3Error):
        m3_delta_fwd(*x)


@pytest.mark.parametrize("rows", [700, 16384, 16385])
def test_many_short_sequences(rows):
    """Packed rows are walked in the order of their lengths, above 16384 rows as they stand: each row's result is that of
    the recurrence on the rows of its length."""
    H, N, P = 1, 32, 32
    lens = torch.tensor([(5, 1, 70, 0, 2)[i % 5] if i < 500 else (1, 2, 0)[i % 3] for i in range(rows)])
    T = int(lens.sum())
    x = ref.inputs(1, T, H, H, N, P, torch.bfloat16, 61)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    h = torch.randn(rows, H, N, P, generator=torch.Generator().manual_seed(62)).cuda()
    o, hL = m3_delta_fwd(*x, h, l2norm=True, cu_seqlens=cu.to(torch.int32).cuda(), max_seqlen=int(lens.max()))
    for n in lens.unique().tolist():
        at = (lens == n).nonzero()[:, 0]
        if n == 0:
            assert torch.equal(hL[at.cuda()], h[at.cuda()])
            continue
        tok = (cu[at][:, None] + torch.arange(n)).cuda()
        wo, wh = ref.forward(*(t[0][tok] for t in x), h[at.cuda()], scale=N ** -0.5, l2norm=True)
        check_o(o[0][tok], wo, "bf16", "length %d" % n)
        check_h(hL[at.cuda()], wh, "length %d" % n)


@pytest.mark.parametrize("io,N,P,B,H,L", [("f32", 32, 32, 2, 3, 16500), ("bf16", 128, 32, 3, 4, 16384), ("bf16", 64, 64, 1, 10, 16449),
                                            ("bf16", 64, 128, 1, 20, 6700), ("f32", 128, 64, 1, 17, 4096)])
def test_long_in_parts(io, N, P, B, H, L):
    """Rows of many chunks on few CUs: the walk runs in parts that hand on the state."""
    say("case parts", io, N, P, B, H, L)
    x = ref.inputs(B, L, H, H, N, P, DT[io], 71)
    h = torch.randn(B, H, N, P, generator=torch.Generator().manual_seed(72)).cuda()
    wo, wh = ref.forward(*x, h, scale=0.2, l2norm=True)
    hl = h.clone()
    o, _ = m3_delta_fwd(*x, hl, h_out=hl, l2norm=True, scale=0.2)
    check_o(o, wo, io, "parts")
    check_h(hl, wh, "parts")
    again, none = m3_delta_fwd(*x, h, l2norm=True, scale=0.2, return_state=False)
    assert none is None and torch.equal(again, o)


def test_long_packed_in_parts():
    """Rows that end in the first part and in later ones; records in slots, one row without a record, a slot named twice."""
    N, P, H = 64, 64, 2
    lens, slots = [16400, 70, 0, 100, 4200, 16390], [2, 0, 5, 2, 3, -1]
    x = ref.inputs(1, sum(lens), H, H, N, P, torch.bfloat16, 81)
    pool = torch.randn(6, H, N, P, generator=torch.Generator().manual_seed(82)).cuda()
    before = pool.clone()
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    o, _ = m3_delta_fwd(*x, pool, l2norm=True, scale=0.2, cu_seqlens=cu.cuda(), max_seqlen=16400,
                        slots=torch.tensor(slots, dtype=torch.int32).cuda())
    for i, (n, s) in enumerate(zip(lens, slots)):
        part = slice(int(cu[i]), int(cu[i + 1]))
        if i == 3:
            assert bool(o[0, part].isnan().all())
            continue
        wo, wh = ref.forward(*(t[:, part] for t in x), before[s:s + 1] if s >= 0 else None, scale=0.2, l2norm=True)
        check_o(o[:, part], wo, "bf16", "row %d" % i)
        if s >= 0:
            check_h(pool[s:s + 1], wh, "row %d" % i)
    for s in (1, 4, 5):
        assert torch.equal(pool[s], before[s])


def test_parts_captured_and_on_two_streams():
    """A call in parts, captured and replayed between eager calls, and two such calls beside each other on streams of their own."""
    B, L, H, N, P = 1, 16449, 10, 64, 64
    x = ref.inputs(B, L, H, H, N, P, torch.bfloat16, 91)
    h = torch.randn(B, H, N, P, generator=torch.Generator().manual_seed(92)).cuda()
    run = lambda: m3_delta_fwd(*x, h, l2norm=True, scale=0.2)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for seed in (93, 94, 95):
        for dst, src in zip(x, ref.inputs(B, L, H, H, N, P, torch.bfloat16, seed)):
            dst.copy_(src)
        want = [t.clone() for t in run()]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [m3_delta_fwd(*x, h, l2norm=True, scale=0.2, stream=s) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
