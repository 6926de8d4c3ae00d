"""Gradient of the gated delta rule on the GPU against the float64 adjoint
recurrence and against differences of the forward kernel.

Tolerance.  Every product's operands are held to 24 bits and every sum to
float32, as in the forward pass.  A gradient passes through at most six such
products one after the other (state, U, the adjoint's three, its own), each of
sums of at most N + 64 + 64 <= 256 terms: 6 * 256 * 2^-24 = 9.2e-5 of the size
of its terms if all roundings fell the same way, for dg once more through the
sum over the chunk's 64 tokens, which float64 holds.  2e-5 of the result's
2-norm is asked for where results are not far smaller than their terms.
"""
import pytest
import torch

import delta_reference as ref
from helpers import say
from mamba_selective_ssm_amd import m3_delta_bwd, m3_delta_fwd

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = 2e-5
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh_in")


def check(got, want, label, tol=TOL):
    errs = {n: ref.rel2(getattr(got, n), want[n]) for n in NAMES if getattr(got, n) is not None}
    say("   %s: %s" % (label, " ".join("%s %.1e" % e for e in errs.items())))
    for n, e in errs.items():
        assert e <= tol, (n, e)


def grads_in(B, L, H, N, P, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(B, L, H, P, generator=gen).to(dtype).cuda(),
            torch.randn(B, H, N, P, generator=gen).cuda(), torch.randn(B, H, N, P, generator=gen).cuda())


CASES = [
    # B, L, H, G, N, P, io, l2norm
    (1, 1, 1, 1, 64, 64, "bf16", True),
    (1, 5, 2, 1, 32, 32, "f32", True),
    (2, 16, 3, 3, 64, 32, "bf16", False),
    (1, 63, 4, 2, 128, 64, "bf16", True),
    (1, 64, 2, 2, 64, 96, "f32", True),
    (2, 65, 4, 1, 64, 64, "bf16", True),
    (1, 130, 3, 3, 128, 128, "bf16", True),
    (1, 200, 2, 1, 128, 128, "f32", True),
    (1, 300, 9, 3, 32, 96, "bf16", True),
    (3, 190, 5, 5, 64, 64, "f32", False),
    (1, 700, 2, 2, 64, 128, "bf16", True),
]


@pytest.mark.parametrize("B,L,H,G,N,P,io,l2", CASES)
def test_gradient(B, L, H, G, N, P, io, l2):
    say("case gradient", B, L, H, G, N, P, io, l2)
    x = ref.inputs(B, L, H, G, N, P, DT[io], 211, raw=not l2)
    do, h, dh = grads_in(B, L, H, N, P, DT[io], 212)
    for h0, d0 in ((h, dh), (None, None)):
        got = m3_delta_bwd(*x, do, h0, d0, scale=0.3, l2norm=l2)
        check(got, ref.backward(*x, do, h0, d0, scale=0.3, l2norm=l2), "given state" if h0 is not None else "zero state")
    got = m3_delta_bwd(*x, do, h, dh, scale=0.3, l2norm=l2, state_grad=False)
    assert got.dh_in is None
    check(got, ref.backward(*x, do, h, dh, scale=0.3, l2norm=l2), "without dh_in")


@pytest.mark.parametrize("io,N,P,H,G", [("bf16", 64, 64, 4, 2), ("f32", 32, 96, 3, 3), ("bf16", 128, 64, 2, 1)])
def test_packed(io, N, P, H, G):
    lens = [5, 0, 64, 1, 130, 63, 0, 65]
    before, behind = 0, 11
    T = before + sum(lens) + behind
    x = ref.inputs(1, T, H, G, N, P, DT[io], 221)
    gen = torch.Generator().manual_seed(222)
    do = torch.randn(1, T, H, P, generator=gen).to(DT[io]).cuda()
    h, dh = (torch.randn(len(lens), H, N, P, generator=gen).cuda() for _ in range(2))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    torch.full((1 << 24,), float("nan"), device="cuda")     # what the outputs' memory held before
    got = m3_delta_bwd(*x, do, h, dh, scale=0.2, l2norm=True, cu_seqlens=cu, max_seqlen=130)
    parts = ref.packed(ref.backward, lens, x + [do], [h, dh], scale=0.2, l2norm=True)
    want = {n: torch.cat([p[n] for p in parts], 0 if n == "dh_in" else 1) for n in NAMES}
    for n in NAMES[:5]:
        assert not bool(getattr(got, n)[:, sum(lens):].any()), n
    check(got._replace(**{n: getattr(got, n)[:, :sum(lens)] for n in NAMES[:5]}), want, "packed")
    for i, n in enumerate(lens):
        if n == 0:
            assert torch.equal(got.dh_in[i], dh[i])


def test_packed_gaps():
    """Tokens before the first sequence and behind the last get zeros."""
    x = ref.inputs(1, 100, 2, 1, 32, 32, torch.bfloat16, 231)
    do, _, _ = grads_in(1, 100, 2, 32, 32, torch.bfloat16, 232)
    cu = torch.tensor([20, 50, 90], dtype=torch.int32, device="cuda")
    got = m3_delta_bwd(*x, do, l2norm=True, cu_seqlens=cu)
    for n in NAMES[:5]:
        t = getattr(got, n)
        assert not bool(t[:, :20].any()) and not bool(t[:, 90:].any()) and bool(t[:, 20:90].any()), n


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_strong_and_absent_decay(io):
    x = ref.inputs(1, 150, 2, 2, 64, 32, DT[io], 241)
    x[3][:, 10] = -float("inf")
    x[3][:, 40:60] = -200.0
    x[3][:, 70:140] = 0.0
    x[4][:, 80:90] = 0.0
    do, h, dh = grads_in(1, 150, 2, 64, 32, DT[io], 242)
    got = m3_delta_bwd(*x, do, h, dh, scale=1.0, l2norm=True)
    check(got, ref.backward(*x, do, h, dh, scale=1.0, l2norm=True), "decays")


def test_differences_of_the_forward_pass():
    """The directional derivative of a loss of m3_delta_fwd along random
    directions, by central differences in float32: the loss has some 1e4 terms
    of size 1 known to 2^-24 times their count's root, and a step of 2^-7
    leaves a third-order term of 2^-14 of the second derivative's size."""
    B, L, H, G, N, P = 1, 90, 2, 1, 32, 32
    x = ref.inputs(B, L, H, G, N, P, torch.float32, 251)
    do, h, dh = grads_in(B, L, H, N, P, torch.float32, 252)

    def loss(x, h):
        o, hl = m3_delta_fwd(*x, h, scale=0.5, l2norm=True)
        return float((o.double() * do.double()).sum() + (hl.double() * dh.double()).sum())

    got = m3_delta_bwd(*x, do, h, dh, scale=0.5, l2norm=True)
    step = 2.0 ** -7
    gen = torch.Generator().manual_seed(253)
    for i, n in enumerate(NAMES):
        base = (x + [h])[i]
        d = torch.randn(base.shape, generator=gen).cuda()
        d /= d.norm()
        up, down = ([t + s * step * d if j == i else t for j, t in enumerate(x + [h])] for s in (1, -1))
        diff = (loss(up[:5], up[5]) - loss(down[:5], down[5])) / (2 * step)
        want = float((getattr(got, n).double() * d.double()).sum())
        say("   %s: differences %.6f, gradient %.6f" % (n, diff, want))
        assert abs(diff - want) <= 2e-3 * max(1.0, abs(want), float(getattr(got, n).norm()) * 0.05)


def test_split_into_calls():
    """A sequence in two calls: the second call's dh_in is the first one's dh_out."""
    x = ref.inputs(2, 200, 4, 2, 64, 64, torch.bfloat16, 261)
    do, h, dh = grads_in(2, 200, 4, 64, 64, torch.bfloat16, 262)
    kw = dict(scale=0.3, l2norm=True)
    a, b = ([t[:, s].contiguous() for t in x] for s in (slice(0, 77), slice(77, 200)))
    _, mid = m3_delta_fwd(*a, h, **kw)
    g2 = m3_delta_bwd(*b, do[:, 77:].contiguous(), mid, dh, **kw)
    g1 = m3_delta_bwd(*a, do[:, :77].contiguous(), h, g2.dh_in, **kw)
    want = ref.backward(*x, do, h, dh, **kw)
    check(g1._replace(**{n: torch.cat([getattr(g1, n), getattr(g2, n)], 1) for n in NAMES[:5]}), want, "two calls")


def test_no_tokens():
    x = ref.inputs(2, 0, 3, 3, 64, 64, torch.bfloat16, 271)
    do, h, dh = grads_in(2, 0, 3, 64, 64, torch.bfloat16, 272)
    got = m3_delta_bwd(*x, do, h, dh)
    assert torch.equal(got.dh_in, dh)
    assert not bool(m3_delta_bwd(*x, do).dh_in.any())


def test_same_results_every_time_captured_and_on_streams():
    x = ref.inputs(2, 333, 4, 2, 64, 64, torch.bfloat16, 281)
    do, h, dh = grads_in(2, 333, 4, 64, 64, torch.bfloat16, 282)
    first = m3_delta_bwd(*x, do, h, dh, l2norm=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(4):
        got = m3_delta_bwd(*x, do, h, dh, l2norm=True, stream=streams[i % 2])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m3_delta_bwd(*x, do, h, dh, l2norm=True)
    for seed in (283, 284, 285):
        for dst, src in zip(x, ref.inputs(2, 333, 4, 2, 64, 64, torch.bfloat16, seed)):
            dst.copy_(src)
        want = m3_delta_bwd(*x, do, h, dh, l2norm=True)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_training_step_of_a_stack():
    """Two mixers in a row with their prefill and gradient, as a training step
    runs them: the first one's output is the second one's value."""
    H, N, P = 2, 64, 64
    x = ref.inputs(1, 150, H, H, N, P, torch.float32, 291)
    y = ref.inputs(1, 150, H, H, N, P, torch.float32, 292)
    do, _, _ = grads_in(1, 150, H, N, P, torch.float32, 293)
    kw = dict(scale=1.0, l2norm=True)
    o1, _ = m3_delta_fwd(*x, **kw)
    g2 = m3_delta_bwd(y[0], y[1], o1, y[3], y[4], do, **kw)
    g1 = m3_delta_bwd(*x, g2.dv, **kw)
    w1, _ = ref.forward(*x, **kw)
    want2 = ref.backward(y[0], y[1], w1, y[3], y[4], do, **kw)
    want1 = ref.backward(*x, want2["dv"], **kw)
    check(g2, want2, "second")
    check(g1, want1, "first")
