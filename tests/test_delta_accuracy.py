"""How exact the gated delta rule's results are: states, float32 outputs,
gradients, and bf16 outputs before their one rounding.

Bounds.  A rounding to float32 is off by at most 2^-24 of the value, by
2^-24 / sqrt(3) in the mean square.  A sum of n terms of either sign is rounded
n times, and its partial sums grow as the root of their count, so in the mean
square it is off by 2^-24 sqrt(n / 6) of its size.  A chunk's products sum at
most N + 2 * 64 = 256 terms: 6.6 * 2^-24 each.  A state or an output has three
such products behind it, one after the other (K S, T R, K^T U; a float32
operand's 24 bits add 2^-24 / sqrt(3) a value, and the four factors of decays and
norms 2^-23 each, which changes nothing): sqrt(3 * 6.6^2 + 4 * 4) * 2^-24 =
12.1 * 2^-24 = 7.2e-7, asked for below as 2^-20.  A gradient has six: 2^-20
sqrt(2).  Both are relative to the 2-norm, for results that are not far smaller
than their terms.

A bf16 output is one rounding of such a value y.  It differs from the rounding
of the exact value only where a boundary lies between the two: for an error d and
a step s with the chance |d| / s, and then by s.  So the mean of |output - rounded
exact value| is that of |d|, whatever the values' spread, and at most the root
mean square of d: 2^-20 of that of y.  (The same in the 2-norm would weigh each
such step by its own size: one step of one large output among 6e5 would be seen.)
A mean over n outputs is off by the root of mean(|d| s) / n, for steps of 2^-8 of
the root mean square 2^-14 / sqrt(n): 0.35 of the bound at the fewest outputs
below, 32768, 0.12 at most elsewhere.

The first tests show on the CPU what these bounds see: the chunked form with
every product's operands held as sums of bf16 values, three of them or, in one
product at a time, two.
"""
import math

import pytest
import torch

import delta_reference as ref
from helpers import say

ACC = 2.0 ** -20
GRAD_ACC = ACC * math.sqrt(2.0)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh_in")


# ------------------------------------------------- the chunked form in planes

def planes(x, n):
    """x as the sum of n bf16 values, each the rounding of what those before it left."""
    left, out = x.clone(), torch.zeros_like(x)
    for _ in range(n):
        p = left.to(torch.bfloat16).double()
        out, left = out + p, left - p
    return out


class Products:
    """Products of operands held in planes: three, or two in the product named `less`."""

    def __init__(self, less=None):
        self.less = less

    def __call__(self, name, a, b):
        n = 2 if name == self.less else 3
        return planes(a, n) @ planes(b, n)


def factors(x, l2norm, eps, scale, c):
    q, k, v, g, beta = (t[0, 64 * c:64 * c + 64, 0].double() for t in x)
    if l2norm:
        q, k = (t / (t.pow(2).sum(-1, keepdim=True) + eps).sqrt() for t in (q, k))
    G = g.cumsum(0)
    D = (G[:, None] - G[None]).exp().tril()
    M = (beta[:, None] * D * (k @ k.T)).tril(-1)
    T = torch.linalg.solve_triangular(M + torch.eye(len(G), dtype=torch.float64), torch.eye(len(G), dtype=torch.float64), upper=False)
    return q, k, v, beta[:, None], G.exp()[:, None], (G[-1] - G).exp()[:, None], D, T, scale * D * (q @ k.T), G[-1].exp()


def chunked(x, h, scale, mm, keep=None, l2norm=True, eps=1e-6):
    """One row and head.  (o before its rounding, last state)"""
    S, out = h[0, 0].double(), []
    for c in range(-(-x[0].shape[1] // 64)):
        q, k, v, beta, e, d, D, T, A, last = factors(x, l2norm, eps, scale, c)
        R = beta * v - beta * e * mm("K S", k, S)
        U = mm("T R", T, R)
        out.append(scale * e * mm("Q S", q, S) + mm("A U", A, U))
        if keep is not None:
            keep.append((S, U))
        S = last * S + mm("K^T U", k.T, d * U)
    return torch.cat(out), S


def chunked_back(x, do, h, dh, scale, mm):
    """Gradients of one row and head, rows as given (no norms)."""
    keep, n = [], -(-x[0].shape[1] // 64)
    chunked(x, h, scale, mm, keep, l2norm=False)
    dS, out = dh[0, 0].double(), []
    for c in reversed(range(n)):
        q, k, v, beta, e, d, D, T, A, last = factors(x, False, 0.0, scale, c)
        S0, U = keep[c]
        o = do[0, 64 * c:64 * c + 64, 0].double()
        dU = mm("A^T dO", A.T, o) + d * mm("K dS", k, dS)
        dR = mm("T^T dU", T.T, dU)
        dA, dM = mm("dO U^T", o, U.T).tril(), -mm("dR U^T", dR, U.T).tril(-1)
        B1, B2 = scale * D * dA, beta * D * dM
        oS, rS, uS = mm("dO S^T", o, S0.T), mm("dR S^T", dR, S0.T), mm("U dS^T", U, dS.T)
        dq = scale * e * oS + mm("B1 K", B1, k)
        dk = mm("B1^T Q", B1.T, q) + mm("B2 K", B2 + B2.T, k) + d * uS - beta * e * rS
        z = B1 * (q @ k.T) + B2 * (k @ k.T)
        us = (d * uS * k).sum(1)
        dG = (scale * e * oS * q).sum(1) - (beta * e * rS * k).sum(1) + z.sum(1) - z.sum(0) - us
        dG[-1] += us.sum() + last * (S0 * dS).sum()
        dbeta = (dR * v).sum(1) - (e * rS * k).sum(1) + (D * (k @ k.T) * dM).sum(1)
        out.insert(0, (dq, dk, beta * dR, dG.flip(0).cumsum(0).flip(0), dbeta))
        dS = last * dS + mm("Q^T dO", q.T, scale * e * o) - mm("K^T dR", k.T, beta * e * dR)
    parts = [torch.cat(t) for t in zip(*out)]
    return dict(zip(NAMES, parts + [dS]))


def inputs(B, L, H, G, N, P, dtype, seed, held, device, raw=False):
    """Token tensors, states and adjoints.  held: decays near 1 and a state and adjoint ten times the writes' size, so that
    the products with them count; else the tokens' own products do."""
    x = ref.inputs(B, L, H, G, N, P, dtype, seed, device=device, raw=raw)
    gen = torch.Generator().manual_seed(seed + 1)
    h, dh = (torch.randn(B, H, N, P, generator=gen) * (10.0 if held else 1.0) for _ in range(2))
    do = torch.randn(B, L, H, P, generator=gen).to(dtype)
    if held:
        x[3] = x[3] * 0.02
    return x, h.to(device), do.to(device), dh.to(device)


def rounding_error(o, want):
    """Mean distance of a bf16 output from the exact value rounded once, over the values' root mean square."""
    return float((o.double().cpu() - want.to(torch.bfloat16).double()).abs().mean() / want.pow(2).mean().sqrt())


@pytest.mark.parametrize("less", [None, "K S", "T R", "K^T U"])
def test_bound_of_the_state_sees_two_planes(less):
    worst = 0.0
    for L, held in ((190, False), (130, True)):
        x, h, _, _ = inputs(1, L, 1, 1, 64, 64, torch.float32, 11, held, "cpu")
        _, S = chunked(x, h, 0.3, Products(less))
        worst = max(worst, ref.rel2(S, ref.forward(*x, h, scale=0.3, l2norm=True)[1][0, 0]))
    say("   less %s: h %.1e" % (less, worst))
    assert (worst > ACC) == (less is not None)


@pytest.mark.parametrize("less", [None, "Q S", "A U"])
def test_bound_of_float32_outputs_sees_two_planes(less):
    worst = 0.0
    for L, held in ((190, False), (130, True)):
        x, h, _, _ = inputs(1, L, 1, 1, 64, 64, torch.float32, 11, held, "cpu")
        o, _ = chunked(x, h, 0.3, Products(less))
        worst = max(worst, ref.rel2(o, ref.forward(*x, h, scale=0.3, l2norm=True)[0][0, :, 0]))
    say("   less %s: o %.1e" % (less, worst))
    assert (worst > ACC) == (less is not None)


@pytest.mark.parametrize("less,L,held", [(None, 1500, False), (None, 64, True), ("A U", 1500, False), ("Q S", 64, True)])
def test_bound_of_bf16_outputs_sees_two_planes(less, L, held):
    got, want = [], []
    for seed in range(21, 45 if held else 22):
        x, h, _, _ = inputs(1, L, 1, 1, 64, 64, torch.bfloat16, seed, held, "cpu")
        got.append(chunked(x, h, 0.3, Products(less))[0].to(torch.bfloat16))
        want.append(ref.forward(*x, h, scale=0.3, l2norm=True)[0][0, :, 0])
    e = rounding_error(torch.cat(got), torch.cat(want))
    say("   less %s: %.1e" % (less, e))
    assert (e > ACC) == (less is not None)


PRODUCTS = ["T R", "A^T dO", "K dS", "T^T dU", "dO U^T", "dR U^T", "dO S^T", "dR S^T", "U dS^T", "B1 K", "B1^T Q", "B2 K",
            "Q^T dO", "K^T dR"]


@pytest.mark.parametrize("less", [None] + PRODUCTS)
def test_bound_of_gradients_sees_two_planes(less):
    worst = 0.0
    for L, held in ((190, False), (130, True)):
        x, h, do, dh = inputs(1, L, 1, 1, 64, 64, torch.float32, 31, held, "cpu", raw=True)
        want = ref.backward(*x, do, h, dh, scale=0.3, l2norm=False)
        got = chunked_back(x, do, h, dh, 0.3, Products(less))
        for n in NAMES:
            if n != "dg" or not held:   # (dg of a held state is far smaller than its terms)
                worst = max(worst, ref.rel2(got[n], want[n][0] if n == "dh_in" else want[n][0, :, 0]))
    say("   less %s: %.1e" % (less, worst))
    assert (worst > GRAD_ACC) == (less is not None)


# ------------------------------------------------------------------ the kernels

FORWARD = [
    # B, L, H, G, N, P, io: every walk, 16, 32 and 64 columns to a workgroup, and in parts
    (2, 500, 8, 8, 64, 64, "bf16"), (1, 300, 8, 4, 128, 128, "bf16"), (4, 200, 6, 2, 32, 96, "bf16"),
    (2, 300, 4, 2, 64, 64, "f32"), (1, 200, 6, 6, 128, 96, "f32"), (2, 130, 5, 5, 32, 32, "f32"),
    (1, 130, 72, 8, 64, 64, "bf16"), (1, 130, 44, 44, 128, 96, "bf16"), (1, 100, 130, 13, 32, 32, "bf16"),
    (1, 130, 132, 12, 64, 64, "bf16"), (1, 70, 130, 13, 128, 64, "bf16"), (2, 70, 40, 40, 32, 128, "bf16"),
    (1, 16400, 8, 4, 128, 32, "bf16"), (1, 16449, 10, 10, 64, 64, "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("B,L,H,G,N,P,io", FORWARD)
def test_prefill(B, L, H, G, N, P, io, held):
    from mamba_selective_ssm_amd import m3_delta_fwd
    say("case prefill", B, L, H, G, N, P, io, held)
    x, h, _, _ = inputs(B, L, H, G, N, P, DT[io], 41, held, "cuda")
    o, hL = m3_delta_fwd(*x, h, l2norm=True, scale=0.3)
    wo, wh = ref.forward(*x, h, scale=0.3, l2norm=True)
    eo = rounding_error(o, wo) if io == "bf16" else ref.rel2(o, wo)
    eh = ref.rel2(hL, wh)
    say("   o %.2e, h %.2e" % (eo, eh))
    assert max(eo, eh) <= ACC


@pytest.mark.gpu
@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("B,H,G,N,P,io", [(64, 8, 8, 64, 64, "bf16"), (32, 8, 2, 128, 128, "bf16"), (64, 8, 8, 32, 96, "f32"),
                                          (32, 4, 1, 128, 64, "f32")])
def test_step(B, H, G, N, P, io, held):
    from mamba_selective_ssm_amd import m3_delta_step
    say("case step", B, H, G, N, P, io, held)
    x, h, _, _ = inputs(B, 1, H, G, N, P, DT[io], 51, held, "cuda")
    wo, wh = ref.forward(*x, h, scale=0.3, l2norm=True)
    o = m3_delta_step(*[t[:, 0].contiguous() for t in x], h, l2norm=True, scale=0.3)
    eo = rounding_error(o, wo[:, 0]) if io == "bf16" else ref.rel2(o, wo[:, 0])
    eh = ref.rel2(h, wh)
    say("   o %.2e, h %.2e" % (eo, eh))
    assert max(eo, eh) <= ACC


@pytest.mark.gpu
@pytest.mark.parametrize("L,N,P,io", [(64, 64, 64, "bf16"), (17, 32, 32, "f32"), (50, 128, 128, "bf16"), (33, 64, 96, "f32")])
def test_decay_of_the_zero_state_has_no_gradient(L, N, P, io):
    """The first token's decay acts on a state of zeros: its dg is a sum over one chunk whose terms, each a product of float32
    values, cancel in pairs.  The pairs are equal bit for bit, so what is left is the sums' own rounding: at most L^2 = 2^12
    terms of 2^-53 each, 2^-41 of their sizes' sum, which is of the size of the 64 other values; asked for as 2^-36 of their
    root mean square."""
    from mamba_selective_ssm_amd import m3_delta_bwd
    x, _, do, _ = inputs(2, L, 4, 2, N, P, DT[io], 71, False, "cuda")
    got = m3_delta_bwd(*x, do, l2norm=True, scale=0.3)
    dg = got.dg.double()
    worst = float(dg[:, 0].abs().max() / dg.pow(2).mean().sqrt())
    say("   %.1e of the others" % worst)
    assert worst <= 2.0 ** -36
    # the others are what they should be
    assert ref.rel2(got.dg, ref.backward(*x, do, scale=0.3, l2norm=True)["dg"]) <= GRAD_ACC


@pytest.mark.gpu
@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("B,L,H,G,N,P,io,l2", [
    (2, 300, 4, 4, 64, 64, "bf16", True), (1, 200, 4, 1, 128, 128, "bf16", True), (2, 130, 6, 2, 32, 96, "bf16", False),
    (1, 300, 4, 2, 64, 64, "f32", True), (1, 130, 2, 2, 128, 64, "f32", False), (1, 200, 3, 3, 32, 128, "f32", True),
    (1, 130, 2, 1, 128, 128, "f32", True)])
def test_gradient(B, L, H, G, N, P, io, l2, held):
    from mamba_selective_ssm_amd import m3_delta_bwd
    say("case gradient", B, L, H, G, N, P, io, l2, held)
    x, h, do, dh = inputs(B, L, H, G, N, P, DT[io], 61, held, "cuda", raw=not l2)
    got = m3_delta_bwd(*x, do, h, dh, scale=0.3, l2norm=l2)
    want = ref.backward(*x, do, h, dh, scale=0.3, l2norm=l2)
    errs = {n: ref.rel2(getattr(got, n), want[n]) for n in NAMES}
    say("   " + " ".join("%s %.1e" % e for e in errs.items()))
    for n, e in errs.items():
        assert e <= GRAD_ACC or (n == "dg" and held), (n, e)
