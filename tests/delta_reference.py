"""The gated delta rule and its adjoint in float64, token by token on the CPU,
and seeded inputs for its tests."""
import torch


def unit_rows(x, l2norm, eps):
    x = x.double().cpu()
    return x / (x.pow(2).sum(-1, keepdim=True) + eps).sqrt() if l2norm else x


def decay(g):
    """exp(g), as the library defines it for values without a finite float32 exponential."""
    return g.double().cpu().exp()


def forward(q, k, v, g, beta, h=None, scale=1.0, l2norm=False, eps=1e-6, keep=None):
    """One dense batch: q, k [B, L, G, N], v [B, L, H, P], g, beta [B, L, H],
    h [B, H, N, P].  (o, state after the last token); `keep` collects the
    states and writes of every token."""
    B, L, G, N = q.shape
    H, P = v.shape[2:]
    head = torch.arange(H) // (H // G)
    q, k = (unit_rows(x, l2norm, eps)[:, :, head] for x in (q, k))
    v, a, beta = v.double().cpu(), decay(g), beta.double().cpu()
    S = torch.zeros(B, H, N, P, dtype=torch.float64) if h is None else h.double().cpu().clone()
    o = torch.zeros(B, L, H, P, dtype=torch.float64)
    for t in range(L):
        Sa = S * a[:, t, :, None, None]
        r = v[:, t] - (Sa * k[:, t, :, :, None]).sum(2)
        u = beta[:, t, :, None] * r
        if keep is not None:
            keep.append((S, Sa, r, u))
        S = Sa + k[:, t, :, :, None] * u[:, :, None]
        o[:, t] = scale * (S * q[:, t, :, :, None]).sum(2)
    return o, S


def backward(q, k, v, g, beta, do, h=None, dh=None, scale=1.0, l2norm=False, eps=1e-6):
    """dq, dk, dv, dg, dbeta, dh_in of sum(do o) + sum(dh S_L), one dense batch."""
    keep = []
    _, S = forward(q, k, v, g, beta, h, scale, l2norm, eps, keep)
    B, L, G, N = q.shape
    H, P = v.shape[2:]
    head = torch.arange(H) // (H // G)
    qn, kn = (unit_rows(x, l2norm, eps)[:, :, head] for x in (q, k))
    a, b = decay(g), beta.double().cpu()
    do = do.double().cpu()
    dS = torch.zeros_like(S) if dh is None else dh.double().cpu().clone()
    dq, dk = torch.zeros_like(qn), torch.zeros_like(kn)
    dv, dg, db = torch.zeros_like(do), torch.zeros_like(a), torch.zeros_like(a)
    for t in reversed(range(L)):
        S0, Sa, r, u = keep[t]
        kt, qt, go = kn[:, t, :, :, None], qn[:, t, :, :, None], scale * do[:, t, :, None]
        St = Sa + kt * u[:, :, None]
        dq[:, t] = (St * go).sum(3)
        dS = dS + qt * go
        du = (dS * kt).sum(2)
        dk[:, t] = (dS * u[:, :, None]).sum(3)
        dv[:, t] = b[:, t, :, None] * du
        db[:, t] = (du * r).sum(2)
        dSa = dS - kt * dv[:, t][:, :, None]
        dk[:, t] -= (Sa * dv[:, t][:, :, None]).sum(3)
        dg[:, t] = (dSa * Sa).sum((2, 3))
        dS = dSa * a[:, t, :, None, None]

    def to_rows(raw, d):
        d = d.reshape(B, L, G, H // G, N).sum(3)
        if not l2norm:
            return d
        raw = raw.double().cpu()
        i = (raw.pow(2).sum(-1, keepdim=True) + eps).rsqrt()
        x = raw * i
        return i * (d - x * (x * d).sum(-1, keepdim=True))

    return dict(dq=to_rows(q, dq), dk=to_rows(k, dk), dv=dv, dg=dg, dbeta=db, dh_in=dS)


def packed(fn, lens, tensors, rows=(), **kw):
    """fn on every sequence of [1, T, ...] tensors by itself; `rows` are per-sequence tensors."""
    out, at = [], 0
    for i, n in enumerate(lens):
        part = [t[:, at:at + n] for t in tensors]
        out.append(fn(*part, *[None if r is None else r[i:i + 1] for r in rows], **kw))
        at += n
    return out


def inputs(B, L, H, G, N, P, dtype, seed, device="cuda", step=False, raw=False):
    """Token tensors: q and k share a part (repeating keys), sigmoid write
    strengths, log decays of mixed rates.  raw: rows scaled to unit length
    already, for calls without l2norm."""
    gen = torch.Generator().manual_seed(seed)
    tok = (B,) if step else (B, L)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    common = normal(*tok, G, N)
    q, k = normal(*tok, G, N) + 0.5 * common, normal(*tok, G, N) + 0.5 * common
    if raw:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    v = normal(*tok, H, P)
    rate = torch.exp(torch.rand(H, generator=gen) * 2 - 1)
    g = -rate * torch.nn.functional.softplus(normal(*tok, H) - 2.0)
    beta = torch.sigmoid(normal(*tok, H))
    return [x.to(dtype).to(device) for x in (q, k, v)] + [g.to(device), beta.to(device)]


def rel2(got, ref):
    """2-norm of the difference over that of the reference."""
    got, ref = got.double().cpu(), ref.double().cpu()
    n = float(ref.norm())
    return float((got - ref).norm()) / n if n else float((got - ref).norm())
