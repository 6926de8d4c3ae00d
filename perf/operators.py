"""Cases of the gated delta rule (prefill, one-token step, gradient) and of the
pool of state records (copy, fork, compact, free), each with a plain form in
elementary torch operations and the library's call.

The operators:
    S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t (v_t - (a_t S_{t-1})^T k_t),
    o_t = scale S_t^T q_t,          a_t = exp(g_t)
per (batch row or sequence, head), S of N x P values in float32; q and k are
shared by groups of heads, and with `l2norm` each of their rows is divided by
sqrt(sum of squares + eps) first.  A pool keeps one record per slot, along the
leading axis of each of its arrays.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lib():
    if own:
        import mamba_selective_ssm_amd as m3_
        return m3_
    return None


# ------------------------------------------------------------------ the cases

def _mix(name, op, batch, heads, groups, seqlen, N, P, io="bf16", l2norm=True, packed=0, slots=0, state=False):
    """seqlen: tokens of a batch row, or of all `packed` sequences together."""
    return dict(name=name, op=op, batch=batch, heads=heads, groups=groups, seqlen=seqlen, dstate=N, headdim=P, io=io,
                l2norm=l2norm, packed=packed, slots=slots, state=state)


def _pool(name, op, slots, count, heads, rank, N, P, mixer):
    """mixer: the Mamba-3 record (h, B_prev, x_prev), else the delta rule's h alone."""
    return dict(name=name, op=op, slots=slots, count=count, heads=heads, rank=rank, dstate=N, headdim=P, mixer=mixer)


def listed():
    return [
        # one short prompt (37 tokens, one chunk, ragged): what a prompt's latency is made of
        _mix("prefill short prompt", "prefill", 1, 16, 16, 37, 64, 64),
        # one layer of a training batch or of batched prompts, the shape of the library's single-layer prefill
        _mix("prefill layer", "prefill", 4, 16, 16, 2048, 64, 64),
        # a long document in one call: few heads, very many chunks
        _mix("prefill long document", "prefill", 1, 32, 32, 65536, 128, 64),
        # serving: prompts of different lengths packed, continued from and written back to a pool's slots, heads in groups
        _mix("prefill packed into slots", "prefill", 1, 32, 8, 20011, 128, 128, packed=13, slots=24, state=True),
        # float32 model, odd length, rows as given
        _mix("prefill float32", "prefill", 2, 8, 8, 777, 64, 32, io="f32", l2norm=True, state=True),
        # one user, one token: latency
        _mix("step one user", "step", 1, 16, 16, 1, 64, 64, state=True),
        # a full decode batch on a pool, the shape of the library's decode workload
        _mix("step full batch in slots", "step", 256, 32, 32, 1, 128, 64, slots=320, state=True),
        # gradient of the layer above: a training step's part
        _mix("gradient layer", "gradient", 4, 16, 16, 2048, 64, 64),
        # gradient with shared heads, odd packed sequences and a carried state
        _mix("gradient packed groups", "gradient", 1, 16, 4, 4099, 128, 64, packed=7, state=True),
        # a few new samples forked from live sequences: latency
        _pool("fork samples", "fork", 64, 8, 16, 1, 64, 64, True),
        # snapshot of sequences into another pool (prefix cache), full records
        _pool("copy to snapshot pool", "copy", 256, 96, 32, 4, 128, 64, True),
        # half of a large pool has ended: the live records move to the front
        _pool("compact after endings", "compact", 512, 250, 32, 1, 128, 64, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "gradient", "gradient", "fork", "copy", "compact"])
    N, P = rng.choice([32, 64, 128]), rng.choice([32, 64, 96, 128])
    groups = _log(rng, 1, 16)
    heads = groups * rng.choice([1, 1, 2, 4])
    if op in ("fork", "copy", "compact"):
        slots = _log(rng, 4, 300)
        return dict(op=op, slots=slots, count=max(1, min(slots // 2, _log(rng, 1, 150))), heads=heads,
                    rank=rng.choice([1, 2, 4]), dstate=N, headdim=P, mixer=rng.random() < 0.7)
    io = "f32" if rng.random() < 0.25 else "bf16"
    case = dict(op=op, batch=_log(rng, 1, 8), heads=heads, groups=groups, seqlen=_log(rng, 1, 4000), dstate=N, headdim=P,
                io=io, l2norm=True, packed=0, slots=0, state=rng.random() < 0.5)
    if op == "step":
        case.update(batch=_log(rng, 1, 200), seqlen=1, state=True)
        if rng.random() < 0.5:
            case["slots"] = case["batch"] + rng.randrange(0, 40)
    elif rng.random() < 0.4:
        case.update(packed=case["batch"], batch=1, seqlen=case["seqlen"] * case["batch"])
        if op == "prefill" and rng.random() < 0.5:
            case.update(slots=case["packed"] + rng.randrange(0, 20), state=True)
    most = 65536 * 32 * 192   # no more than the long document's values
    if case["batch"] * case["seqlen"] * heads * (N + P) > most:
        case["seqlen"] = most // (case["batch"] * heads * (N + P))
    if op == "gradient":   # the exact adjoint keeps a float64 state per token
        per = 8 * case["heads"] * N * P
        most = int(12e9 / per)
        if case["batch"] * case["seqlen"] > most:
            case["seqlen"] = max(case["packed"], most // case["batch"], 1)
    return case


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(case, seed):
    """Lengths of the packed sequences: all different, their sum the token count; from the seed on the host."""
    n, T = case["packed"], case["seqlen"]
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(n, generator=g, dtype=torch.float64) + 0.1
    cut = (torch.cumsum(w, 0) / w.sum() * T).round().long()
    cut[-1] = T
    return [int(x) for x in torch.diff(cut, prepend=torch.zeros(1, dtype=torch.long))]


def prepare(case, seed):
    gen = _generator(seed)
    if case["op"] in ("fork", "copy", "compact"):
        return _prepare_pool(case, gen)
    B, L, H, G, N, P = (case[k] for k in ("batch", "seqlen", "heads", "groups", "dstate", "headdim"))
    dt = DTYPES[case["io"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    tok = (B,) if case["op"] == "step" else (B, L)
    s = dict(case=case, op=case["op"], scale=N ** -0.5, cu=None, max_seqlen=None, slots=None, h=None)
    # q and k share a part, as they do where both come from one hidden state
    common = normal(*tok, G, N)
    s["q"] = (normal(*tok, G, N) + 0.5 * common).to(dt)
    s["k"] = (normal(*tok, G, N) + 0.5 * common).to(dt)
    s["v"] = normal(*tok, H, P).to(dt)
    # log decay -exp(a) softplus(.), write strength sigmoid(.)
    rate = torch.exp(torch.rand(H, generator=gen, device="cuda") * 2 - 1)
    s["g"] = -rate * torch.nn.functional.softplus(normal(*tok, H) - 2.0)
    s["beta"] = torch.sigmoid(normal(*tok, H))
    rows = case["packed"] or B
    if case["packed"]:
        lens = _lengths(case, seed)
        s["lens"] = lens
        cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(lens), 0)
        s["cu"], s["max_seqlen"] = cu.cuda(), max(lens)
    if case["slots"]:
        s["slots"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:rows].to(torch.int32)
    if case["state"]:
        s["h"] = 0.3 * normal(case["slots"] or rows, H, N, P)
    if case["op"] == "gradient":
        s["do"] = normal(*tok, H, P).to(dt)
        s["dh"] = 0.3 * normal(rows, H, N, P)
    return s


def _prepare_pool(case, gen):
    S, n, H, R, N, P = (case[k] for k in ("slots", "count", "heads", "rank", "dstate", "headdim"))

    def record(slots):
        h = torch.randn((slots, H, N, P), generator=gen, device="cuda")
        if not case["mixer"]:
            return (h,)
        return (h, torch.randn((slots, H, R, N), generator=gen, device="cuda").to(torch.bfloat16),
                torch.randn((slots, H, R, P), generator=gen, device="cuda").to(torch.bfloat16))

    s = dict(case=case, op=case["op"], pool=record(S))
    order = torch.randperm(S, generator=gen, device="cuda")
    live = torch.zeros(S, dtype=torch.int32, device="cuda")
    if case["op"] == "fork":
        live[order[: S - n]] = 1
        s["parents"] = order[: S - n][torch.randint(0, S - n, (n,), generator=gen, device="cuda")].to(torch.int32)
        s["live_out"], s["children"] = torch.empty_like(live), torch.empty(n, dtype=torch.int32, device="cuda")
    elif case["op"] == "copy":
        s["to"] = record(n)
        s["src"] = order[:n].to(torch.int32)
        s["dst"] = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
    else:
        live[order[:n]] = 1
        s["new_slot"] = torch.empty(S, dtype=torch.int32, device="cuda")
        s["count_out"] = torch.empty(1, dtype=torch.int32, device="cuda")
    s["live"] = live
    return s


# ---------------------------------------------------------------- the passes

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    lib = _lib()
    op = s["op"]
    if op == "prefill":
        kw = dict(scale=s["scale"], l2norm=s["case"]["l2norm"], norm_eps=EPS, cu_seqlens=s["cu"], max_seqlen=s["max_seqlen"])
        if s["slots"] is not None:   # the pool's records are continued in place
            o, h = lib.m3_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h"], h_out=s["h"], slots=s["slots"], **kw)
        else:
            o, h = lib.m3_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h"], **kw)
        return {"o": o, "h": h}
    if op == "step":
        o = lib.m3_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h"], scale=s["scale"], l2norm=s["case"]["l2norm"],
                              norm_eps=EPS, slots=s["slots"])
        return {"o": o, "h": s["h"]}
    if op == "gradient":
        r = lib.m3_delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], s["h"], s["dh"], scale=s["scale"],
                             l2norm=s["case"]["l2norm"], norm_eps=EPS, cu_seqlens=s["cu"], max_seqlen=s["max_seqlen"])
        return {"dq": r.dq, "dk": r.dk, "dv": r.dv, "dg": r.dg, "dbeta": r.dbeta, "dh": r.dh_in}
    if op == "fork":
        lib.m3_pool_fork(s["pool"], s["live"], s["parents"], children=s["children"], live_out=s["live_out"])
        return {"pool": s["pool"], "children": s["children"], "live": s["live_out"]}
    if op == "copy":
        lib.m3_pool_copy(s["pool"], s["to"], s["src"], s["dst"])
        return {"to": s["to"]}
    lib.m3_pool_compact(s["pool"], s["live"], new_slot=s["new_slot"], count=s["count_out"])
    return {"pool": s["pool"], "new_slot": s["new_slot"], "count": s["count_out"]}


def _unpack(s):
    """Row indices [sequences, longest] of packed tokens, and which of them are tokens."""
    start = s["cu"][:-1].long()[:, None]
    at = torch.arange(s["max_seqlen"], device="cuda")[None]
    real = at < (s["cu"][1:].long()[:, None] - start)
    return (start + at) * real, real


def _rows(x, l2norm):
    x = x.float()
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS) if l2norm else x


def _heads_first(s, q, k, v, g, beta):
    """[rows, heads, tokens, ...] float32 operands of a batch or of packed sequences."""
    reach = s["case"]["heads"] // s["case"]["groups"]
    q, k = (x.repeat_interleave(reach, dim=2) for x in (q, k))
    if s["cu"] is not None:
        at, real = _unpack(s)
        q, k, v, g, beta = (x[0][at] * real.reshape(real.shape + (1,) * (x.dim() - 2)) for x in (q, k, v, g, beta))
    return [x.transpose(1, 2) for x in (q, k, v, g, beta)]


def _inverse(M):
    """(I + M)^-1 of strictly lower triangular M [..., 64, 64], blocks of 1, 2, 4, .. joined pairwise."""
    n, size = M.shape[0], 1
    T = torch.eye(64, device=M.device).repeat(n, 1, 1)
    while size < 64:
        pairs = 64 // (2 * size)
        i = torch.arange(pairs, device=M.device)
        Mb = M.reshape(n, pairs, 2 * size, pairs, 2 * size)[:, i, :, i, :].transpose(0, 1)
        Tb = T.reshape(n, pairs, 2 * size, pairs, 2 * size)[:, i, :, i, :].transpose(0, 1)
        a, d, m = Tb[:, :, :size, :size], Tb[:, :, size:, size:], Mb[:, :, size:, :size]
        low = -(d.contiguous() @ (m.contiguous() @ a.contiguous()))
        top = torch.cat([a, torch.zeros_like(a)], -1)
        both = torch.cat([top, torch.cat([low, d], -1)], -2)
        T = (both[:, :, :, None, :] * torch.eye(pairs, device=M.device)[None, :, None, :, None]).reshape(n, 64, 64)
        size *= 2
    return T


def _plain_delta(q, k, v, g, beta, S, scale):
    """The chunked form, 64 tokens to a chunk, on [rows, heads, tokens, ...] float32; g float64.  (o, last state)"""
    R, H, L, N = q.shape
    P, n = v.shape[-1], -(-L // 64)
    pad = n * 64 - L

    def chunks(x):
        x = torch.nn.functional.pad(x, (0, 0, 0, pad) if x.dim() == 4 else (0, pad))
        return x.reshape(R * H, n, 64, *x.shape[3:])

    q, k, v, g, beta = (chunks(x) for x in (q, k, v, g, beta))
    G = torch.cumsum(g, -1)
    low = torch.ones(64, 64, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).float()
    e, d, last = torch.exp(G).float(), torch.exp(G[..., -1:] - G).float(), torch.exp(G[..., -1]).float()
    kt = k.transpose(-1, -2).contiguous()
    M = (beta[..., None] * D * (k @ kt)).tril(-1)
    T = _inverse(M.reshape(-1, 64, 64)).reshape(M.shape)
    A = D * (q @ kt)
    U0 = T @ (beta[..., None] * v)
    W = T @ ((beta * e)[..., None] * k)
    qe, ktd = q * e[..., None], (k * d[..., None]).transpose(-1, -2).contiguous()
    S = q.new_zeros(R * H, N, P) if S is None else S.reshape(R * H, N, P)
    out = []
    for c in range(n):
        U = U0[:, c] - W[:, c] @ S
        out.append(qe[:, c] @ S + A[:, c] @ U)
        S = last[:, c, None, None] * S + ktd[:, c] @ U
    o = scale * torch.stack(out, 1).reshape(R, H, n * 64, P)[:, :, :L]
    return o, S.reshape(R, H, N, P)


def _run_plain(s):
    op, case = s["op"], s["case"]
    if op == "fork":
        free = torch.nonzero(s["live"] == 0).reshape(-1)[: s["parents"].numel()]
        for x in s["pool"]:
            x[free] = x[s["parents"].long()]
        live = s["live"].clone()
        live[free] = 1
        return {"pool": s["pool"], "children": free.to(torch.int32), "live": live}
    if op == "copy":
        for a, b in zip(s["pool"], s["to"]):
            b[s["dst"].long()] = a[s["src"].long()]
        return {"to": s["to"]}
    if op == "compact":
        on = s["live"] != 0
        n = on.sum()
        at = torch.arange(on.numel(), device="cuda")
        holes, moved = torch.nonzero(~on & (at < n)).reshape(-1), torch.nonzero(on & (at >= n)).reshape(-1)
        for x in s["pool"]:
            x[holes] = x[moved]
        new = torch.where(on, at, -1)
        new[moved] = holes
        return {"pool": s["pool"], "new_slot": new.to(torch.int32), "count": n.reshape(1).to(torch.int32)}

    if op == "step":
        reach = case["heads"] // case["groups"]
        q, k = (_rows(x, case["l2norm"]).repeat_interleave(reach, dim=1) for x in (s["q"], s["k"]))
        at = slice(None) if s["slots"] is None else s["slots"].long()
        S = s["h"][at] * torch.exp(s["g"])[..., None, None]
        u = s["beta"][..., None] * (s["v"].float() - (S * k[..., None]).sum(-2))
        S = S + k[..., None] * u[..., None, :]
        s["h"][at] = S
        return {"o": (s["scale"] * (S * q[..., None]).sum(-2)).to(s["v"].dtype), "h": s["h"]}

    if op == "prefill":
        ops = _heads_first(s, _rows(s["q"], case["l2norm"]), _rows(s["k"], case["l2norm"]), s["v"].float(), s["g"].double(), s["beta"])
        S = s["h"]
        if s["slots"] is not None:
            S = S[s["slots"].long()]
        o, S = _plain_delta(*ops, S, s["scale"])
        o = o.transpose(1, 2)
        if s["cu"] is not None:
            _, real = _unpack(s)
            o = o[real][None]
        if s["slots"] is not None:
            s["h"][s["slots"].long()] = S
            S = s["h"]
        return {"o": o.to(s["v"].dtype).contiguous(), "h": S}

    leaves = [s[n].float().requires_grad_() for n in ("q", "k", "v")]
    leaves += [s["g"].double().requires_grad_(), s["beta"].clone().requires_grad_()]
    rows = case["packed"] or case["batch"]
    h = torch.zeros_like(s["dh"]) if s["h"] is None else s["h"].clone()
    leaves.append(h.requires_grad_())
    q, k, v, g, beta, h = leaves
    o, S = _plain_delta(*_heads_first(s, _rows(q, case["l2norm"]), _rows(k, case["l2norm"]), v, g, beta), h, s["scale"])
    o = o.transpose(1, 2)
    if s["cu"] is not None:
        _, real = _unpack(s)
        o = o[real][None]
    grads = torch.autograd.grad([o, S], leaves, [s["do"].float(), s["dh"]])
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dh"), (x.float() for x in grads)))


# ------------------------------------------------------------------ the work

def work(case):
    if case["op"] in ("fork", "copy", "compact"):
        record = case["heads"] * (4 * case["dstate"] * case["headdim"]
                                  + (2 * case["rank"] * (case["dstate"] + case["headdim"]) if case["mixer"] else 0))
        n = case["count"]
        if case["op"] == "compact":   # live records past the front, as many as the front has holes: on average
            n = n * (case["slots"] - n) / case["slots"]
        return {"bytes": 2 * n * record + 4 * case["slots"], "flops": 0}
    B, L, H, G, N, P = (case[k] for k in ("batch", "seqlen", "heads", "groups", "dstate", "headdim"))
    e = 4 if case["io"] == "f32" else 2
    rows = case["packed"] or B
    state = 4 * rows * H * N * P
    tok = B * L
    if case["op"] == "step":
        return {"bytes": 2 * state + tok * (2 * G * N * e + 2 * H * P * e + 8 * H), "flops": 7 * rows * H * N * P}
    # a chunk of 64 and a head: k k^T, q k^T, the triangular solve, and five products with the state or the chunk
    fwd = 2 * 64 * N + 64 * N + 64 * 64 / 3 + 3 * 64 * P + 6 * N * P
    if case["op"] == "prefill":
        return {"bytes": tok * (2 * G * N * e + 2 * H * P * e + 8 * H) + state * (2 if case["state"] else 1), "flops": tok * H * fwd}
    return {"bytes": tok * (2 * G * N * (e + 4) + H * P * (2 * e + 4) + 16 * H) + state * (3 if case["state"] else 2),
            "flops": tok * H * (3 * fwd)}


# ----------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("fork", "copy", "compact"):
        return None   # records are moved, nothing is computed
    H, G, N, P = (case[k] for k in ("heads", "groups", "dstate", "headdim"))

    def unit(x):
        x = x.double()
        return x / (x.pow(2).sum(-1, keepdim=True) + EPS).sqrt() if case["l2norm"] else x

    head_of = torch.arange(H, device="cuda") // (H // G)
    q, k, v, g, beta = unit(s["q"]), unit(s["k"]), s["v"].double(), s["g"].double(), s["beta"].double()
    if op == "step":
        q, k, v, g, beta = (x[:, None] for x in (q, k, v, g, beta))
    # tokens first, one row per sequence; past a sequence's end nothing decays and nothing is written
    if s["cu"] is not None:
        nseq, top = len(s["lens"]), max(s["lens"])
        q, k, v, g, beta = (torch.stack([torch.cat([x[0, a:a + n], x.new_zeros(top - n, *x.shape[2:])])
                                         for a, n in zip(s["cu"].tolist(), s["lens"])]) for x in (q, k, v, g, beta))
    q, k = q[:, :, head_of], k[:, :, head_of]
    rows, T = q.shape[:2]
    at = torch.arange(rows, device="cuda") if s["slots"] is None else s["slots"].long()
    S = torch.zeros(rows, H, N, P, dtype=torch.float64, device="cuda") if s["h"] is None else s["h"].double()[at]
    a = g.exp()
    if op != "gradient":
        o = torch.empty(rows, T, H, P, dtype=torch.float64, device="cuda")
        for t in range(T):
            S = S * a[:, t, :, None, None]
            u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2))
            S = S + k[:, t, :, :, None] * u[:, :, None, :]
            o[:, t] = s["scale"] * (S * q[:, t, :, :, None]).sum(2)
        if op == "step":
            o = o[:, 0]
        elif s["cu"] is not None:
            o = torch.cat([o[i, :n] for i, n in enumerate(s["lens"])])[None]
        if s["slots"] is not None:
            h = s["h"].double()
            h[at] = S
            S = h
        return {"o": o, "h": S}

    do = s["do"].double()
    if s["cu"] is not None:
        do = torch.stack([torch.cat([do[0, b:b + n], do.new_zeros(top - n, H, P)]) for b, n in zip(s["cu"].tolist(), s["lens"])])
    before, us = [], []
    for t in range(T):
        before.append(S)
        S = S * a[:, t, :, None, None]
        us.append(beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2)))
        S = S + k[:, t, :, :, None] * us[-1][:, :, None, :]
    dS = s["dh"].double()
    dq, dk, dv, dg, db = (torch.empty_like(x) for x in (q, k, v, g, beta))
    for t in reversed(range(T)):
        kt, qt = k[:, t, :, :, None], q[:, t, :, :, None]
        Sa = before.pop() * a[:, t, :, None, None]
        u = us.pop()
        St = Sa + kt * u[:, :, None, :]
        go = s["scale"] * do[:, t, :, None, :]
        dq[:, t] = (St * go).sum(3)
        dS = dS + qt * go
        du = (dS * kt).sum(2)
        dk[:, t] = (dS * u[:, :, None, :]).sum(3)
        dv[:, t] = beta[:, t, :, None] * du
        db[:, t] = (du * (v[:, t] - (Sa * kt).sum(2))).sum(2)
        dp = -dv[:, t][:, :, None, :]
        dS = dS + kt * dp
        dk[:, t] += (Sa * dp).sum(3)
        dg[:, t] = (dS * Sa).sum((2, 3))
        dS = dS * a[:, t, :, None, None]

    def back(x):
        return x if s["cu"] is None else torch.cat([x[i, :n] for i, n in enumerate(s["lens"])])[None]

    def rows_back(raw, d):
        raw, d = raw.double(), back(d)
        d = d.reshape(*d.shape[:2], G, H // G, N).sum(3)
        if not case["l2norm"]:
            return d
        r = (raw.pow(2).sum(-1, keepdim=True) + EPS).rsqrt()
        x = raw * r
        return r * (d - x * (x * d).sum(-1, keepdim=True))

    return {"dq": rows_back(s["q"], dq), "dk": rows_back(s["k"], dk), "dv": back(dv), "dg": back(dg), "dbeta": back(db), "dh": dS}
