"""Pools of state records on the GPU: copy, fork, compact and free against the
same on the host, bit for bit, and a run of them between decode steps."""
import pytest
import torch

import delta_reference as ref
from helpers import say
from mamba_selective_ssm_amd import (State, m3_decode_step, m3_delta_fwd, m3_delta_step, m3_pool_compact,
                                     m3_pool_copy, m3_pool_fork, m3_pool_free, zero_state)

pytestmark = pytest.mark.gpu
DEV = "cuda"

# shapes of a record's arrays: the mixers' records, rows of odd byte counts, one larger than a piece by a little
RECORDS = {
    "mamba": [((3, 64, 64), torch.float32), ((3, 2, 64), torch.bfloat16), ((3, 2, 64), torch.bfloat16)],
    "delta": [((2, 32, 32), torch.float32)],
    "odd": [((5,), torch.uint8), ((3, 7), torch.bfloat16), ((9,), torch.float32), ((4097,), torch.float32), ((1,), torch.uint8)],
}


def record(kind, slots, seed):
    gen = torch.Generator().manual_seed(seed)
    return tuple(torch.randint(0, 256, (slots,) + s + (torch.empty(0, dtype=dt).element_size(),), generator=gen,
                               dtype=torch.uint8).view(dt).reshape((slots,) + s).to(DEV) for s, dt in RECORDS[kind])


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def host_copy(src, dst, ss, ds):
    out = [d.clone() for d in dst]
    for s, d in zip(ss, ds):
        if s >= src[0].shape[0] or d < 0 or d >= dst[0].shape[0]:
            continue
        for x, y in zip(src, out):
            y[d] = x[s] if s >= 0 else torch.zeros_like(y[d])
    return out


@pytest.mark.parametrize("kind", list(RECORDS))
def test_copy_to_another_pool(kind):
    src, dst = record(kind, 9, 1), record(kind, 7, 2)
    ss, ds = [8, 0, 3, -1, 5, 9, 2, 2], [0, 6, 1, 2, 0, 3, 7, -2]   # slot 0 twice; 9, 7 and -2 lie outside
    want = host_copy(src, dst, ss, ds)
    m3_pool_copy(src, dst, ints(*ss), ints(*ds))
    assert same(dst, want)


@pytest.mark.parametrize("kind", list(RECORDS))
@pytest.mark.parametrize("ss,ds", [
    ([0, 1], [1, 0]),                                  # swap
    ([0, 1, 2, 3, 4], [1, 2, 3, 4, 0]),                # rotate
    ([0, 0, 0], [1, 2, 3]),                            # one to many
    ([0, 1, 2], [1, 2, 3]),                            # chain
    ([3, 3, 4], [3, 5, 5]),                            # onto itself; one slot twice
    ([-1, 0, 9], [0, 2, 0]),                           # cleared slot that is a source too; a pair outside
    ([1, 5, 1], [5, 1, 5]),                            # swap, one pair twice
])
def test_copy_in_place(kind, ss, ds):
    pool = record(kind, 6, 3)
    want = host_copy([x.clone() for x in pool], pool, ss, ds)
    m3_pool_copy(pool, pool, ints(*ss), ints(*ds))
    assert same(pool, want)


def test_copy_random_in_place_many():
    gen = torch.Generator().manual_seed(4)
    pool = record("odd", 700, 5)
    ss = torch.randint(-1, 720, (1500,), generator=gen).tolist()
    ds = torch.randint(-2, 710, (1500,), generator=gen).tolist()
    want = host_copy([x.clone() for x in pool], pool, ss, ds)
    m3_pool_copy(pool, pool, ints(*ss), ints(*ds))
    assert same(pool, want)


def test_copy_nothing():
    pool = record("delta", 4, 6)
    before = [x.clone() for x in pool]
    m3_pool_copy(pool, pool, ints(), ints())
    assert same(pool, before)


def host_fork(pool, live, parents):
    pool, live = [x.clone() for x in pool], list(live)
    was = list(live)
    children = []
    for p in parents:
        ok = p < 0 or (p < len(was) and was[p])
        free = [i for i, v in enumerate(live) if not v]
        if not ok or not free:
            children.append(-1)
            continue
        c = free[0]
        live[c] = 1
        children.append(c)
        for x in pool:
            x[c] = x[p] if p >= 0 else torch.zeros_like(x[c])
    return pool, live, children


@pytest.mark.parametrize("kind", list(RECORDS))
@pytest.mark.parametrize("live,parents", [
    ([1, 0, 1, 0, 0, 1], [0, 5, 0]),
    ([1, 0, 1, 0, 0, 1], [2, 2, -1, 2, 2]),            # more than are free; a cleared record
    ([1, 0, 1, 0, 0, 1], [1, 7, 0]),                   # a parent that is free, one outside
    ([1, 1, 1, 1, 1, 1], [0]),                         # full
    ([0, 0, 0, 0, 0, 0], [-1, 0, -1]),                 # empty
    ([1, 0, 3, 0, -1, 1], [4]),                        # any value but 0 is live
])
def test_fork(kind, live, parents):
    pool = record(kind, 6, 7)
    want, wl, wc = host_fork(pool, live, parents)
    lv = ints(*live)
    out = torch.empty_like(lv)
    children = m3_pool_fork(pool, lv, ints(*parents), live_out=out)
    assert children.tolist() == wc and out.tolist() == wl and lv.tolist() == live
    assert same(pool, want)
    again = m3_pool_fork(pool, lv, ints(*parents))      # marks changed in place
    assert again.tolist() == wc and lv.tolist() == wl


@pytest.mark.parametrize("slots,share", [(1, 1.0), (1, 0.0), (7, 0.5), (64, 0.1), (1023, 0.7), (1024, 0.5), (5000, 0.3)])
def test_fork_and_compact_of_larger_pools(slots, share):
    gen = torch.Generator().manual_seed(slots)
    pool = record("odd", slots, 8)[:3]
    live = (torch.rand(slots, generator=gen) < share).int().tolist()
    parents = torch.randint(-1, slots + 2, (min(slots, 1500),), generator=gen).tolist()
    want, wl, wc = host_fork(pool, live, parents)
    lv = ints(*live)
    assert m3_pool_fork(pool, lv, ints(*parents)).tolist() == wc
    assert lv.tolist() == wl and same(pool, want)
    want, new, n = host_compact(pool, wl)
    cnt = torch.empty(1, dtype=torch.int32, device=DEV)
    got = m3_pool_compact(pool, lv, count=cnt, live_out=lv)
    assert got.tolist() == new and cnt.item() == n and lv.tolist() == [1] * n + [0] * (slots - n)
    assert all(torch.equal(x[:n].view(torch.uint8), y[:n].view(torch.uint8)) for x, y in zip(pool, want))


def host_compact(pool, live):
    pool = [x.clone() for x in pool]
    n = sum(1 for v in live if v)
    new = [i if v else -1 for i, v in enumerate(live)]
    holes = [i for i in range(n) if not live[i]]
    moved = [i for i in range(n, len(live)) if live[i]]
    for h, m in zip(holes, moved):
        new[m] = h
        for x in pool:
            x[h] = x[m]
    return pool, new, n


@pytest.mark.parametrize("kind", list(RECORDS))
@pytest.mark.parametrize("live", [[0, 1, 1, 0, 1, 1], [1] * 6, [0] * 6, [0, 0, 0, 0, 0, 1], [1, 1, 0, 0, 0, 0], [0, 0, 0, 1, 1, 1]])
def test_compact(kind, live):
    pool = record(kind, 6, 9)
    want, new, n = host_compact(pool, live)
    lv = ints(*live)
    got = m3_pool_compact(pool, lv)
    assert got.tolist() == new and lv.tolist() == live
    assert same(pool, want)


def test_free():
    live = ints(1, 1, 2, 1, 0)
    m3_pool_free(live, ints(2, 2, 4, -1, 5, 0))
    assert live.tolist() == [0, 1, 0, 1, 0]
    m3_pool_free(live, ints())


def test_records_past_two_gib():
    row = 1 << 20
    pool = torch.empty(2300, row, dtype=torch.uint8, device=DEV)
    pool[2299].random_(0, 255)
    pool[0].zero_()
    m3_pool_copy((pool,), (pool,), ints(2299), ints(0))
    assert torch.equal(pool[0], pool[2299])


def test_serving_run_of_both_mixers():
    """Prompts in slots, samples forked, steps, endings, compaction, more
    steps: every sample against its own recurrence; the Mamba-3 records of the
    same slots go along."""
    H, N, P, slots = 2, 64, 64, 8
    pool = torch.zeros(slots, H, N, P, device=DEV)
    m3 = zero_state(slots, H, P, N, 1, torch.bfloat16, DEV)
    gen = torch.Generator().manual_seed(10)
    m3.h.copy_(torch.randn(slots, H, N, P, generator=gen))
    live = torch.zeros(slots, dtype=torch.int32, device=DEV)
    rec = (pool,) + tuple(m3)

    owner = m3_pool_fork(rec, live, ints(-1, -1, -1))
    assert owner.tolist() == [0, 1, 2] and live.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
    assert not pool[:3].any() and not m3.h[:3].any()
    lens = [30, 70, 5]
    x = ref.inputs(1, sum(lens), H, H, N, P, torch.bfloat16, 11)
    cu = ints(0, 30, 100, 105)
    m3_delta_fwd(*x, pool, l2norm=True, scale=1.0, cu_seqlens=cu, slots=owner)
    want = [w[1][0] for w in ref.packed(ref.forward, lens, x, [None], scale=1.0, l2norm=True)]

    kids = m3_pool_fork(rec, live, ints(1, 1))
    assert kids.tolist() == [3, 4]
    want += [want[1].clone(), want[1].clone()]

    def step(seed, names):
        """One token for the slots `names`; names[i] is the index into `want`."""
        sl = ints(*[at[i] for i in names])
        y = ref.inputs(len(names), 1, H, H, N, P, torch.bfloat16, seed, step=True)
        o = m3_delta_step(*y, pool, l2norm=True, scale=1.0, slots=sl)
        wo, wh = ref.forward(*[t[:, None] for t in y], torch.stack([want[i] for i in names]), scale=1.0, l2norm=True)
        assert ref.rel2(o, wo[:, 0]) <= 2.0 ** -8
        for j, i in enumerate(names):
            want[i] = wh[j]

    at = {0: 0, 1: 1, 2: 2, 3: 3, 4: 4}
    for t in range(3):
        step(20 + t, [0, 1, 2, 3, 4])
    m3_pool_free(live, ints(0, 2))
    marks = m3.h[[1, 3, 4]].clone()
    new = m3_pool_compact(rec, live, live_out=live)
    assert new.tolist() == [-1, 1, -1, 0, 2, -1, -1, -1] and live.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
    assert torch.equal(m3.h[[1, 0, 2]], marks)
    at = {1: 1, 3: 0, 4: 2}
    for t in range(3):
        step(30 + t, [4, 1, 3])
    for i, s in at.items():
        e = ref.rel2(pool[s], want[i])
        say("   sequence %d in slot %d: %.2e" % (i, s, e))
        assert e <= 320 * 2.0 ** -24

    # a Mamba-3 decode step on the compacted front of the pool
    n = 3
    front = State(*(t[:n] for t in m3))
    z = [torch.randn(n, H, 1, d, generator=gen).to(torch.bfloat16).to(DEV) for d in (P, N, N)]
    f = [torch.rand(n, H, generator=gen).to(DEV), -torch.ones(H, device=DEV), torch.zeros(n, H, N // 2, device=DEV),
         torch.ones(n, H, device=DEV)]
    y = m3_decode_step(*z, f[0], f[1], f[2], f[3], front)
    assert bool(y.isfinite().all())


def test_captured_and_replayed():
    pool = record("mamba", 12, 12)
    start = [x.clone() for x in pool]
    live = ints(1, 0, 1, 1, 0, 0, 1, 0, 1, 0, 0, 1)
    parents = ints(2, 11, 0)
    out, new, cnt = torch.empty_like(live), torch.empty_like(live), ints(0)
    ss, ds = ints(0, 1, 2), ints(1, 2, 0)
    ch = torch.empty_like(parents)

    def run():
        m3_pool_copy(pool, pool, ss, ds)
        m3_pool_fork(pool, live, parents, children=ch, live_out=out)
        m3_pool_free(out, ss)
        m3_pool_compact(pool, out, new_slot=new, count=cnt, live_out=out)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(3):
        parents.copy_(ints(*[(2, 11, 0), (3, -1, 6), (8, 8, 1)][k]))
        for x, s in zip(pool, start):
            x.copy_(s)
        run()
        want = [x.clone() for x in pool] + [t.clone() for t in (ch, out, new, cnt)]
        for x, s in zip(pool, start):
            x.copy_(s)
        for t in (ch, out, new, cnt):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(list(pool) + [ch, out, new, cnt], want)
