"""hss_evict_blocks against a plain sort (the result is exact, no tolerance)."""
import numpy as np
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_block_lowrank_gb300 import _build

    _build.build()
    hss.load()


def plain(w, table, lengths, ctx, budgets, bs, first, last):
    stay_t, stay_w, freed, offs, foffs, nctx = [], [], [], [0], [0], []
    at = 0
    for s, n in enumerate(lengths):
        part, ids = w[at:at + n], table[at:at + n]
        at += n
        hi = n - last if ctx is None else min(n - last, max(int(ctx[s]), 0) // bs)
        cand = list(range(min(first, n), max(hi, min(first, n))))
        lost = min(max(n - max(int(budgets[s]), 0), 0), len(cand))

        def key(j):
            x = float(part[j])
            return (np.inf if np.isnan(x) else x + 0.0, j)

        gone = set(sorted(cand, key=key)[:lost])
        for j in range(n):
            (freed if j in gone else stay_t).append(int(ids[j]))
            if j not in gone:
                stay_w.append(part[j])
        offs.append(len(stay_t))
        foffs.append(len(freed))
        nctx.append(0 if ctx is None else int(ctx[s]) - lost * bs)
    return stay_t, stay_w, freed, offs, foffs, nctx


def run(w, table, lengths, ctx, budgets, bs, first, last):
    total, S = len(w), len(lengths)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    offs = i32([0] + np.cumsum(lengths).tolist())
    nt, fr = i32([99] * total), i32([99] * total)
    nw = torch.full((total,), 99.0, device=DEV)
    no, fo, nc = i32([99] * (S + 1)), i32([99] * (S + 1)), i32([99] * S)
    hss.hss_evict_blocks(torch.tensor(w, device=DEV), i32(table), offs,
                         None if ctx is None else i32(ctx), i32(budgets), S, total, bs, first, last,
                         nt, no, nw, None if ctx is None else nc, fr, fo)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (nt, nw, fr, no, fo, nc)]


def check(w, lengths, ctx, budgets, bs, first, last, seed=0):
    w = np.asarray(w, dtype=np.float32)
    table = np.random.default_rng(seed).permutation(len(w) + 5)[:len(w)]
    want = plain(w, table, lengths, ctx, budgets, bs, first, last)
    nt, nw, fr, no, fo, nc = run(w, table, lengths, ctx, budgets, bs, first, last)
    k, f = len(want[0]), len(want[2])
    assert no.tolist() == want[3] and fo.tolist() == want[4]
    assert nt[:k].tolist() == want[0] and (nt[k:] == -1).all()
    assert np.array_equal(nw[:k].view(np.int32), np.asarray(want[1], np.float32).view(np.int32))
    assert (nw[k:] == 0).all()
    assert fr[:f].tolist() == want[2] and (fr[f:] == -1).all()
    if ctx is not None:
        assert nc.tolist() == want[5]


@pytest.mark.parametrize("lengths", [
    [1], [2], [31], [32], [33], [511], [512], [513], [8191], [8192], [8193], [0, 5, 0, 300, 1],
    [16385], [40000], [70000], [131073], [20000] + [3] * 40, [65536] * 3])
@pytest.mark.parametrize("share", [0.0, 0.5, 0.97])
def test_evict_lengths(lengths, share):
    rng = np.random.default_rng(sum(lengths))
    w = rng.lognormal(0, 2, sum(lengths))
    w[rng.random(len(w)) < 0.1] = 0.0
    bs = 16
    ctx = [max(0, n * bs - int(rng.integers(0, 2 * bs))) for n in lengths]
    check(w, lengths, ctx, [int(n * share) for n in lengths], bs, 1, 2)


def test_evict_ties_and_special_weights():
    special = [0.0, -0.0, np.nan, np.inf, -np.inf, 1.0, 1.0, np.float32(1e-45), -1.0, 3e38]
    rng = np.random.default_rng(3)
    w = rng.choice(np.asarray(special, np.float32), 3000)
    for budget in (0, 1, 5, 1499, 1500, 2999, 3000, 5000, -4):
        check(w, [1000, 1700, 300], None, [budget // 3, budget // 2, budget], 16, 0, 0)
    check(np.full(50000, 2.5), [50000], None, [123], 16, 7, 9)  # one key: ties all the way
    check(np.full(9000, np.nan), [9000], None, [8000], 32, 0, 0)


def test_evict_protected_ends():
    rng = np.random.default_rng(4)
    w = rng.random(400)
    for first, last in ((0, 0), (4, 4), (100, 0), (0, 100), (60, 60), (1000, 0), (0, 1000)):
        check(w, [100, 100, 200], [1600, 37, 0], [10, 10, 10], 16, first, last)
        check(w, [100, 100, 200], None, [10, 99, 300], 16, first, last)


def test_evict_many_sequences():
    rng = np.random.default_rng(5)
    lengths = rng.integers(0, 90, 2500).tolist()
    w = rng.random(sum(lengths))
    check(w, lengths, [n * 16 for n in lengths], rng.integers(0, 90, 2500).tolist(), 16, 1, 1)


def test_evict_repeats_on_another_stream():
    rng = np.random.default_rng(6)
    w = torch.tensor(rng.random(30000), dtype=torch.float32, device=DEV)
    table = torch.arange(30000, dtype=torch.int32, device=DEV)
    offs = torch.tensor([0, 10000, 30000], dtype=torch.int32, device=DEV)
    budgets = torch.tensor([77, 9000], dtype=torch.int32, device=DEV)
    outs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        nt, fr = torch.empty_like(table), torch.empty_like(table)
        nw, no, fo = torch.empty_like(w), torch.empty_like(offs), torch.empty_like(offs)
        hss.hss_evict_blocks(w, table, offs, None, budgets, 2, 30000, 16, 1, 1, nt, no, nw, None,
                             fr, fo, stream)
        outs.append((nt, nw, fr, no, fo))
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
