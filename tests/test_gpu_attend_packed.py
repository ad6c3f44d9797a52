"""hss_attend_packed against softmax and sums in 64 bits over the cache's values.

Tolerances, from the kernels' arithmetic.  A weight times its value's scale is rounded to bf16, half
a step or 2^-8 of it at most (many rows: the weight alone, to fp16), and the result once more: 2^-8
sum p |v| + 2^-8 |out|, where |out| <= sum p |v|.  A score is a sum of head_dim exact products in fp32, off by less than (head_dim + 8)
2^-23 of the sum of their sizes; exp2 and the sums of up to a few hundred weights a thread add less
than 4e-5: that much of lse, and of sum p |v| once more.
"""
import numpy as np
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss
import packed_util as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_block_lowrank_gb300 import _build

    _build.build()
    hss.load()


class Case:
    def __init__(self, hd, nq, nkv, bs, ctx, rows, window=0, sinks=0, scale=None, spare=3, seed=0,
                 short=0, max_q=None, pages_at=0):
        self.hd, self.nq, self.nkv, self.bs = hd, nq, nkv, bs
        self.ctx, self.rows, self.window, self.sinks = ctx, rows, window, sinks
        self.scale = hd ** -0.5 if scale is None else scale
        g = torch.Generator().manual_seed(seed + hd + sum(ctx) + sum(rows))
        n = [max(0, -(-(max(c, 0) + r) // bs) - short) for c, r in zip(ctx, rows)]
        total = sum(n)
        self.max_blocks = total + spare + pages_at
        self.table = pages_at + torch.randperm(total + spare, generator=g)[:total].int()
        self.offs = torch.tensor([0] + np.cumsum(n).tolist(), dtype=torch.int32)
        self.q_offs = torch.tensor([0] + np.cumsum(rows).tolist(), dtype=torch.int32)
        self.total_q, self.total = sum(rows), total
        self.max_q = max_q or max(rows + [1])
        self.dims = hss.hss_dims(1, nq, nkv, hd, 16, bs, self.max_blocks)
        size = hss.hss_packed_page_bytes(self.dims)
        gd = torch.Generator(device=DEV).manual_seed(seed + 1)
        tiles = (total + spare) * nkv * (bs // 16)
        cache = torch.randint(0, 256, (tiles, P.tile_bytes(hd)), generator=gd, device=DEV,
                              dtype=torch.uint8)
        scales = torch.rand(tiles, hd, generator=gd, device=DEV) * 0.5 + 0.02
        cache[:, 16 * hd:] = scales.bfloat16().view(torch.uint8)
        self.cache = cache.view(total + spare, size)
        if pages_at:
            whole = torch.empty(self.max_blocks, size, device=DEV, dtype=torch.uint8)
            whole[pages_at:] = self.cache
            self.cache = whole
        self.q = torch.randn(self.total_q, nq, hd, generator=gd, device=DEV).bfloat16()

    def call(self, work=None, status=None, table=None, cache=None, ctx=None):
        size = hss.hss_attend_packed_workspace_bytes(self.dims, len(self.ctx), self.max_q,
                                                     self.total, self.window, self.sinks)
        if work is None:
            work = torch.full((size,), 0xFF, device=DEV, dtype=torch.uint8)
        self.kept = hss.AttendPacked(
            self.dims, self.q_offs.to(DEV), self.total_q, self.max_q,
            (self.table if table is None else table).to(DEV), self.offs.to(DEV),
            torch.tensor(self.ctx if ctx is None else ctx, dtype=torch.int32, device=DEV),
            len(self.ctx), self.total, self.window, self.sinks, self.scale, work, work.numel(),
            status)
        out = torch.full_like(self.q, 7.0)
        lse = torch.full((self.total_q, self.nq), 7.0, device=DEV)
        self.kept(self.q, self.cache if cache is None else cache, out, lse)
        return out, lse

    def check(self, out, lse, table=None, cache=None):
        table = (self.table if table is None else table).numpy()
        cache = self.cache if cache is None else cache
        offs, q_offs = self.offs.tolist(), self.q_offs.tolist()
        for s, (c, r) in enumerate(zip(self.ctx, self.rows)):
            a, b = q_offs[s], q_offs[s + 1]
            want, ln, size, most = P.attend(
                self.q[a:b].double().cpu().numpy(), cache, self.nkv, self.bs, self.hd,
                table[offs[s]:offs[s + 1]], max(c, 0), r, self.window, self.sinks, self.scale,
                self.max_blocks)
            slack = 4e-5 + (self.hd + 8) * 2.0 ** -23 * most
            got = out[a:b].double().cpu().numpy()
            room = 2.0 ** -8 * (size + np.abs(want)) + 2 * slack[..., None] * size
            assert (np.abs(got - want) <= room).all(), (s, np.abs(got - want).max())
            got = lse[a:b].double().cpu().numpy()
            none = np.isneginf(ln)
            assert (np.isneginf(got) == none).all(), s
            off = np.abs(np.where(none, 0, got) - np.where(none, 0, ln))
            assert (off <= slack + 2.0 ** -23 * np.abs(np.where(none, 0, ln))).all(), (s, off.max())


CASES = [
    dict(hd=128, nq=32, nkv=8, bs=16, ctx=[1000], rows=[1]),
    dict(hd=128, nq=4, nkv=4, bs=16, ctx=[0, 1, 15, 16, 17, 300], rows=[1] * 6),
    dict(hd=64, nq=9, nkv=3, bs=32, ctx=[0, 77, 5, 200, 0], rows=[1, 7, 0, 3, 2]),
    dict(hd=64, nq=8, nkv=1, bs=48, ctx=[513], rows=[2]),
    dict(hd=128, nq=16, nkv=1, bs=64, ctx=[100, 40], rows=[1, 1]),
    dict(hd=192, nq=6, nkv=2, bs=16, ctx=[333, 31], rows=[5, 1]),
    dict(hd=192, nq=2, nkv=2, bs=128, ctx=[129], rows=[1]),
    dict(hd=256, nq=8, nkv=2, bs=16, ctx=[250, 2], rows=[1, 2]),
    dict(hd=256, nq=10, nkv=2, bs=256, ctx=[700], rows=[4]),
    dict(hd=128, nq=5, nkv=1, bs=16, ctx=[90, 0], rows=[61, 130]),
    dict(hd=64, nq=14, nkv=2, bs=16, ctx=[200], rows=[40]),
    dict(hd=128, nq=128, nkv=1, bs=16, ctx=[50], rows=[3]),
    # many rows: one and several row tiles, ends inside a job, rows of nothing among them
    dict(hd=64, nq=4, nkv=1, bs=32, ctx=[700, 0, 33], rows=[9, 150, 0]),
    dict(hd=128, nq=8, nkv=1, bs=16, ctx=[1000], rows=[100]),
    dict(hd=128, nq=3, nkv=1, bs=48, ctx=[65, 400], rows=[13, 90]),
    dict(hd=192, nq=8, nkv=2, bs=16, ctx=[129, 5], rows=[40, 70]),
    dict(hd=256, nq=4, nkv=1, bs=16, ctx=[300, 64], rows=[50, 9]),
    dict(hd=256, nq=1, nkv=1, bs=128, ctx=[77], rows=[140]),
    dict(hd=128, nq=2, nkv=2, bs=16, ctx=[50, 60, 70, 80] * 10, rows=[20, 17, 1, 33] * 10),
    dict(hd=64, nq=2, nkv=2, bs=32, ctx=[600, 20], rows=[130, 200], window=100, sinks=20),
    dict(hd=128, nq=8, nkv=1, bs=16, ctx=[900], rows=[80], window=256, sinks=4),
    dict(hd=256, nq=2, nkv=1, bs=16, ctx=[333], rows=[66], window=1, sinks=0),
    dict(hd=192, nq=5, nkv=1, bs=64, ctx=[700], rows=[30], window=64, sinks=100),
    dict(hd=128, nq=4, nkv=1, bs=16, ctx=[100], rows=[30], scale=-0.2),
    dict(hd=64, nq=4, nkv=1, bs=16, ctx=[100], rows=[30], scale=0.0),
    dict(hd=64, nq=4, nkv=1, bs=32, ctx=[5000], rows=[70]),
    dict(hd=128, nq=4, nkv=1, bs=16, ctx=[5000], rows=[70]),
    dict(hd=192, nq=4, nkv=1, bs=16, ctx=[5000], rows=[40]),
    dict(hd=256, nq=4, nkv=1, bs=16, ctx=[5000], rows=[40]),
    # windows: shorter and longer than a tile, than the rows; sinks inside the window
    dict(hd=128, nq=8, nkv=2, bs=16, ctx=[500, 3, 0], rows=[1, 1, 1], window=100, sinks=4),
    dict(hd=64, nq=4, nkv=4, bs=32, ctx=[300], rows=[9], window=1, sinks=0),
    dict(hd=64, nq=4, nkv=4, bs=32, ctx=[300], rows=[9], window=1, sinks=1),
    dict(hd=128, nq=6, nkv=2, bs=16, ctx=[200, 64], rows=[70, 33], window=40, sinks=17),
    dict(hd=128, nq=8, nkv=8, bs=48, ctx=[700, 10], rows=[2, 3], window=129, sinks=400),
    dict(hd=192, nq=3, nkv=1, bs=16, ctx=[260], rows=[20], window=16, sinks=16),
    dict(hd=256, nq=4, nkv=1, bs=64, ctx=[1000], rows=[6], window=333, sinks=33),
    dict(hd=128, nq=2, nkv=1, bs=16, ctx=[100], rows=[5], window=2 ** 31 - 1, sinks=2 ** 31 - 1),
    # other scales
    dict(hd=64, nq=4, nkv=2, bs=16, ctx=[140], rows=[3], scale=-0.3),
    dict(hd=128, nq=4, nkv=2, bs=16, ctx=[140], rows=[3], scale=0.0),
    dict(hd=128, nq=4, nkv=2, bs=16, ctx=[400], rows=[3], scale=2.0),
    # a negative context counts as none
    dict(hd=64, nq=2, nkv=2, bs=16, ctx=[-5, 20], rows=[4, 1]),
]


@pytest.mark.parametrize("kw", CASES)
def test_against_64_bits(kw):
    c = Case(**kw)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = c.call(status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    c.check(out, lse)


@pytest.mark.parametrize("rows", [1, 8])
def test_long_and_short_together(rows):
    """Ranges that begin and end inside sequences, units that several CTAs share, and whole ones."""
    g = np.random.default_rng(rows)
    ctx = [5000] + g.integers(0, 200, 150).tolist() + [3000, 0, 1]
    c = Case(64, 4, 2, 16, ctx, g.integers(0, rows + 1, len(ctx)).tolist(), max_q=rows)
    first = c.call()
    second = c.call(work=torch.zeros(1 << 23, device=DEV, dtype=torch.uint8))
    torch.cuda.synchronize()
    c.check(*first)
    for a, b in zip(first, second):
        assert torch.equal(a, b)  # the same bits, whatever the workspace holds


@pytest.mark.parametrize("hd,nq,nkv,seqs,rows", [(64, 2, 1, 700, 1), (128, 4, 2, 530, 2),
                                                (256, 2, 2, 300, 1), (128, 32, 2, 20, 1)])
@pytest.mark.parametrize("window", [20, 700])
def test_windows_of_many_short_sequences(hd, nq, nkv, seqs, rows, window):
    """Around the number of units and the length from which on they are listed."""
    g = np.random.default_rng(seqs + window)
    ctx = g.integers(0, 400 if seqs > 100 else 3000, seqs).tolist()
    c = Case(hd, nq, nkv, 32, ctx, g.integers(0, rows + 1, seqs).tolist(), window=window, sinks=5,
             max_q=rows)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = c.call(status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    c.check(out, lse)


@pytest.mark.parametrize("hd,window,more", [(64, 0, 1), (128, 50, 1), (256, 0, 1), (64, 50, 20),
                                            (128, 0, 20), (192, 50, 20), (256, 0, 20)])
def test_hidden_places_hold_anything(hd, window, more):
    """NaN scales past the end, in front of the window and in rows' futures; pages that no row sees
    with ids that do not exist."""
    c = Case(hd, 4, 2, 16, [130, 40, 7], [3 * more, 2 * more, more], window=window,
             sinks=3 if window else 0)
    clean = [t.clone() for t in c.call()]
    cache = c.cache.clone().view(c.max_blocks, 2, 1, -1)
    table, offs = c.table.clone(), c.offs.tolist()
    nan = torch.tensor([float("nan")], dtype=torch.bfloat16, device=DEV).view(torch.uint8)
    spoiled = 0
    for s in range(3):
        for e in range(offs[s], offs[s + 1]):
            for t in range(16):
                pos = (e - offs[s]) * 16 + t
                first = c.ctx[s]
                seen = pos < first + c.rows[s] and (
                    not window or pos < c.sinks or pos > first - window)
                if not seen:
                    spoiled += 1
                    tile = cache[table[e].item(), :, 0]
                    for value in (False, True):
                        at = 2 * P.scale_place(t, 0, hd, value)
                        tile[:, at:at + hd // 16] = nan.repeat(hd // 32)
    assert spoiled > 0
    if window:
        for s in range(3):
            for e in range(offs[s], offs[s + 1]):
                last = (e - offs[s]) * 16 + 15
                if last <= c.ctx[s] - window and last - 15 >= c.sinks:
                    table[e] = -7 if e % 2 else 1 << 30
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = c.call(table=table, cache=cache, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for a, b in zip(got, clean):
        assert torch.equal(a, b)


def test_a_row_sees_no_later_rows_values():
    """A NaN in the second row's own token reaches that row and those behind it, not the first."""
    hd = 128
    c = Case(hd, 2, 1, 16, [20], [4])
    cache = c.cache.clone()
    t = 21
    tile = cache[c.table[t // 16].item()]
    nan = torch.tensor([float("nan")], dtype=torch.bfloat16, device=DEV).view(torch.uint8)
    at = 2 * P.scale_place(t % 16, 1, hd, True)
    tile[at:at + 2] = nan
    out, lse = c.call(cache=cache)
    torch.cuda.synchronize()
    got = out.cpu()
    assert torch.isfinite(got[0]).all() and torch.isfinite(lse.cpu()).all()
    assert torch.isnan(got[1:, :, 32:64]).all()
    assert torch.isfinite(got[1:, :, :32]).all() and torch.isfinite(got[1:, :, 64:]).all()


@pytest.mark.parametrize("hd,value,scale", [
    (128, True, float("nan")), (64, False, float("nan")), (256, True, 1000.0),
    (128, False, 2.0 ** -20), (192, True, 2.0 ** 30), (128, False, 3.0e38)])
def test_scales_that_fp16_has_no_place_for(hd, value, scale):
    """Many rows, one group of one token with a scale outside what the tensor cores' operands hold:
    rows before the token as without it, the others as the definition has them."""
    c = Case(hd, 4, 1, 16, [40, 90], [30, 40])
    clean = [t.clone() for t in c.call()]
    cache = c.cache.clone()
    t = 40 + 11                                    # the first sequence's row 11
    tile = cache[c.table[t // 16].item()].view(-1)
    at = 2 * P.scale_place(t % 16, 1, hd, value)
    tile[at:at + 2] = torch.tensor([scale], dtype=torch.bfloat16, device=DEV).view(torch.uint8)
    byte, _ = (P.value_place if value else P.key_place)(t % 16, 32, hd)
    out, lse = c.call(cache=cache)
    torch.cuda.synchronize()
    assert hss.hss_read_device_error() == 0
    if scale != scale:
        got = out.cpu()
        assert torch.isfinite(got[:11]).all() and torch.isfinite(got[30:]).all()
        if value:
            assert torch.isnan(got[11:30, :, 32:64]).all()
            assert torch.isfinite(got[11:30, :, :32]).all()
        else:
            assert torch.isnan(got[11:30]).all() and torch.isnan(lse.cpu()[11:30]).all()
        for a, b in zip((out, lse), clean):
            assert torch.allclose(a[:11].float(), b[:11].float(), atol=0.05)
    elif scale < 1e10:
        c.check(out, lse, cache=cache)
    else:
        assert torch.isfinite(out.cpu()[:11].float()).all()
        assert torch.isfinite(out.cpu()[30:].float()).all()


@pytest.mark.parametrize("hd,value,scale", [
    (64, True, 1000.0), (128, False, 2.0 ** -20), (192, True, 1000.0), (256, False, 2.0 ** -20)])
def test_such_a_scale_in_a_long_context(hd, value, scale):
    """The same where several CTAs share a row, so that the second attempt's pieces are joined."""
    c = Case(hd, 8, 2, 16, [5000, 3], [70, 12])
    cache = c.cache.clone()
    at = 2 * P.scale_place(4000 % 16, 1, hd, value)
    tile = cache[c.table[4000 // 16].item()].view(-1)
    tile[at:at + 2] = torch.tensor([scale], dtype=torch.bfloat16, device=DEV).view(torch.uint8)
    out, lse = c.call(cache=cache)
    torch.cuda.synchronize()
    assert hss.hss_read_device_error() == 0
    c.check(out, lse, cache=cache)
    assert torch.equal(out, c.call(cache=cache)[0])


def test_device_errors_hide_tokens():
    c = Case(128, 4, 2, 16, [100, 60], [2, 2])
    table = c.table.clone()
    table[2], table[9] = -1, c.max_blocks
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = c.call(table=table, status=status)
    torch.cuda.synchronize()
    assert status.item() == hss.HSS_ERR_OUT_OF_RANGE
    assert hss.hss_read_device_error() == hss.HSS_ERR_OUT_OF_RANGE
    c.check(out, lse, table=table)
    c = Case(128, 4, 1, 16, [100, 60], [20, 12])
    table = c.table.clone()
    table[2], table[9] = -1, c.max_blocks
    status.zero_()
    out, lse = c.call(table=table, status=status)
    torch.cuda.synchronize()
    assert status.item() == hss.HSS_ERR_OUT_OF_RANGE == hss.hss_read_device_error()
    c.check(out, lse, table=table)
    # tables too short: one that ends before the rows, and a sequence without any
    for kw in (dict(ctx=[100, 40], rows=[2, 3]), dict(ctx=[10, 3], rows=[1, 2])):
        c = Case(64, 4, 2, 16, short=1, **kw)
        status.zero_()
        out, lse = c.call(status=status)
        torch.cuda.synchronize()
        assert status.item() == hss.HSS_ERR_OUT_OF_RANGE
        c.check(out, lse)
    assert torch.isneginf(lse).all() and (out == 0).all()
    # more rows than max_q: those past it are left as they were
    c = Case(64, 2, 2, 16, [30, 30], [6, 4])
    c.max_q, status[0] = 5, 0
    out, lse = c.call(status=status)
    torch.cuda.synchronize()
    assert status.item() == hss.HSS_ERR_INVALID_ARGUMENT
    assert (out[5] == 7).all() and (lse[5] == 7).all()
    hss.hss_read_device_error()


def test_many_rows_captured_and_repeated():
    """The same bits on every call and replay, whatever the workspace held."""
    c = Case(128, 8, 2, 16, [3000, 500], [90, 40], window=700, sinks=9)
    first = [t.clone() for t in c.call()]
    c.check(*first)
    work = torch.zeros(1 << 27, device=DEV, dtype=torch.uint8)
    second = c.call(work=work)
    torch.cuda.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    out, lse = torch.empty_like(c.q), torch.empty_like(first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.kept(c.q, c.cache, out, lse)
        c.kept(c.q, c.cache, out, lse)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (out, lse)):
        assert torch.equal(a, b)


def test_captured_replayed_and_on_two_streams():
    """A captured call follows what its tensors hold; calls on two streams, each with a workspace."""
    c = Case(128, 8, 2, 16, [700, 100], [1, 1], window=300, sinks=5)
    c.call()
    torch.cuda.synchronize()
    q, out = c.q.clone(), torch.empty_like(c.q)
    lse = torch.empty(c.total_q, c.nq, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.kept(q, c.cache, out, lse)
    for seed in range(2):
        q.normal_(generator=torch.Generator(device=DEV).manual_seed(seed))
        graph.replay()
        c.q = q
        torch.cuda.synchronize()
        c.check(out, lse)
    cases = [Case(64, 4, 2, 16, [900 + i], [2], seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for x, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(x.call())
        torch.cuda.synchronize()
        for x, y in zip(cases, got):
            x.check(*y)


@pytest.mark.parametrize("hd,rows", [(128, [1, 1]), (64, [2, 1]), (128, [70, 12])])
def test_long_contexts_replayed_with_other_lengths_and_scales(hd, rows):
    """A graph over one workspace follows the lengths and the cache from replay to replay: nothing is
    left of a replay that cut its sequences elsewhere or that had to run by the other method."""
    c = Case(hd, 8, 2, 16, [5000, 900], rows)
    c.call()
    ctx = torch.tensor(c.ctx, dtype=torch.int32, device=DEV)
    size = hss.hss_attend_packed_workspace_bytes(c.dims, 2, c.max_q, c.total, 0, 0)
    work = torch.full((size,), 0xFF, device=DEV, dtype=torch.uint8)
    call = hss.AttendPacked(c.dims, c.q_offs.to(DEV), c.total_q, c.max_q, c.table.to(DEV),
                            c.offs.to(DEV), ctx, 2, c.total, 0, 0, c.scale, work, size)
    out, lse = torch.empty_like(c.q), torch.empty(c.total_q, c.nq, device=DEV)
    at = 2 * P.scale_place(3, 0, hd, True)
    tile = c.cache[c.table[1].item()].view(-1)      # tokens 16 to 31 of the first sequence
    fit = tile[at:at + 2].clone()
    unfit = torch.tensor([1000.0], dtype=torch.bfloat16, device=DEV).view(torch.uint8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c.q, c.cache, out, lse)
    for lengths, scale in (([5000, 900], fit), ([40, 0], unfit), ([5000, 900], unfit),
                           ([0, 900], fit), ([4987, 1], fit)):
        c.ctx = lengths
        ctx.copy_(torch.tensor(lengths, dtype=torch.int32))
        tile[at:at + 2] = scale
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert hss.hss_read_device_error() == 0
        c.check(out, lse)


def test_pages_past_32_bits():
    """Pages whose bytes lie behind the first 2^32 of the cache."""
    hd, nkv, bs = 128, 8, 256
    page = nkv * 16 * P.tile_bytes(hd)
    c = Case(hd, 8, nkv, bs, [600], [2], pages_at=(1 << 32) // page + 5)
    out, lse = c.call()
    torch.cuda.synchronize()
    small = c.cache[(1 << 32) // page + 5:].clone()
    table = c.table - ((1 << 32) // page + 5)
    c.check(out, lse, table=table, cache=small)


def test_no_lse_and_no_rows():
    c = Case(128, 4, 2, 16, [50, 20], [1, 0])
    out, lse = c.call()
    again = torch.zeros_like(out)
    c.kept(c.q, c.cache, again)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
