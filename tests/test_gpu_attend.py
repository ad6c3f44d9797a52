"""hss_attend_tree against the definition in 64 bits.

Tolerances, from the kernel's arithmetic.  A score is an fp32 sum of head_dim products: off by
at most e = 2 head_dim 2^-23 scale sum |q k| + 2^-20 (the second term covers the exponential's
argument and the exponential itself), so a weight p is off by a factor within 2 e of 1 and
  lse      within e + 2^-20 |lse|,
  weights  within (2 e + 2^-16) of the weight an entry got, plus fp32 rounding of the old one,
  out      within 2^-8 |out| (its rounding to bf16) + (2^-8 + 2 e) sum p |v| (the weights'
           rounding to bf16 before the product, and their own error).
"""
import math

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


def tree_bits(n, kind, g):
    """[n, n] truth values: which node sees which."""
    see = torch.zeros(n, n, dtype=torch.bool)
    for j in range(n):
        if kind == "tree" and j > 0:
            see[j] = see[int(torch.randint(0, j, (1,), generator=g))]
        if kind == "holes":  # some nodes see nothing at all, some not themselves
            see[j] = torch.rand(n, generator=g) < 0.3
            if j % 3 == 0:
                see[j] = False
            continue
        see[j, j] = True
    return see


def words_of(sees, words):
    rows = []
    for see in sees:
        n = see.shape[0]
        b = torch.zeros(n, 64 * words, dtype=torch.bool)
        m = min(n, 64 * words)
        b[:, :m] = see[:, :m]
        rows.append((b.view(n, words, 64).long() << torch.arange(64)).sum(-1))
    return torch.cat(rows) if rows else torch.zeros(0, words, dtype=torch.int64)


class Case:
    def __init__(self, hd, nq, nkv, bs, ctx, nodes, kind="tree", seed=0, std=1.5, spare=3,
                 extra_entries=0, max_blocks=None, fill=None):
        g = torch.Generator().manual_seed(seed)
        self.hd, self.nq, self.nkv, self.bs, self.kind = hd, nq, nkv, bs, kind
        self.ctx, self.nodes, self.S = ctx, nodes, len(ctx)
        self.blocks = [(c + t + bs - 1) // bs + extra_entries for c, t in zip(ctx, nodes)]
        self.total_blocks, self.total_q = sum(self.blocks), sum(nodes)
        self.max_q = max(nodes) if nodes else 0
        self.max_blocks = max_blocks or max(1, self.total_blocks + spare)
        table = torch.randperm(self.total_blocks + spare, generator=g)[:self.total_blocks]
        if max_blocks:
            table = table + (max_blocks - self.total_blocks - spare)
        self.table = table.int()
        self.q = (torch.randn(self.total_q, nq, hd, generator=g) * std).bfloat16()
        # the sequences' own tokens; everything else in the pool holds `fill`
        self.k = [torch.randn(c + t, nkv, hd, generator=g).bfloat16() for c, t in zip(ctx, nodes)]
        self.v = [torch.randn(c + t, nkv, hd, generator=g).bfloat16() for c, t in zip(ctx, nodes)]
        self.fill = fill
        if kind == "chain":
            self.sees = [torch.ones(t, t).tril().bool() for t in nodes]
            self.words, self.mask = 0, None
        else:
            self.sees = [tree_bits(t, kind, g) for t in nodes]
            self.words = (self.max_q + 63) // 64
            self.mask = words_of(self.sees, self.words)
        self.w_in = torch.rand(self.total_blocks, generator=g) * 3
        self.scale, self.decay = 1.0 / math.sqrt(hd), 0.75

    def caches(self):
        shape = (self.max_blocks, self.bs, self.nkv, self.hd)
        out = []
        for rows in (self.k, self.v):
            if self.fill is None and self.max_blocks < 100000:
                c = torch.randn(shape, device=DEV).bfloat16()
            else:
                c = torch.empty(shape, device=DEV, dtype=torch.bfloat16)
                if self.fill is not None:
                    c.fill_(self.fill)
            at = 0
            for x, n in zip(rows, self.blocks):
                ids = self.table[at:at + n].long().to(DEV)
                at += n
                p = torch.arange(x.shape[0], device=DEV)
                c[ids[p // self.bs], p % self.bs] = x.to(DEV)
            out.append(c)
        return out

    def gpu(self, weights=True, lse=True, w_in=True, stream=None, table=None, status=None,
            max_q=None):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        d = hss.hss_dims(1, self.nq, self.nkv, self.hd, 16, self.bs, self.max_blocks)
        cum = lambda x: i32([0] + torch.tensor(x, dtype=torch.int64).cumsum(0).tolist())
        self.max_q = max_q or self.max_q
        size = hss.hss_attend_tree_workspace_bytes(d, self.S, self.max_q, self.total_blocks,
                                                   weights)
        ws = torch.zeros(max(size, 1), dtype=torch.uint8, device=DEV)
        if not hasattr(self, "cache"):
            self.cache = self.caches()
        st = status if status is not None else torch.zeros(1, dtype=torch.int32, device=DEV)
        call = hss.AttendTree(d, cum(self.nodes), self.total_q, self.max_q,
                              None if self.mask is None else self.mask.to(DEV), self.words,
                              (self.table if table is None else table).to(DEV),
                              cum(self.blocks), i32(self.ctx), self.S, self.total_blocks,
                              self.scale, self.decay, ws, size, st)
        q = self.q.to(DEV)
        out = torch.full((self.total_q, self.nq, self.hd), 55.0, device=DEV).bfloat16()
        ls = torch.full((self.total_q, self.nq), 55.0, device=DEV) if lse else None
        wo = torch.full((self.total_blocks,), 55.0, device=DEV) if weights else None
        wi = self.w_in.to(DEV) if w_in else None
        torch.cuda.synchronize()
        for _ in range(2):  # the second call finds the workspace as the first left it
            call(q, self.cache[0], self.cache[1], out, ls, wi, wo, stream)
        torch.cuda.synchronize()
        if status is None:
            assert st.item() == 0 and hss.hss_read_device_error() == 0
        return out, ls, wo

    def check(self, got, hide=None, w_in=True):
        out, lse, wo = got
        at_q = at_b = 0
        g = self.nq // self.nkv
        for s in range(self.S):
            t, c, nb = self.nodes[s], self.ctx[s], self.blocks[s]
            q = self.q[at_q:at_q + t].to(DEV).double()                     # [t, nq, hd]
            k = self.k[s].to(DEV).double().repeat_interleave(g, 1)         # [n, nq, hd]
            v = self.v[s].to(DEV).double().repeat_interleave(g, 1)
            see = torch.ones(t, c + t, dtype=torch.bool, device=DEV)
            see[:, c:] = self.sees[s].to(DEV)
            if hide is not None:
                see &= ~hide[s].to(DEV)[None]
            seen = see.any(0)  # tokens that no row sees may hold anything: left out by hand
            k, v = k[seen], v[seen]
            see = see[:, seen]
            z = torch.einsum("thd,nhd->htn", q, k) * self.scale
            size = torch.einsum("thd,nhd->htn", q.abs(), k.abs()) * abs(self.scale)
            z = z.masked_fill(~see[None], -math.inf)
            e = 2 * self.hd * 2.0 ** -23 * (size * see[None]).amax(-1) + 2.0 ** -20 \
                if z.shape[-1] else torch.zeros(z.shape[:2], device=DEV).double() + 2.0 ** -20
            some = see.any(1)
            want_lse = torch.logsumexp(z, -1) if z.shape[-1] else torch.full(
                z.shape[:2], -math.inf, device=DEV).double()
            p = (z - want_lse[..., None]).exp().masked_fill(~see[None], 0.0)
            p = torch.where(some[None, :, None], p, torch.zeros_like(p))
            want = torch.einsum("htn,nhd->thd", p, torch.where(see.any(0)[:, None, None], v, 0 * v))
            spread = torch.einsum("htn,nhd->thd", p, v.abs())
            o = out[at_q:at_q + t].double()
            eh = e.transpose(0, 1)[..., None]
            room = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * eh) * spread
            finite = want.isfinite()
            assert not ((o - want).abs() > room)[finite].any(), (
                s, ((o - want).abs() - room)[finite].max().item())
            assert o[finite].isfinite().all()
            assert not o[~finite].isfinite().any()
            if lse is not None:
                got_l, want_l = lse[at_q:at_q + t].double(), want_lse.transpose(0, 1)
                empty = ~some
                assert (got_l[empty] == -math.inf).all() and (o[empty] == 0).all()
                off = (got_l - want_l).abs() - (e.transpose(0, 1) + 2.0 ** -20 * want_l.abs())
                assert not (off[some] > 0).any(), off[some].max().item()
            if wo is not None:
                mass = torch.zeros(nb * self.bs, device=DEV).double()
                err = mass.clone()
                where = torch.arange(c + t, device=DEV)[seen]
                mass[where] = p.sum((0, 1))
                err[where] = (p * (2 * e[..., None] + 2.0 ** -16)).sum((0, 1))
                old = self.w_in[at_b:at_b + nb].to(DEV).double() * (self.decay if w_in else 0.0)
                want_w = mass.view(nb, self.bs).sum(1) + old
                room = err.view(nb, self.bs).sum(1) + 2.0 ** -21 * want_w.abs()
                off = (wo[at_b:at_b + nb].double() - want_w).abs() - room
                assert not (off > 0).any(), off.max().item()
            at_q += t
            at_b += nb
        return True


LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500]


@pytest.mark.parametrize("hd,nq,nkv,bs", [(128, 8, 2, 16), (64, 3, 1, 32), (192, 4, 4, 48),
                                          (256, 5, 1, 16), (128, 16, 1, 144), (64, 2, 2, 256)])
def test_single_tokens(hd, nq, nkv, bs):
    c = Case(hd, nq, nkv, bs, LENGTHS, [1] * len(LENGTHS), "chain", seed=hd + nq)
    c.check(c.gpu())


@pytest.mark.parametrize("hd,nq,nkv,bs", [(128, 32, 8, 16), (64, 9, 3, 32), (192, 6, 2, 16),
                                          (256, 4, 2, 64), (128, 7, 1, 48)])
@pytest.mark.parametrize("kind", ["tree", "chain", "holes"])
def test_trees(hd, nq, nkv, bs, kind):
    ctx = [0, 5, 130, 256, 0, 700, 33, 120]
    nodes = [7, 1, 13, 64, 65, 3, 0, 130]
    c = Case(hd, nq, nkv, bs, ctx, nodes, kind, seed=nq + len(kind))
    c.check(c.gpu())


@pytest.mark.parametrize("nq,nkv", [(128, 1), (100, 1), (16, 16), (48, 3), (10, 2)])
def test_head_groups(nq, nkv):
    c = Case(128, nq, nkv, 16, [200, 1, 77], [5, 2, 1], "tree", seed=nq)
    c.check(c.gpu())


@pytest.mark.parametrize("hd,nq,nkv", [(128, 32, 4), (64, 16, 2), (192, 8, 1), (256, 8, 1)])
def test_many_rows(hd, nq, nkv):
    # several tiles of rows, and a mask of several words
    c = Case(hd, nq, nkv, 16, [300, 40], [150, 201], "tree", seed=hd)
    c.check(c.gpu())
    c = Case(hd, nq, nkv, 32, [1000], [333], "chain", seed=hd + 1)
    c.check(c.gpu())


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
def test_long_context_is_split_and_joined(hd):
    c = Case(hd, 4, 2, 16, [20000], [1], "chain", seed=hd)
    c.check(c.gpu())
    c = Case(hd, 16, 2, 16, [9001, 3, 0, 12000], [21, 1, 9, 2], "tree", seed=hd, std=4.0)
    c.check(c.gpu())


def test_long_context_of_many_row_tiles():
    c = Case(128, 64, 2, 16, [9000, 100], [40, 9], "tree", seed=5)
    c.check(c.gpu())


def test_many_sequences():
    g = torch.Generator().manual_seed(9)
    ctx = torch.randint(0, 90, (700,), generator=g).tolist()
    nodes = torch.randint(0, 3, (700,), generator=g).tolist()
    c = Case(64, 4, 2, 16, ctx, nodes, "tree", seed=10)
    c.check(c.gpu())


def test_scores_far_apart():
    # scores of hundreds: almost all weight on few tokens, and a maximum that keeps moving
    for std in (30.0, 100.0):
        c = Case(128, 8, 2, 16, [3000, 200], [4, 9], "tree", seed=11, std=std)
        c.check(c.gpu())
    c = Case(64, 4, 1, 16, [4000], [3], "chain", seed=12, std=4.0)
    k = c.k[0]
    c.k[0] = (k.float() * torch.linspace(0.1, 5.0, k.shape[0])[:, None, None]).bfloat16()
    c.check(c.gpu())


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("hd", [64, 128, 192, 256])
def test_memory_past_the_tokens_may_hold_anything(fill, hd):
    c = Case(hd, 8, 2, 32, [0, 1, 100, 127, 300], [1, 3, 2, 1, 7], "tree", seed=13, fill=fill,
             extra_entries=1)
    c.check(c.gpu())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("hd,nodes", [(128, 9), (64, 150), (192, 9), (256, 9)])
def test_nodes_that_no_row_sees_may_hold_anything(bad, hd, nodes):
    c = Case(hd, 8, 2, 16, [123, 0], [nodes, nodes], "tree", seed=14)
    for s in range(2):
        for j in (2, 5, nodes - 1):
            c.sees[s][:, j] = False
            c.k[s][c.ctx[s] + j] = bad
            c.v[s][c.ctx[s] + j] = bad
    c.mask = words_of(c.sees, c.words)
    c.check(c.gpu())


@pytest.mark.parametrize("hd,nodes", [(128, 9), (64, 150), (192, 9), (256, 9)])
def test_a_bad_value_reaches_only_the_rows_that_see_it(hd, nodes):
    c = Case(hd, 8, 2, 16, [123, 64], [nodes, nodes], "tree", seed=15, std=0.5)
    for s in range(2):
        c.v[s][c.ctx[s] + 3, 1, 5] = math.inf
        c.v[s][c.ctx[s] + 4, 0, 60] = math.nan
    out, lse, w = c.gpu()
    g = 4
    at = 0
    for s in range(2):
        o = out[at:at + nodes].cpu()
        for node, head, dim in ((3, 1, 5), (4, 0, 60)):
            rows = c.sees[s][:, node]
            part = o[:, head * g:(head + 1) * g, dim]
            assert not part[rows].isfinite().any() and part[~rows].isfinite().all()
        o = o.clone()
        o[:, g:, 5] = 0
        o[:, :g, 60] = 0
        assert o.isfinite().all()
        at += nodes


def test_bad_ids_hide_their_tokens_and_are_reported():
    c = Case(128, 8, 2, 16, [200, 90], [3, 2], "chain", seed=16)
    table = c.table.clone()
    table[4] = -5
    table[c.blocks[0] + 1] = c.max_blocks
    hide = [torch.zeros(x + t, dtype=torch.bool) for x, t in zip(c.ctx, c.nodes)]
    hide[0][64:80] = True
    hide[1][16:32] = True
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    hss.hss_read_device_error()
    got = c.gpu(table=table, status=st)
    assert st.item() == hss.HSS_ERR_OUT_OF_RANGE
    assert hss.hss_read_device_error() == hss.HSS_ERR_OUT_OF_RANGE
    c.check(got, hide=hide)


def test_table_too_short_is_reported():
    c = Case(128, 4, 2, 16, [100, 30], [2, 1], "chain", seed=17)
    c.ctx[0] += 16  # one block more than the table has
    c.k[0] = torch.cat([c.k[0], torch.zeros(16, 2, 128).bfloat16()])
    c.v[0] = torch.cat([c.v[0], torch.zeros(16, 2, 128).bfloat16()])
    keep = c.blocks[0] * 16
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.k[0], c.v[0] = c.k[0][:keep], c.v[0][:keep]
    got = c.gpu(status=st)
    assert st.item() == hss.HSS_ERR_OUT_OF_RANGE
    hss.hss_read_device_error()
    c.k[0] = torch.cat([c.k[0], torch.zeros(118 - keep, 2, 128).bfloat16()])
    c.v[0] = torch.cat([c.v[0], torch.zeros(118 - keep, 2, 128).bfloat16()])
    hide = [torch.arange(118) >= keep, torch.zeros(31, dtype=torch.bool)]
    c.check(got, hide=hide)


def test_more_rows_than_max_q_is_reported():
    c = Case(64, 4, 2, 16, [20, 9], [5, 2], "chain", seed=18)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.total_q = 7
    got = c.gpu(status=st, max_q=4)
    assert st.item() == hss.HSS_ERR_INVALID_ARGUMENT
    hss.hss_read_device_error()
    assert (got[0][4] == 55.0).all()  # the row past max_q is not written


def test_outputs_left_out():
    c = Case(128, 8, 2, 16, [300, 40], [5, 1], "tree", seed=19)
    full = c.gpu()
    c.check(full)
    out, lse, w = c.gpu(weights=False, lse=False)
    assert lse is None and w is None
    assert torch.equal(out.view(torch.int16), full[0].view(torch.int16))
    got = c.gpu(lse=False, w_in=False)
    c.check(got, w_in=False)
    assert torch.equal(got[0].view(torch.int16), full[0].view(torch.int16))


def test_no_rows_only_decay():
    c = Case(128, 8, 2, 16, [300, 40], [0, 0], "chain", seed=20)
    c.check(c.gpu())


def test_scale_zero_and_negative():
    for scale in (0.0, -0.2):
        c = Case(128, 4, 2, 16, [150, 3], [2, 5], "tree", seed=21)
        c.scale = scale
        c.check(c.gpu())


def test_weights_in_place():
    c = Case(128, 8, 2, 16, [300, 40], [5, 1], "tree", seed=22)
    out, lse, w = c.gpu()
    w2 = c.w_in.to(DEV)
    d = hss.hss_dims(1, c.nq, c.nkv, c.hd, 16, c.bs, c.max_blocks)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    size = hss.hss_attend_tree_workspace_bytes(d, 2, c.max_q, c.total_blocks, True)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    call = hss.AttendTree(d, i32([0, 5, 6]), 6, c.max_q, c.mask.to(DEV), c.words,
                          c.table.to(DEV), i32([0, c.blocks[0], c.total_blocks]), i32(c.ctx), 2,
                          c.total_blocks, c.scale, c.decay, ws, size)
    call(c.q.to(DEV), *c.cache, torch.empty_like(out), None, w2, w2)
    torch.cuda.synchronize()
    assert torch.equal(w, w2)


def test_same_bits_every_time_and_on_another_stream():
    c = Case(128, 16, 2, 16, [5000, 40, 900], [9, 1, 30], "tree", seed=23)
    first = c.gpu()
    side = torch.cuda.Stream()
    for stream in (None, side):
        again = c.gpu(stream=stream)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16))
        assert torch.equal(first[1], again[1]) and torch.equal(first[2], again[2])


def test_cache_past_32_bits():
    # 150,000 blocks of 16,384 elements: the blocks used lie past element 2^31
    c = Case(128, 8, 8, 16, [700], [3], "tree", seed=24, max_blocks=150000)
    assert int(c.table.min()) * 16 * 8 * 128 > 2 ** 31
    c.check(c.gpu())


# Many short sequences of many rows: most (sequence, head) items lie whole in one CTA's range.
@pytest.mark.parametrize("hd,nq,nkv,bs", [(64, 16, 4, 16), (128, 21, 3, 48), (192, 8, 2, 16),
                                          (256, 12, 4, 32)])
@pytest.mark.parametrize("kind", ["tree", "chain", "holes"])
def test_many_short_sequences_of_many_rows(hd, nq, nkv, bs, kind):
    ctx = [(37 * i) % 131 for i in range(45)]
    nodes = [1 + (53 * i) % 97 for i in range(45)]
    c = Case(hd, nq, nkv, bs, ctx, nodes, kind, seed=40 + hd)
    c.check(c.gpu())


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
def test_a_bad_value_among_many_short_sequences(hd):
    n = 70
    c = Case(hd, 8, 2, 16, [(29 * i) % 90 for i in range(40)], [n] * 40, "tree", seed=50, std=0.5)
    for s in range(0, 40, 3):
        c.v[s][c.ctx[s] + 3, 1, 5] = math.inf
        c.v[s][c.ctx[s] + 66, 0, 60] = math.nan
    out, lse, w = c.gpu()
    assert w.isfinite().all() and lse.isfinite().all()
    o = out.cpu().view(40, n, 8, hd)
    for s in range(40):
        for node, head, dim in ((3, 1, 5), (66, 0, 60)):
            rows = c.sees[s][:, node] if s % 3 == 0 else torch.zeros(n, dtype=torch.bool)
            part = o[s, :, head * 4:head * 4 + 4, dim]
            assert not part[rows].isfinite().any() and part[~rows].isfinite().all()
    o = o.clone()
    o[:, :, 4:, 5] = 0
    o[:, :, :4, 60] = 0
    assert o.isfinite().all()


@pytest.mark.parametrize("hd,nodes", [(64, [150, 150, 80]), (128, [3, 2, 4]), (192, [90, 1, 2]),
                                      (256, [150, 70, 80])])
def test_rows_of_a_sequence_without_tokens_are_zero(hd, nodes):
    c = Case(hd, 8, 2, 16, [0, 0, 30], nodes, "tree", seed=60)
    a, b = c.blocks[0], c.blocks[0] + c.blocks[1]
    c.table = torch.cat([c.table[:a], c.table[b:]])
    c.w_in = torch.cat([c.w_in[:a], c.w_in[b:]])
    c.blocks[1] = 0
    c.total_blocks = sum(c.blocks)
    keep = c.k[1], c.v[1]
    c.k[1], c.v[1] = keep[0][:0], keep[1][:0]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = c.gpu(status=st)
    assert st.item() == hss.HSS_ERR_OUT_OF_RANGE
    hss.hss_read_device_error()
    c.k[1], c.v[1] = keep
    hide = [torch.zeros(x + t, dtype=torch.bool) for x, t in zip(c.ctx, c.nodes)]
    hide[1][:] = True
    # (nothing of the hidden sequence's weights can be asked for: it has no entries)
    lse, at = got[1], c.nodes[0]
    assert (got[0][at:at + c.nodes[1]] == 0).all()
    assert (lse[at:at + c.nodes[1]] == -math.inf).all()
    c.check((got[0], lse, None), hide=hide)


@pytest.mark.parametrize("hd,ctx", [(64, 0), (128, 37), (192, 0), (256, 70)])
def test_a_bad_value_in_a_long_chain_reaches_the_rows_from_its_node_on(hd, ctx):
    n = 300
    c = Case(hd, 8, 2, 16, [ctx, ctx + 5], [n, n], "chain", seed=70, std=0.5)
    spots = ((3, 1, 5, math.inf), (130, 0, 60, math.nan), (131, 1, 7, -math.inf),
             (n - 1, 0, 1, math.inf))
    for node, head, dim, bad in spots:
        c.v[0][ctx + node, head, dim] = bad
    out, lse, w = c.gpu()
    assert w.isfinite().all() and lse.isfinite().all()
    o = out.cpu().view(2, n, 8, hd).clone()
    assert o[1].isfinite().all()
    for node, head, dim, bad in spots:
        part = o[0, :, head * 4:head * 4 + 4, dim]
        assert part[:node].isfinite().all() and not part[node:].isfinite().any()
        part[node:] = 0
    assert o.isfinite().all()
