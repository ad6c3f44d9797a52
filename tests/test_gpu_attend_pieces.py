"""hss_attend_tree where a CTA walks many short pieces one after another: what it keeps of a piece
(the flag of a non-finite value) must last until every warp has read it, and no longer."""
import math

import pytest
import torch
from test_gpu_attend import DEV, Case, built  # noqa: F401 (the fixture builds the library)

import kv_cache_block_lowrank_gb300 as hss

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view(torch.int16)


# (kind, heads, kv heads, pattern of (context, nodes, has a bad value), sequences)
PATTERNS = [
    # two row tiles a CTA; one-node chains that end a tile of 64 are not looked over for values
    ("chain", 64, 1, [(30, 3, True), (63, 1, False), (30, 3, False), (63, 1, False)], 2432),
    ("chain", 64, 1, [(90, 4, True), (63, 1, False), (127, 1, False), (60, 4, False)], 2432),
    ("chain", 64, 1, [(30, 3, False), (63, 1, False), (30, 3, True)], 2433),
    # a softmax group for the odd tiles, most of whose warps have no rows, and pieces of one tile
    # in which it has nothing to do
    ("tree", 4, 1, [(150, 3, True), (20, 3, False), (20, 2, False), (150, 3, False)], 2432),
    ("tree", 4, 1, [(150, 3, True), (20, 1, False), (170, 3, False)], 2433),
]


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("kind,nq,nkv,pattern,n", PATTERNS)
def test_a_bad_value_stays_with_its_piece(hd, kind, nq, nkv, pattern, n):
    rows = (pattern * n)[:n]
    ctx, nodes, bad = [list(x) for x in zip(*rows)]
    c = Case(hd, nq, nkv, 16, ctx, nodes, kind, seed=80 + hd, std=0.5)
    expected = torch.zeros(c.total_q, nq, hd, dtype=torch.bool)
    spots, at = [], 0
    for s in range(n):
        if bad[s]:
            spots.append(s)
            c.v[s][ctx[s] + 1, 0, 5] = 0.0
            expected[at:at + nodes[s], :, 5] |= c.sees[s][:, 1][:, None]
        at += nodes[s]
    expected = expected.to(DEV)
    clean = c.gpu()
    assert clean[0].isfinite().all()
    for i, s in enumerate(spots):
        c.v[s][ctx[s] + 1, 0, 5] = (math.inf, math.nan, -math.inf)[i % 3]
    del c.cache
    got = c.gpu()
    assert not got[0][expected].isfinite().any()
    assert torch.equal(bits(got[0])[~expected], bits(clean[0])[~expected])
    assert torch.equal(got[1], clean[1]) and torch.equal(got[2], clean[2])


@pytest.mark.parametrize("hd,nodes", [(64, [2, 90, 1]), (128, [3, 5, 0]), (192, [40, 2, 1]),
                                      (256, [3, 20, 1])])
@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("far", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 65, 2 ** 20])
def test_a_context_far_past_the_table(hd, nodes, kind, far):
    # every token of the table counts as context, a non-finite one too, and no node is seen
    c = Case(hd, 8, 2, 16, [93, 70, 128], nodes, kind, seed=90 + hd, std=0.5, fill=0.0)
    keep = [b * 16 for b in c.blocks]
    c.v[0][40, 1, 5] = math.inf
    c.v[1][69, 0, 60] = math.nan  # (the last whole tile of the table, which is looked over)
    ctx = c.ctx
    c.ctx = [far, far - 1, far]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse, w = c.gpu(status=st)
    assert st.item() == hss.HSS_ERR_OUT_OF_RANGE
    hss.hss_read_device_error()
    # the same as chains whose nodes no row sees, over contexts as long as the table
    pad = lambda x, n: torch.cat([x, torch.zeros(n - x.shape[0], *x.shape[1:]).bfloat16()])
    d = Case(hd, 8, 2, 16, keep, nodes, "tree", seed=1)
    d.q, d.w_in, d.fill = c.q, c.w_in.new_zeros(d.total_blocks), c.fill
    at = 0
    for s, n in enumerate(c.blocks):
        d.w_in[sum(d.blocks[:s]):sum(d.blocks[:s]) + n] = c.w_in[at:at + n]
        at += n
        d.k[s], d.v[s] = pad(c.k[s], keep[s] + nodes[s]), pad(c.v[s], keep[s] + nodes[s])
        d.sees[s] = torch.zeros(nodes[s], nodes[s], dtype=torch.bool)
    d.mask = torch.zeros(d.total_q, d.words, dtype=torch.int64)
    want = d.gpu()
    assert torch.equal(out.isfinite(), want[0].isfinite())
    assert not out[:nodes[0], 4:, 5].isfinite().any()
    assert not out[nodes[0]:nodes[0] + nodes[1], :4, 60].isfinite().any()
    some = out.isfinite()
    assert ((out.float() - want[0].float())[some].abs() <= 2.0 ** -6).all()
    assert torch.allclose(lse, want[1], rtol=1e-5, atol=1e-5)
    at = 0
    for s, n in enumerate(c.blocks):
        b = sum(d.blocks[:s])
        assert torch.allclose(w[at:at + n], want[2][b:b + n], rtol=1e-4, atol=1e-5)
        at += n
