"""hss_attend_tree where a CTA walks many short pieces one after another: what it keeps of a piece
(the flag of a non-finite value) must last until every warp has read it, and no longer."""
import math

import pytest
import torch
from test_gpu_attend import DEV, Case, built  # noqa: F401 (the fixture builds the library)

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
