"""What the workspace of hss_attend_tree holds before a call does not matter: not NaN and set flags,
not what another call of any other shape has left there."""
import pytest
import torch
from test_gpu_attend import DEV, Case, built  # noqa: F401 (the fixture builds the library)

import kv_cache_block_lowrank_gb300 as hss

pytestmark = pytest.mark.gpu


class Call:
    """A case bound to a workspace of its own or a given one."""

    def __init__(self, c, weights):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        cum = lambda x: i32([0] + torch.tensor(x, dtype=torch.int64).cumsum(0).tolist())
        self.c, self.weights = c, weights
        self.dims = hss.hss_dims(1, c.nq, c.nkv, c.hd, 16, c.bs, c.max_blocks)
        self.size = hss.hss_attend_tree_workspace_bytes(self.dims, c.S, c.max_q, c.total_blocks,
                                                        weights)
        self.cache = c.caches()
        self.q, self.w_in = c.q.to(DEV), c.w_in.to(DEV)
        self.bound = (cum(c.nodes), c.total_q, c.max_q, None if c.mask is None else c.mask.to(DEV),
                      c.words, c.table.to(DEV), cum(c.blocks), i32(c.ctx), c.S, c.total_blocks,
                      c.scale, c.decay)

    def run(self, ws):
        c = self.c
        out = torch.full((c.total_q, c.nq, c.hd), 55.0, device=DEV).bfloat16()
        lse = torch.full((c.total_q, c.nq), 55.0, device=DEV)
        w = torch.full((c.total_blocks,), 55.0, device=DEV) if self.weights else None
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        assert ws.numel() >= self.size
        hss.AttendTree(self.dims, *self.bound, ws, self.size, st)(self.q, *self.cache, out, lse,
                                                                  self.w_in, w)
        torch.cuda.synchronize()
        assert st.item() == 0
        return out, lse, w


# head_dim, heads, kv heads, block, contexts, nodes, kind: single tokens, one row tile, two row
# tiles of a pair, several; short items by the hundred; sequences without rows; a long context cut
# into pieces
CASES = [
    (128, 32, 8, 16, [20000], [1], "chain"),
    (128, 32, 8, 16, [700, 0, 33, 4000], [1, 1, 0, 1], "chain"),
    (128, 8, 2, 16, [9001, 3, 0, 12000], [21, 1, 9, 2], "tree"),
    (128, 64, 8, 16, [3000, 70], [61, 20], "tree"),
    (128, 64, 8, 16, [1200, 5, 900], [300, 1, 40], "chain"),
    (64, 16, 4, 16, [37 * i % 131 for i in range(60)], [1 + 53 * i % 97 for i in range(60)], "holes"),
    (64, 3, 1, 32, [15, 0, 500], [7, 1, 3], "tree"),
    (192, 6, 2, 48, [5000, 64], [90, 3], "tree"),
    (192, 4, 4, 16, [300, 20], [2, 5], "chain"),
    (256, 12, 4, 32, [29 * i % 90 for i in range(40)], [70 - i for i in range(40)], "tree"),
    (256, 8, 1, 16, [8000], [33], "chain"),
    (128, 100, 1, 16, [200, 1, 77], [5, 2, 1], "tree"),
]


def cases(weights):
    return [Call(Case(*x, seed=200 + i), weights) for i, x in enumerate(CASES)]


@pytest.mark.parametrize("weights", [True, False])
def test_a_workspace_full_of_ones(weights):
    for call in cases(weights):
        ws = torch.full((call.size + 512,), 255, dtype=torch.uint8, device=DEV)
        call.c.check(call.run(ws))
        assert (ws[call.size:] == 255).all()  # and nothing is written past its end


def test_a_workspace_shared_by_calls_of_all_shapes():
    both = [c for pair in zip(cases(True), cases(False)) for c in pair]
    ws = torch.full((max(c.size for c in both),), 255, dtype=torch.uint8, device=DEV)
    alone = []
    for call in both:
        alone.append(call.run(torch.zeros(call.size, dtype=torch.uint8, device=DEV)))
        call.c.check(alone[-1])
    order = torch.randperm(2 * len(both), generator=torch.Generator().manual_seed(3)) % len(both)
    for i in order.tolist():
        got = both[i].run(ws)
        for a, b in zip(got, alone[i]):
            assert (a is None and b is None) or torch.equal(a.view(torch.int16),
                                                            b.view(torch.int16))
