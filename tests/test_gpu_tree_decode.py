"""The example loop: rotary writes, tree attention and eviction together, every step's attention
against a plain calculation.  (Tolerances: a weight is off by a few 2^-20 of itself in lse, the
outputs by the rounding of the weights and of the result to bf16, 2^-7 of sum p |v| in all.)"""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("budget,nodes,heads,head_dim,block_size", [
    (8, 6, (8, 2), 64, 16), (5, 9, (6, 2), 128, 32), (1000, 3, (4, 4), 64, 16)])
def test_tree_decode_loop(budget, nodes, heads, head_dim, block_size):
    from kv_cache_block_lowrank_gb300 import _build

    _build.build()
    import tree_decode

    def check(step, x, y):
        g = x["q"].shape[1] // x["k"].shape[2]
        at = e0 = 0
        for ctx, see, n in zip(x["ctx"], x["sees"], x["lengths"]):
            t = len(see)
            ids = x["table"][e0:e0 + n].long()
            k = x["k"][ids].flatten(0, 1)[:ctx + t].double().repeat_interleave(g, 1)
            v = x["v"][ids].flatten(0, 1)[:ctx + t].double().repeat_interleave(g, 1)
            q = x["q"][at:at + t].double()
            vis = torch.ones(t, ctx + t, dtype=torch.bool, device=q.device)
            for i, bits in enumerate(see):
                for j in range(t):
                    vis[i, ctx + j] = bool(bits >> j & 1)
            z = torch.einsum("thd,nhd->htn", q, k) * x["scale"]
            z = z.masked_fill(~vis[None], float("-inf"))
            p = z.softmax(-1)
            want = torch.einsum("htn,nhd->thd", p, v)
            room = torch.einsum("htn,nhd->thd", p, v.abs()) * 2.0 ** -7
            assert ((y["out"][at:at + t].double() - want).abs() <= room).all()
            lse = torch.logsumexp(z, -1).T
            assert ((y["lse"][at:at + t].double() - lse).abs() <= 1e-4).all()
            mass = torch.zeros(n * block_size, dtype=torch.float64, device=q.device)
            mass[:ctx + t] = p.sum((0, 1))
            w = x["before"][e0:e0 + n].double() * x["decay"] + mass.view(n, -1).sum(1)
            assert ((y["weights"][e0:e0 + n].double() - w).abs() <= 1e-3 * w + 1e-6).all()
            at += t
            e0 += n

    lines = []
    state = tree_decode.run(steps=10, budget=budget, nodes=nodes, heads=heads,
                            head_dim=head_dim, block_size=block_size, check=check,
                            log=lines.append)
    assert len(lines) == 10
    for s in state:
        assert len(s.blocks) <= max(budget, 3)
        assert s.position > s.ctx if budget < 100 else s.position == s.ctx
