#!/usr/bin/env python3
"""Tree decoding over a paged cache that is cut to a budget: one layer, a few steps.

Each step, for every sequence:
  1. the queries, keys and values of a drafted tree (random here; a model's projections
     otherwise) are rotated and written into the cache behind the context, one launch
     (hss_rope_tokens), and the rotated keys are projected into the low-rank store
     (hss_write_kv_tokens);
  2. the tree attends over the context and itself, and every block's attention weight is
     accumulated (hss_attend_tree);
  3. one path of the tree is accepted: its keys and values move up behind the context (the same
     rotary write, at their final slots), and the context grows;
  4. sequences over their budget lose the whole blocks with the least accumulated weight
     (hss_evict_blocks); the freed ids go back to the pool.

    python examples/tree_decode.py [--steps 12] [--budget 12]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


class Sequence:
    def __init__(self):
        self.blocks: list[int] = []  # physical ids, in order
        self.weights: list[float] = []
        self.ctx = 0                 # tokens in the cache
        self.position = 0            # of the next token (evicted tokens still count)


def draw_tree(gen, nodes):
    """Parents of a random tree (-1: the context's last token)."""
    import torch

    return [-1] + [int(torch.randint(-1, j, (1,), generator=gen)) for j in range(1, nodes)]


def run(steps=12, budget=12, seqs=3, nodes=6, block_size=16, heads=(8, 2), head_dim=64, r=16,
        pool=128, prompt=150, seed=0, check=None, log=print):
    """Runs the loop; `check(step, inputs, outputs)` is called after every attention."""
    import torch

    import kv_cache_block_lowrank_gb300 as hss

    dev = "cuda"
    nq, nkv = heads
    gen = torch.Generator().manual_seed(seed)
    dims = hss.hss_dims(1, nq, nkv, head_dim, r, block_size, pool)
    normal = lambda *s: torch.randn(*s, generator=gen).bfloat16().to(dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=dev)
    offsets = lambda n: i32([0] + torch.tensor(n).cumsum(0).tolist())

    turns = torch.zeros(head_dim // 2, dtype=torch.int64)
    hss.hss_rope_table(hss.hss_rope(head_dim, hss.HSS_ROPE_SCALE_RAMP, 10000.0, 4.0, 8192.0, 1.0,
                                    32.0), turns)
    turns = turns.to(dev)
    P = normal(head_dim, r) / math.sqrt(r)
    k_cache = torch.zeros(pool, block_size, nkv, head_dim, dtype=torch.bfloat16, device=dev)
    v_cache = torch.zeros_like(k_cache)
    A_g = torch.zeros(1, pool, nkv, block_size, r, dtype=torch.bfloat16, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    free = list(range(pool))
    state = [Sequence() for _ in range(seqs)]

    def grow(s, tokens):
        """Blocks for `tokens` tokens behind s's context."""
        while len(s.blocks) * block_size < s.ctx + tokens:
            s.blocks.append(free.pop())
            s.weights.append(0.0)

    def slot(s, at):
        return s.blocks[at // block_size] * block_size + at % block_size

    def write(qkv, positions, slots):
        """Rotary write of rows [n, (nq + 2 nkv) head_dim]; the rotated queries."""
        n, width = qkv.shape
        q = torch.empty(n, nq, head_dim, dtype=torch.bfloat16, device=dev)
        k = torch.empty(n, nkv, head_dim, dtype=torch.bfloat16, device=dev)
        call = hss.RopeTokens(dims, head_dim, hss.HSS_ROPE_HALF, turns, 1.0, i64(positions),
                              i64(slots), n, width, width, width, status)
        at = qkv.data_ptr()
        call(at, at + 2 * nq * head_dim, at + 2 * (nq + nkv) * head_dim, q, k, k_cache, v_cache)
        hss.hss_write_kv_tokens(dims, P, k, i64(slots), n, None, A_g, 0, status)
        return q

    def rows(n):
        return normal(n, (nq + 2 * nkv) * head_dim)

    for s in state:  # the prompts
        grow(s, prompt)
        write(rows(prompt), list(range(prompt)), [slot(s, i) for i in range(prompt)])
        s.ctx = s.position = prompt

    for step in range(steps):
        # 1. the drafts' rows go behind the contexts
        trees = [draw_tree(gen, nodes) for _ in state]
        depth, sees = [], []
        for parents in trees:
            d, see = [], []
            for j, parent in enumerate(parents):
                d.append(0 if parent < 0 else d[parent] + 1)
                see.append((see[parent] if parent >= 0 else 0) | 1 << j)
            depth.append(d)
            sees.append(see)
        qkv = rows(seqs * nodes)
        positions, slots = [], []
        for s, d in zip(state, depth):
            grow(s, nodes)
            positions += [s.position + x for x in d]
            slots += [slot(s, s.ctx + j) for j in range(nodes)]
        q = write(qkv, positions, slots)

        # 2. attention, with the blocks' weights accumulated in place
        lengths = [len(s.blocks) for s in state]
        total = sum(lengths)
        table = i32([b for s in state for b in s.blocks])
        weights = torch.tensor([w for s in state for w in s.weights], device=dev)
        size = hss.hss_attend_tree_workspace_bytes(dims, seqs, nodes, total, True)
        work = torch.zeros(size, dtype=torch.uint8, device=dev)
        mask = i64([m for see in sees for m in see])
        attend = hss.AttendTree(dims, offsets([nodes] * seqs), seqs * nodes, nodes, mask, 1, table,
                                offsets(lengths), i32([s.ctx for s in state]), seqs, total,
                                head_dim ** -0.5, 0.9, work, size, status)
        out = torch.empty_like(q)
        lse = torch.empty(seqs * nodes, nq, device=dev)
        before = weights.clone()
        attend(q, k_cache, v_cache, out, lse, weights, weights)
        if check is not None:
            check(step, dict(q=q, k=k_cache, v=v_cache, table=table, lengths=lengths,
                             ctx=[s.ctx for s in state], sees=sees, before=before, decay=0.9,
                             scale=head_dim ** -0.5), dict(out=out, lse=lse, weights=weights))

        # 3. the deepest node's path is accepted
        moved, at_pos, at_slot = [], [], []
        for n, (s, parents, d) in enumerate(zip(state, trees, depth)):
            node = d.index(max(d))
            path = []
            while node >= 0:
                path.insert(0, node)
                node = parents[node]
            moved += [n * nodes + j for j in path]
            at_pos += list(range(s.position, s.position + len(path)))
            at_slot += [slot(s, s.ctx + i) for i in range(len(path))]
            s.ctx += len(path)
            s.position += len(path)
        write(qkv[i64(moved)].contiguous(), at_pos, at_slot)

        # 4. the caches are cut to the budget: the first block and the last two stay
        new_table, freed = torch.empty_like(table), torch.empty_like(table)
        new_weights = torch.empty_like(weights)
        new_offs, freed_offs = offsets([0] * seqs), offsets([0] * seqs)
        new_ctx = i32([0] * seqs)
        hss.hss_evict_blocks(weights, table, offsets(lengths), i32([s.ctx for s in state]),
                             i32([budget] * seqs), seqs, total, block_size, 1, 2, new_table,
                             new_offs, new_weights, new_ctx, freed, freed_offs)
        o, f = new_offs.tolist(), freed_offs.tolist()
        kept, w, gone, ctx = (x.tolist() for x in (new_table, new_weights, freed, new_ctx))
        for n, s in enumerate(state):
            s.blocks, s.weights = kept[o[n]:o[n + 1]], w[o[n]:o[n + 1]]
            s.ctx = ctx[n]
            free.extend(gone[f[n]:f[n + 1]])
        if status.item() != 0:
            raise RuntimeError(f"device status {status.item()}")
        log(f"step {step}: " + "; ".join(
            f"{len(s.blocks)} blocks, {s.ctx} of {s.position} tokens cached" for s in state) +
            f"; {f[-1]} freed")
    used = [b for s in state for b in s.blocks]
    assert sorted(used + free) == list(range(pool)), "a block id was lost or doubled"
    return state


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=12)
    p.add_argument("--budget", type=int, default=12)
    a = p.parse_args()
    run(a.steps, a.budget)
