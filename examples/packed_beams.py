#!/usr/bin/env python3
"""Beams over a paged cache in 4 bits, with a sliding window: one layer, a few steps.

The prompts are written and attended in chunks.  Then, each step:
  1. the beams are put in a new order: some go on, some fork and some are dropped; their tables,
     the page counts and the copies of pages that part come from one plan (hss_fork_pages,
     hss_copy_pages), which also gives every beam room for its new tokens;
  2. the queries and keys of the new tokens (random here; a model's projections otherwise) are
     normed and rotated (hss_norm_rope_tokens), and keys and values packed into the cache
     (hss_pack_kv_tokens);
  3. they attend over the window and the first tokens (hss_attend_packed);
  4. the last of the drafted tokens is rejected: the next plan cuts it off;
  5. every few steps the used pages move to the front of the pool (hss_compact_pages).

    python examples/packed_beams.py [--steps 12] [--beams 6]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def run(steps=12, beams=6, prompts=2, drafted=3, block_size=16, heads=(8, 2), head_dim=64,
        pool=160, prompt=150, chunk=64, window=96, sinks=4, seed=0, check=None, log=print):
    """Runs the loop; `check(step, inputs, outputs)` is called after every attention."""
    import torch

    import kv_cache_block_lowrank_gb300 as hss

    dev = "cuda"
    nq, nkv = heads
    gen = torch.Generator().manual_seed(seed)
    dims = hss.hss_dims(1, nq, nkv, head_dim, 16, block_size, pool)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device=dev)
    empty = lambda n: torch.empty(n, dtype=torch.int32, device=dev)
    offsets = lambda n: i32([0] + torch.tensor(n).cumsum(0).tolist())
    page = hss.hss_packed_page_bytes(dims)
    cache = torch.zeros(pool, page, dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    turns = torch.zeros(head_dim // 2, dtype=torch.int64)
    hss.hss_rope_table(hss.hss_rope(head_dim, hss.HSS_ROPE_SCALE_NONE, 10000.0), turns)
    turns = turns.to(dev)
    weights = [torch.randn(head_dim, generator=gen).bfloat16().to(dev) for _ in range(2)]

    table, table_offs = empty(0), offsets([])    # of the present sequences
    refs = torch.zeros(pool, dtype=torch.int32, device=dev)
    lengths = []                                 # tokens of each that stand
    history = []                                 # of each: keys and values as they were packed

    def plan(parents, keep, room):
        """The tables of the next step; copies pages that part."""
        nonlocal table, table_offs, refs
        new = len(parents)
        most = sum(-(-(n + r) // block_size) for n, r in zip(keep, room))
        out, offs, counts = empty(most), empty(new + 1), empty(4)
        new_refs, moves = torch.empty_like(refs), torch.empty(2, new, dtype=torch.int32, device=dev)
        size = hss.hss_fork_pages_workspace_bytes(new, pool)
        work = torch.empty(size, dtype=torch.uint8, device=dev)
        hss.hss_fork_pages(table, table_offs, len(table_offs) - 1, len(table), refs, pool, None, 0,
                           i32(parents), i32(keep), i32(room), new, block_size, most, out, offs,
                           new_refs, moves[0], moves[1], counts, work, size, status)
        hss.hss_copy_pages(moves[0], moves[1], counts[1:], new, cache, None, page, pool, 1, status)
        table, table_offs, refs = out, offs, new_refs
        return counts

    def step_tokens(step, rows, ctx):
        """Writes `rows` tokens of each sequence behind its ctx tokens and attends them."""
        n, width = rows * len(ctx), (nq + 2 * nkv) * head_dim
        qkv = (torch.randn(n, width, generator=gen) * 2).bfloat16().to(dev)
        offs, flat = table_offs.tolist(), table.tolist()
        positions = [c + j for c in ctx for j in range(rows)]
        slots = [flat[offs[s] + p // block_size] * block_size + p % block_size
                 for s, c in enumerate(ctx) for p in range(c, c + rows)]
        q = torch.empty(n, nq, head_dim, dtype=torch.bfloat16, device=dev)
        k = torch.empty(n, nkv, head_dim, dtype=torch.bfloat16, device=dev)
        at = qkv.data_ptr()
        norm = hss.NormRopeTokens(dims, head_dim, hss.HSS_ROPE_HALF, turns, 1.0, i64(positions),
                                  None, n, width, width, width, 0, 0, 1e-6, 1.0, status)
        norm(at, at + 2 * nq * head_dim, None, weights[0], weights[1], q, k, None, None)
        pack = hss.PackTokens(dims, i64(slots), n, nkv * head_dim, width, status)
        pack.pack(k, at + 2 * (nq + nkv) * head_dim, cache)
        size = hss.hss_attend_packed_workspace_bytes(dims, len(ctx), rows, len(table), window,
                                                     sinks)
        work = torch.empty(size, dtype=torch.uint8, device=dev)
        attend = hss.AttendPacked(dims, offsets([rows] * len(ctx)), n, rows, table, table_offs,
                                  i32(ctx), len(ctx), len(table), window, sinks, head_dim ** -0.5,
                                  work, size, status)
        out = torch.empty_like(q)
        lse = torch.empty(n, nq, device=dev)
        attend(q, cache, out, lse)
        v = qkv[:, (nq + nkv) * head_dim:].view(n, nkv, head_dim)
        for s, c in enumerate(ctx):
            new = slice(s * rows, (s + 1) * rows)
            history[s] = tuple(torch.cat([old[:c], x[new]])
                               for old, x in zip(history[s], (k, v)))
        if status.item() != 0:
            raise RuntimeError(f"device status {status.item()}")
        if check is not None:
            check(step, dict(q=q, history=history, ctx=ctx, rows=rows, window=window, sinks=sinks,
                             scale=head_dim ** -0.5), dict(out=out, lse=lse))

    # the prompts, chunk by chunk
    none = torch.empty(0, nkv, head_dim, dtype=torch.bfloat16, device=dev)
    history = [(none, none)] * prompts
    done = 0
    while done < prompt:
        rows = min(chunk, prompt - done)
        plan([-1] * prompts if done == 0 else list(range(prompts)), [done] * prompts,
             [rows] * prompts)
        step_tokens(-1, rows, [done] * prompts)
        done += rows
    lengths = [prompt] * prompts

    for step in range(steps):
        # 1. beams in a new order
        present = len(lengths)
        parents = [b % prompts for b in range(beams)] if step == 0 else \
            torch.randint(0, present, (beams,), generator=gen).tolist()
        keep = [lengths[p] for p in parents]
        counts = plan(parents, keep, [drafted] * beams)
        history = [history[p] for p in parents]
        # 2. and 3.
        step_tokens(step, drafted, keep)
        # 4. one of the drafted tokens is rejected
        lengths = [n + drafted - 1 for n in keep]
        # 5. the pages move up
        entries, copies, used, missing = counts.tolist()
        line = f"step {step}: {copies} pages copied, {used} in use"
        if step % 3 == 2:
            new_table, new_refs, counts = torch.empty_like(table), torch.empty_like(refs), empty(4)
            moves = torch.empty(2, pool, dtype=torch.int32, device=dev)
            size = hss.hss_compact_pages_workspace_bytes(pool)
            work = torch.empty(size, dtype=torch.uint8, device=dev)
            hss.hss_compact_pages(table, len(table), refs, pool, pool, new_table, new_refs,
                                  moves[0], moves[1], counts, work, size, status)
            hss.hss_copy_pages(moves[0], moves[1], counts, pool, cache, None, page, pool, 1,
                               status)
            table, refs = new_table, new_refs
            line += f", {counts.tolist()[0]} moved to the front"
        log(line)
    flat = table.tolist()
    assert refs.tolist() == [flat.count(p) for p in range(pool)], "a page was lost or doubled"
    return lengths, table, refs


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=12)
    p.add_argument("--beams", type=int, default=6)
    a = p.parse_args()
    run(a.steps, a.beams)
