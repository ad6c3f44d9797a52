"""The comparison with 64 bits for packed attention whose softmax leaves some tokens next to nothing.

Tolerances are those of test_gpu_attend_packed.py, and for weights that fp32 does not hold: the largest
weight of a row is 2^-8 or more, and what is below 2^-126, 2^-118 of it, counts as 0; of every token
that takes away 2^-118 |v| at most from what the largest weights leave.
"""
import numpy as np

import packed_util as P


def check(c, out, lse, cache=None):
    table, offs, q_offs = c.table.numpy(), c.offs.tolist(), c.q_offs.tolist()
    cache = c.cache if cache is None else cache
    for s, (ctx, r) in enumerate(zip(c.ctx, c.rows)):
        a, b = q_offs[s], q_offs[s + 1]
        entries = table[offs[s]:offs[s + 1]]
        want, ln, size, most = P.attend(
            c.q[a:b].double().cpu().numpy(), cache, c.nkv, c.bs, c.hd, entries, max(ctx, 0), r,
            c.window, c.sinks, c.scale, c.max_blocks)
        pos = np.arange(max(ctx, 0) + r)
        v = P.read_tokens(cache, c.nkv, c.bs, c.hd, entries[pos // c.bs] * c.bs + pos % c.bs)[1]
        lost = 2.0 ** -118 * np.abs(v).sum(0)[np.arange(c.nq) // (c.nq // c.nkv)]
        slack = 4e-5 + (c.hd + 8) * 2.0 ** -23 * most
        got = out[a:b].double().cpu().numpy()
        room = 2.0 ** -8 * (size + np.abs(want)) + 2 * slack[..., None] * size + lost
        assert (np.abs(got - want) <= room).all(), (s, np.abs(got - want).max())
        got = lse[a:b].double().cpu().numpy()
        assert (np.abs(got - ln) <= slack + 2.0 ** -23 * np.abs(ln)).all(), s
