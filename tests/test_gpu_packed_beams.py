"""The example loop over the packed cache: normed writes, packing, windowed attention, forks with
page copies, rejected tokens and compaction together, every attention against a plain calculation
over what each beam has packed.  (Tolerances as in the attention's own tests: 2^-8 sum p |v| for the
weights' rounding and 2^-8 |out| for the result's, 4e-5 and (head_dim + 8) 2^-23 of a score's terms
in lse, twice that of sum p |v| in the result.)"""
import os
import sys

import numpy as np
import pytest

from packed_util import quantise

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,head_dim,block_size,window,beams", [
    ((8, 2), 64, 16, 96, 6), ((6, 2), 128, 32, 0, 5), ((4, 1), 192, 16, 40, 3),
    ((16, 1), 256, 48, 300, 4)])
def test_packed_beams_loop(heads, head_dim, block_size, window, beams):
    from kv_cache_block_lowrank_gb300 import _build

    _build.build()
    import packed_beams

    seen = []

    def values(rows):
        codes, scales = quantise(rows.double().cpu().numpy())
        return codes * np.repeat(scales, 32, -1)

    def check(step, x, y):
        g = heads[0] // heads[1]
        for s, (c, (k, v)) in enumerate(zip(x["ctx"], x["history"])):
            k, v = values(k), values(v)
            at = slice(s * x["rows"], (s + 1) * x["rows"])
            q = x["q"][at].double().cpu().numpy()
            out, lse = (y[n][at].double().cpu().numpy() for n in ("out", "lse"))
            pos, own = np.arange(len(k)), c + np.arange(x["rows"])[:, None]
            see = pos <= own
            if x["window"]:
                see &= (pos < x["sinks"]) | (pos > own - x["window"])
            for h in range(heads[0]):
                z = np.where(see, q[:, h] @ k[:, h // g].T * x["scale"], -np.inf)
                ln = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1)) + z.max(1)
                p = np.exp(z - ln[:, None])
                want, size = p @ v[:, h // g], p @ np.abs(v[:, h // g])
                most = (np.abs(q[:, h]) @ np.abs(k[:, h // g]).T).max(1) * x["scale"]
                slack = 4e-5 + (head_dim + 8) * 2.0 ** -23 * most
                assert (np.abs(lse[:, h] - ln) <= slack + 2.0 ** -23 * np.abs(ln)).all()
                room = 2.0 ** -8 * (size + np.abs(want)) + 2 * slack[:, None] * size
                assert (np.abs(out[:, h] - want) <= room).all()
        seen.append(step)

    lines = []
    lengths, table, refs = packed_beams.run(steps=7, beams=beams, heads=heads, head_dim=head_dim,
                                            block_size=block_size, window=window, check=check,
                                            log=lines.append)
    assert seen == [-1, -1, -1] + list(range(7)) and len(lines) == 7
    assert lengths == [150 + 2 * 7] * beams
    assert (refs.cpu()[table.cpu().long()] > 0).all()
