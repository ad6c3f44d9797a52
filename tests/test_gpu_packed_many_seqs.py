"""The packed cache's attention of more sequences than a CTA has threads, few and many rows of each:
every thread looks through several sequences for its CTA's range, and every warp's sum counts."""
import numpy as np
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss
from test_gpu_attend_packed import DEV, Case, built  # noqa: F401  (the library, built once)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd,seqs,rows,most", [
    (64, 1500, 1, 60), (64, 640, 40, 60), (128, 700, 36, 40), (192, 1300, 33, 30),
    (256, 650, 34, 20)])
def test_more_sequences_than_threads(hd, seqs, rows, most):
    """One long sequence between many short ones, so that ranges begin in all of them."""
    g = np.random.default_rng(hd + seqs)
    ctx = g.integers(0, most, seqs)
    n = g.integers(0, min(rows, 2) + 1, seqs)
    # the last sequences, whose threads are in the last warps, have most to do
    ctx[-seqs // 8:] += 400
    ctx[seqs // 2], n[seqs // 2] = 6000, rows
    n[seqs // 3], n[-1] = rows, rows
    c = Case(hd, 2, 2, 16, ctx.tolist(), n.tolist(), max_q=rows)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = c.call(status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 == hss.hss_read_device_error()
    c.check(out, lse)
