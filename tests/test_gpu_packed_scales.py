"""Many rows over a group whose scale fp16 has no place for: the rows that see it, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss
import packed_util as P
from packed_check import check
from test_gpu_attend_packed import DEV, Case, built  # noqa: F401  (the library, built once)

pytestmark = pytest.mark.gpu


def with_scale(c, t, group, value, scale):
    """The cache with another scale for one group of token t of the first sequence."""
    cache = c.cache.clone()
    tile = cache[c.table[t // 16].item()].view(-1)
    at = 2 * P.scale_place(t % 16, group, c.hd, value)
    tile[at:at + 2] = torch.tensor([scale], dtype=torch.bfloat16, device=DEV).view(torch.uint8)
    return cache


@pytest.mark.parametrize("hd,value,scale", [
    (192, True, 2.0 ** 30), (64, True, 2.0 ** 100), (128, True, 65.0), (256, True, 2.0 ** -18),
    (128, True, 2.0 ** -126), (64, False, 100.0), (192, False, 2.0 ** -100)])
@pytest.mark.parametrize("ctx", [[40, 90], [3000, 90]])
def test_rows_that_see_the_scale(hd, value, scale, ctx):
    c = Case(hd, 4, 1, 16, ctx, [30, 40])
    cache = with_scale(c, ctx[0] + 11, 1, value, scale)
    out, lse = c.call(cache=cache)
    torch.cuda.synchronize()
    assert hss.hss_read_device_error() == 0
    check(c, out, lse, cache)


def test_a_key_whose_scores_pass_fp32():
    """Where the token's score is far below the others it has no weight, where it is finite and far
    above them it has all, and a score past 3.4e38 is no number; other rows are as without it."""
    hd, big = 128, 3.0e38
    c = Case(hd, 4, 1, 16, [40, 90], [30, 40])
    t = 51                                             # the first sequence's row 11
    cache = with_scale(c, t, 1, False, big)
    out, lse = (x.double().cpu().numpy() for x in c.call(cache=cache))
    torch.cuda.synchronize()
    assert hss.hss_read_device_error() == 0
    slot = [int(c.table[t // 16]) * 16 + t % 16]
    k, v = P.read_tokens(cache, 1, 16, hd, slot)
    table, q = c.table.numpy(), c.q.double().cpu().numpy()
    kinds = set()
    for first, rows, ctx, tab in ((0, 30, 40, table[:5]), (30, 40, 90, table[5:])):
        args = (1, 16, hd, tab, ctx, rows, 0, 0, c.scale, c.max_blocks)
        want, ln, size, _ = P.attend(q[first:first + rows], cache, *args)
        most = P.attend(q[first:first + rows], c.cache, *args)[3]   # (of scores of ordinary size)
        slack = 4e-5 + (hd + 8) * 2.0 ** -23 * most
        room = 2.0 ** -8 * (size + np.abs(want)) + 2 * slack[..., None] * size
        for i in range(rows):
            for h in range(4):
                got, at = out[first + i, h], lse[first + i, h]
                score = 0.0
                if first == 0 and i >= 11:
                    score = q[i, h] @ k[0, 0] * c.scale * math.log2(math.e)
                    assert abs(abs(score) / 3.4e38 - 1) > 0.01   # (the seed's: none on the border)
                if score > 3.4e38:
                    kinds.add("past")
                    assert np.isnan(got).all() and np.isnan(at)
                elif score > 0:
                    kinds.add("all")
                    assert (np.abs(got - v[0, 0]) <= 2.0 ** -7 * np.abs(v[0, 0])).all()
                    assert abs(at - ln[i, h]) <= 1e-4 * abs(ln[i, h])
                else:
                    kinds.add("none")
                    assert (np.abs(got - want[i, h]) <= room[i, h]).all()
                    assert abs(at - ln[i, h]) <= slack[i, h] + 2.0 ** -23 * abs(ln[i, h])
    assert {"past", "none"} <= kinds
