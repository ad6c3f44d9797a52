"""The packed cache's attention of queries, factors and values near the ends of fp32's range, against
64 bits (packed_check.py has the tolerances)."""
import numpy as np
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss
import packed_util as P
from packed_check import check
from test_gpu_attend_packed import DEV, Case, built  # noqa: F401  (the library, built once)

pytestmark = pytest.mark.gpu


def scales_of(c, value):
    """The scales of K or V of all tiles, a view of the cache."""
    words = c.cache.view(torch.bfloat16).view(-1, 9 * c.hd)
    n = 16 * (c.hd // 32)
    return words[:, 8 * c.hd + (n if value else 0):][:, :n]


@pytest.mark.parametrize("hd,up,down,scale", [
    (64, 112, -112, None), (64, 117, -117, None), (128, 118, -118, None), (64, 114, -117, 1.0),
    (128, 120, -120, 0.01), (128, 126, -118, None), (64, 100, -117, 2.0 ** 17),
    (128, 113, -60, 2.0 ** -55), (64, 60, -117, 2.0 ** 57), (192, 118, -118, None),
    (256, 120, -120, -0.05)])
@pytest.mark.parametrize("ctx", [[300, 7], [5000, 40]])
def test_queries_of_any_size(hd, up, down, scale, ctx):
    """Queries of 2^up over keys of 2^down; rows of other sizes beside them."""
    c = Case(hd, 4, 2, 16, ctx, [2, 1], scale=scale)
    scales_of(c, False).mul_(2.0 ** down)
    size = torch.tensor([up, up, up - 3, -126], device=DEV).double().exp2()
    c.q = (c.q.double().clamp(-1.9, 1.9) * size[None, :, None]).bfloat16()
    assert torch.isfinite(c.q).all()
    out, lse = c.call()
    torch.cuda.synchronize()
    assert hss.hss_read_device_error() == 0
    check(c, out, lse)


def test_one_large_query_among_ordinary_ones():
    """Its scores are finite and the largest takes all.  (Its neighbours' bits may differ from those
    without it: the maximum that weights go by moves for all rows of a warp at once.)"""
    c = Case(128, 4, 1, 16, [700], [2])
    c.q[0, 2] = (c.q[0, 2].double() * 2.0 ** 118).bfloat16()
    out, lse = c.call()
    torch.cuda.synchronize()
    check(c, out, lse)


@pytest.mark.parametrize("hd,nq", [(64, 2), (128, 8), (64, 12), (192, 1), (256, 4)])
@pytest.mark.parametrize("ctx", [900, 3000])
def test_values_near_the_end(hd, nq, ctx):
    """Weights that are 2^7.5 times those of the first tokens, over values of up to 2^125."""
    c = Case(hd, nq, 1, 16, [ctx], [1])
    scales_of(c, True).mul_(2.0 ** 122)
    c.q[:] = c.q[0, 0].clone()
    table = c.table.numpy()
    t = np.arange(200, ctx, 7)
    slots = table[t // 16] * 16 + t % 16
    k, _ = P.read_tokens(c.cache, 1, 16, hd, slots)
    score = k[:, 0] @ c.q[0, 0].double().cpu().numpy() * c.scale / np.log(2)
    few = np.flatnonzero(score > 1.0)[:8]
    assert len(few) >= 3
    keys = scales_of(c, False)
    old = keys.clone().view(c.max_blocks * 16, hd // 32)
    keys.zero_()                                # every score is 0 but for a few that are 7.5
    for x, at in zip(score[few], slots[few]):
        keys[at // 16, at % 16 * (hd // 32):][:hd // 32] = (old[at].double() * 7.5 / x).bfloat16()
    out, lse = c.call()
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    check(c, out, lse)


@pytest.mark.parametrize("hd,nq,rows", [(64, 4, 20), (128, 8, 9), (192, 2, 40), (256, 1, 50)])
def test_many_rows_whose_factor_is_past_fp32(hd, nq, rows):
    """Scores of 0 in spite of a query of 2^126 and a factor of 2^12: the keys are 0."""
    c = Case(hd, nq, 1, 16, [200], [rows], scale=2.0 ** 12)
    scales_of(c, False).zero_()
    c.q[:, :, 5] = 2.0 ** 126
    out, lse = c.call()
    torch.cuda.synchronize()
    assert hss.hss_read_device_error() == 0
    assert torch.isfinite(out).all()
    check(c, out, lse)


@pytest.mark.parametrize("hd,rows", [(64, 1), (128, 20), (256, 3)])
def test_scores_past_fp32_are_not_taken_for_nothing(hd, rows):
    """A row with a score past 3.4e38 is not a number; it does not read as a row that sees nothing."""
    c = Case(hd, 2, 1, 16, [100], [rows], scale=2.0 ** 12)
    c.q[0, 1] = (c.q[0, 1].double() * 2.0 ** 124).bfloat16()
    out, lse = c.call()
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
