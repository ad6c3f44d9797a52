"""The paged-cache operators' arguments at their limits, on the host: sizes that pass 32 bits, and
refusals that must come before anything is enqueued."""
import math

import numpy as np
import pytest
from test_cache_abi import FAKE, attend, dims, lib, status_of  # noqa: F401 (lib builds)

import kv_cache_block_lowrank_gb300 as hss

INT_MAX = 2 ** 31 - 1
size_of = hss.hss_attend_tree_workspace_bytes


@pytest.mark.parametrize("hd,nq,nkv", [(128, 64, 8), (64, 128, 1), (192, 3, 1), (256, 8, 8),
                                       (256, 128, 1)])
@pytest.mark.parametrize("weights", [False, True])
def test_workspace_never_shrinks_with_max_q(hd, nq, nkv, weights):
    d = dims(head_dim=hd, num_q_heads=nq, num_kv_heads=nkv)
    sizes = sorted({q + k for p in range(32) for q in (2 ** p,) for k in (-1, 0, 1)
                    if q + k <= INT_MAX} | set(range(INT_MAX - 300, INT_MAX + 1)))
    last, refused = 0, False
    for q in sizes:
        size = size_of(d, 1, q, 8224, weights)
        refused = refused or size == 0
        assert size == 0 if refused else size >= last, (q, size, last)
        last = size
    assert refused  # 2^31 - 1 rows of a tree are more than a call can have


@pytest.mark.parametrize("max_q", [INT_MAX, INT_MAX - 1, INT_MAX - 100, 2 ** 30])
def test_a_max_q_that_is_too_large_is_refused(max_q):
    # without reaching CUDA, whatever the workspace is said to hold
    assert status_of(attend, dims(num_q_heads=64), total_q=512, max_q=max_q, total=8224,
                     wsb=1 << 62) == hss.HSS_ERR_INVALID_ARGUMENT


def test_counts_whose_products_pass_64_bits_are_refused():
    d = dims(num_q_heads=64, num_kv_heads=64, block_size=256)
    assert size_of(d, INT_MAX, INT_MAX, INT_MAX, True) == 0
    assert size_of(d, 1, 1, 2 ** 62, True) == 0
    assert status_of(attend, d, S=INT_MAX, total_q=INT_MAX, max_q=INT_MAX, total=INT_MAX,
                     wsb=1 << 62) == hss.HSS_ERR_INVALID_ARGUMENT


HEADS = dict(num_q_heads=64, num_kv_heads=8, head_dim=128, block_size=16)


@pytest.mark.parametrize("seqs,max_q,blocks,heads,plain,weighted", [
    # what hss.h says, in MB
    (64, 1, 64 * 1024 + 64, {"num_q_heads": 32}, None, 13),
    (1, 512, 8192 + 32, {}, 39, 1560),
    (64, 2048, 64 * 257 + 128, {}, 4790, 17440),
    (1, 2048, 257 + 127, {}, 95, 382),
    (63, 1, 63 * 257, {}, 5.5, 11)])
def test_workspace_bytes_as_documented(seqs, max_q, blocks, heads, plain, weighted):
    d = dims(**(HEADS | heads))
    for want, weights in ((plain, False), (weighted, True)):
        if want is not None:
            assert size_of(d, seqs, max_q, blocks, weights) / 1e6 == pytest.approx(want, rel=0.04)


@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("g", [1, 3, 8, 16, 42, 65, 128])
@pytest.mark.parametrize("nkv,seqs", [(1, 1), (8, 1), (8, 64), (2, 300)])
def test_workspace_within_its_bound(hd, g, nkv, seqs):
    d = dims(head_dim=hd, num_q_heads=g * nkv, num_kv_heads=nkv)
    tile = 128 // g
    for max_q in list(range(1, 300)) + [333, 511, 512, 513, 1000, 2047, 2048, 2049, 4096, 10000]:
        one = max_q <= tile
        step = 1 if one else (tile if hd == 256 else 2 * tile)
        nodes = (max_q + step - 1) // step * step
        # a row's O, and its maximum and sum; a flag of a piece and a start of a range besides
        rows = seqs * nodes * g * nkv * (4 * hd + 8)
        bound = rows * (2 if one or hd == 256 else 1) * 4 / 3 + 42e6 + 40 * seqs * nodes * nkv
        size = size_of(d, seqs, max_q, seqs * 600, False)
        assert 0 < size <= bound, (max_q, size, bound)
        # with weights, five bytes more for 16 tokens of a row (the tokens as whole tiles, with
        # what the list holds besides: three tiles of 128 or four of 64 a sequence), and its lse
        tokens = seqs * (600 * 16 + 400)
        more = nodes * g * nkv * (tokens * 5 / 16 + 4 * seqs) * 4 / 3 + 4096
        assert size_of(d, seqs, max_q, seqs * 600, True) <= bound + more, max_q


def test_a_grid_that_is_too_large_is_refused_before_any_launch():
    # 2^29 sequences of one row of 128 heads: the attention's own grid is 152 CTAs, the join's and
    # the weights' together more than 2^31
    d = dims(num_q_heads=128, num_kv_heads=1)
    seqs = 2 ** 29 - 200
    assert size_of(d, seqs, 1, 10, True) == 0 < size_of(d, seqs, 1, 10, False)
    assert status_of(attend, d, S=seqs, total_q=1, max_q=1, total=10, wsb=1 << 62) == \
        hss.HSS_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("rope", [
    (4, hss.HSS_ROPE_SCALE_BASE, 1e4, 1e155, 0, 0, 0),    # base 1e314
    (128, hss.HSS_ROPE_SCALE_BASE, 1e300, 1e9, 0, 0, 0),
    (4, hss.HSS_ROPE_SCALE_BASE, 1e-300, 1e-20, 0, 0, 0),  # base 0
    (64, hss.HSS_ROPE_SCALE_RAMP, 1e4, 4.0, 8192, -1e308, 1e308)])
def test_rope_table_refuses_what_passes_a_double(rope):
    out = np.zeros(128, dtype=np.uint64)
    assert status_of(hss.hss_rope_table, hss.hss_rope(*rope), out.ctypes.data) == \
        hss.HSS_ERR_INVALID_ARGUMENT


def test_rope_table_of_a_base_near_the_end_of_a_double():
    out = np.zeros(2, dtype=np.uint64)
    hss.hss_rope_table(hss.hss_rope(4, hss.HSS_ROPE_SCALE_BASE, 1e4, 1e150, 0, 0, 0),
                       out.ctypes.data)
    # base 1e304, the second frequency 1e-152: less than half of a 2^-64th of a turn
    assert out[0] == pytest.approx(2 ** 64 / (2 * math.pi), rel=1e-15) and out[1] == 0
