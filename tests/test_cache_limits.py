"""The paged-cache operators' arguments at their limits, on the host: sizes that pass 32 bits, and
refusals that must come before anything is enqueued."""
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
