"""Limits of the packed attention's arguments (nothing here reaches a launch)."""
import pytest

import kv_cache_block_lowrank_gb300 as hss
from test_packed_abi import attend, lib, status_of  # noqa: F401  (the library, built once)


@pytest.mark.parametrize("scale", [2.0 ** 101, -2.0 ** 101, 3.0e38, -3.0e38])
def test_factors_past_the_limit(scale):
    assert status_of(attend, scale=scale) == hss.HSS_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("scale", [2.0 ** 100, -2.0 ** 100, 0.0, 1e-45])
def test_factors_up_to_the_limit(scale):
    attend(scale=scale, total_q=0)
