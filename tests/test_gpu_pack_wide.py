"""Packing and reading back of as many tokens and heads as are taken a whole tile at a time, for every
head size, and of one head fewer: exact, by the checks of the other packing tests."""
import pytest

import test_gpu_pack as P
import test_gpu_pack_ties as T
from test_gpu_pack import built  # noqa: F401  (the library, built once)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd,nkv,bs,tokens,order", [
    (64, 8, 16, 4500, "run"), (64, 9, 48, 4200, "any"), (64, 7, 16, 4100, "run"),
    (128, 4, 48, 5000, "parts"), (128, 4, 16, 4096, "any"), (128, 3, 16, 4200, "run"),
    (192, 3, 16, 4100, "any"), (192, 3, 64, 4500, "run"), (192, 2, 16, 4300, "run"),
    (256, 2, 32, 4200, "run"), (256, 2, 16, 5000, "parts"), (256, 1, 16, 4200, "any")])
def test_round_trip(hd, nkv, bs, tokens, order):
    P.test_round_trip(hd, nkv, bs, tokens, order)


@pytest.mark.parametrize("hd,nkv,bs", [(64, 8, 16), (128, 4, 48), (192, 3, 16), (256, 2, 32)])
def test_ties_go_to_the_even_code(hd, nkv, bs):
    T.test_ties_go_to_the_even_code(4300, "run", hd, nkv, bs)
