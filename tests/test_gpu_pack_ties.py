"""Packing of elements that lie exactly between two codes: they go to the even one."""
import numpy as np
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss
from packed_util import quantise, read_tokens
from test_gpu_pack import DEV, built, same  # noqa: F401  (the library, built once)

pytestmark = pytest.mark.gpu

# scales whose halves are bf16 numbers up to 6.5 times, 7 times them too: an odd part of at most 19
ODD = [1, 3, 5, 7, 9, 11, 13, 15, 17, 19]


def tied_group(odd, exponent, sign):
    """32 elements of scale odd 2^exponent: every half between -7 and 7, every whole, the largest."""
    scale = odd * 2.0 ** exponent
    steps = np.concatenate([np.arange(-6.5, 7), np.arange(-7, 8), [0.5, -0.5, 2.5]])
    return sign * steps * scale


@pytest.mark.parametrize("tokens,order", [(80, "any"), (4800, "run")])
@pytest.mark.parametrize("hd,nkv,bs", [(64, 2, 16), (128, 1, 48), (192, 1, 16), (256, 1, 32)])
def test_ties_go_to_the_even_code(tokens, order, hd, nkv, bs):
    groups = [tied_group(odd, e, s) for odd in ODD for e in (-120, -100, -20, -3, 0, 4, 60, 115)
              for s in (1, -1)]
    groups = np.stack(groups)
    n = tokens * nkv * hd // 32
    g = np.random.default_rng(hd)
    x = groups[np.arange(n) % len(groups)]
    x = np.take_along_axis(x, g.permuted(np.tile(np.arange(32), (n, 1)), axis=1), 1)
    x = x.reshape(tokens, nkv, hd)
    k = torch.from_numpy(x).bfloat16()
    assert (k.double().numpy() == x).all()             # every element is a bf16 number
    codes, scales = quantise(x)
    halves = np.abs(x / np.repeat(scales, 32, -1)) % 1 == 0.5
    assert halves.mean() > 0.4 and (codes[halves] % 2 == 0).all()
    blocks = tokens // bs + 2
    slots = torch.arange(tokens) + (5 if order == "run" else 0)
    if order == "any":
        slots = torch.randperm(blocks * bs, generator=torch.Generator().manual_seed(1))[:tokens]
    d = hss.hss_dims(1, nkv, nkv, hd, 16, bs, blocks)
    cache = torch.zeros(blocks, hss.hss_packed_page_bytes(d), dtype=torch.uint8, device=DEV)
    v = -k.flip(0)
    hss.PackTokens(d, slots.to(DEV), tokens, nkv * hd, nkv * hd).pack(k.to(DEV), v.to(DEV), cache)
    torch.cuda.synchronize()
    assert hss.hss_read_device_error() == 0
    got = read_tokens(cache, nkv, bs, hd, slots.numpy())
    want = codes * np.repeat(scales, 32, -1)
    assert same(got[0], want)
    assert same(got[1], -want[::-1])
