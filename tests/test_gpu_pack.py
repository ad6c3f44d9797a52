"""Packing tokens into the 4-bit cache and reading them back: exact, against the definition."""
import numpy as np
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss
from packed_util import quantise, read_tokens, tile_bytes

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_block_lowrank_gb300 import _build

    _build.build()
    hss.load()


def rows(g, *shape):
    x = torch.randn(shape, generator=g, device=DEV)
    return (x * torch.randn(shape[:-1], generator=g, device=DEV).exp()[..., None]).bfloat16()


def same(got, want):
    return np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("hd,nkv,bs,tokens,order", [
    (128, 8, 16, 1, "any"), (128, 2, 32, 77, "run"), (64, 3, 48, 100, "run"),
    (64, 1, 16, 16, "run"), (192, 3, 16, 45, "any"), (192, 2, 128, 300, "run"),
    (256, 1, 64, 33, "any"), (256, 5, 16, 64, "run"), (128, 1, 256, 513, "run"), (64, 9, 16, 700, "run"),
    (192, 2, 48, 500, "run"), (256, 3, 16, 400, "run"), (128, 8, 32, 300, "any"),
    (128, 3, 16, 600, "parts"), (64, 2, 64, 1000, "parts"),
    # enough for whole tiles to be taken together
    (64, 2, 16, 4500, "run"), (128, 2, 48, 5000, "parts"), (192, 1, 16, 4100, "any"),
    (256, 1, 32, 4200, "run"), (128, 5, 16, 4096, "run"), (192, 3, 128, 5200, "parts")])
def test_round_trip(hd, nkv, bs, tokens, order):
    g = torch.Generator(device=DEV).manual_seed(hd * tokens + bs)
    blocks = tokens // bs + 3
    k, v = rows(g, tokens, nkv, hd), rows(g, tokens, nkv, hd)
    k[0, 0, :32] = 0.0                      # a group of zeros
    v[-1, -1, 32:64] = 1e-40                # one whose scale is no normal number
    k[tokens // 2, 0, 5] = float("inf")     # groups that cannot be coded
    v[tokens // 2, 0, 37] = float("nan")
    k[-1, -1, :64] = torch.arange(64, device=DEV) - 31.5   # ties
    if order == "run":  # tokens in a row, from inside a page on
        at = torch.arange(tokens, device=DEV) + bs // 2
        slots = torch.randperm(blocks, generator=g, device=DEV)[at // bs] * bs + at % bs
    elif order == "parts":  # runs of many lengths, as prompts' ends lie side by side
        cuts = torch.randint(0, 40, (blocks,), generator=g, device=DEV)
        free = torch.arange(blocks * bs, device=DEV)
        slots = free[(free // bs * 7 + free % bs) % 11 != cuts[free // bs] % 11][:tokens]
        tokens = len(slots)
        k, v = k[:tokens].contiguous(), v[:tokens].contiguous()
    else:
        slots = torch.randperm(blocks * bs, generator=g, device=DEV)[:tokens]
    pad = torch.zeros(tokens, dtype=torch.bool, device=DEV)
    pad[1::9 if tokens < 100 else 97] = True
    slots[pad] = -1
    d = hss.hss_dims(1, nkv, nkv, hd, 16, bs, blocks)
    size = hss.hss_packed_page_bytes(d)
    cache = torch.randint(0, 256, (blocks, size), generator=g, device=DEV, dtype=torch.uint8)
    before = cache.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = hss.PackTokens(d, slots, tokens, nkv * hd, nkv * hd, status)
    call.pack(k, v, cache)
    torch.cuda.synchronize()
    assert status.item() == 0
    real = (~pad).cpu().numpy()
    where = slots.cpu().numpy()[real]
    got = read_tokens(cache, nkv, bs, hd, where)
    wants = []
    for x, y in ((k, got[0]), (v, got[1])):
        codes, scales = quantise(x.double().cpu().numpy()[real])
        wants.append(codes * np.repeat(scales, 32, -1))
        assert same(y, wants[-1])
    # nothing but those tokens has changed
    left = np.setdiff1d(np.arange(blocks * bs), where)
    for x, y in zip(read_tokens(cache, nkv, bs, hd, left), read_tokens(before, nkv, bs, hd, left)):
        assert same(x, y)
    # read back: rounded once; rows of padding as they were
    back = [torch.full((tokens, nkv, hd), 9.0, device=DEV, dtype=torch.bfloat16)
            for _ in range(2)]
    call.unpack(cache, *back)
    torch.cuda.synchronize()
    for x, want in zip(back, wants):
        y = x.cpu()
        assert (y[~torch.from_numpy(real)] == 9.0).all()
        assert same(y[torch.from_numpy(real)].double().numpy(),
                    torch.from_numpy(want).float().bfloat16().double().numpy())


def test_halves_strides_and_errors():
    hd, nkv, bs, tokens, blocks = 128, 4, 16, 30, 4
    g = torch.Generator(device=DEV).manual_seed(3)
    wide = rows(g, tokens, 2 * nkv + 1, hd)
    slots = torch.arange(tokens, device=DEV) + 9
    slots[4] = blocks * bs
    d = hss.hss_dims(1, nkv, nkv, hd, 16, bs, blocks)
    cache = torch.full((blocks * hss.hss_packed_page_bytes(d),), 0x99, device=DEV,
                       dtype=torch.uint8)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stride = (2 * nkv + 1) * hd
    call = hss.PackTokens(d, slots, tokens, stride, stride, status)
    at = wide.data_ptr()
    real = [i for i in range(tokens) if i != 4]
    where = slots.cpu().numpy()[real]
    first = read_tokens(cache, nkv, bs, hd, where)
    call.pack(None, at + 2 * nkv * hd, cache)
    torch.cuda.synchronize()
    assert status.item() == hss.HSS_ERR_OUT_OF_RANGE
    assert hss.hss_read_device_error() == hss.HSS_ERR_OUT_OF_RANGE
    got = read_tokens(cache, nkv, bs, hd, where)
    assert same(got[0], first[0])  # the keys are left alone
    codes, scales = quantise(wide[:, nkv:2 * nkv].double().cpu().numpy()[real])
    assert same(got[1], codes * np.repeat(scales, 32, -1))
    call.pack(at, None, cache)
    only = torch.zeros(tokens, 2 * nkv + 1, hd, device=DEV, dtype=torch.bfloat16)
    call.unpack(cache, only.data_ptr(), None)
    torch.cuda.synchronize()
    codes, scales = quantise(wide[:, :nkv].double().cpu().numpy()[real])
    want = torch.from_numpy(codes * np.repeat(scales, 32, -1)).float().bfloat16()
    assert torch.equal(only.cpu()[real][:, :nkv], want)
    assert (only[:, nkv:] == 0).all() and (only[4] == 0).all()
    assert same(read_tokens(cache, nkv, bs, hd, where)[1], got[1])
    assert hss.hss_read_device_error() == hss.HSS_ERR_OUT_OF_RANGE  # (again, by those two calls)


def test_slots_past_32_bits():
    """Bytes past 2^32 of a cache, and slots whose byte offset needs 64 bits."""
    hd, nkv, bs = 64, 1, 256
    page = 16 * tile_bytes(hd)
    blocks = (1 << 32) // page + 40
    d = hss.hss_dims(1, nkv, nkv, hd, 16, bs, blocks)
    cache = torch.zeros(blocks * page, device=DEV, dtype=torch.uint8)
    g = torch.Generator(device=DEV).manual_seed(4)
    k, v = rows(g, 3, nkv, hd), rows(g, 3, nkv, hd)
    slots = torch.tensor([blocks * bs - 1, 5, (blocks - 3) * bs + 17], device=DEV)
    call = hss.PackTokens(d, slots, 3, hd, hd)
    call.pack(k, v, cache)
    back = [torch.empty_like(k), torch.empty_like(v)]
    call.unpack(cache, *back)
    tail = cache[-40 * page:].clone()
    torch.cuda.synchronize()
    assert hss.hss_read_device_error() == 0
    for x, y in ((k, back[0]), (v, back[1])):
        codes, scales = quantise(x.double().cpu().numpy())
        assert torch.equal(y.cpu(), torch.from_numpy(
            codes * np.repeat(scales, 32, -1)).float().bfloat16())
    got = read_tokens(tail, nkv, bs, hd, np.array([40 * bs - 1, 37 * bs + 17]))
    codes, scales = quantise(k.double().cpu().numpy()[[0, 2]])
    assert same(got[0], codes * np.repeat(scales, 32, -1))
