"""hss_rope_tokens against the rotation in 64 bits.

Tolerance, from the kernel's arithmetic: the angle is a whole-number product cut to 2^-32 of a
turn and rounded to fp32 (2^-25 of at most half a turn: 1e-7 radians), sine, cosine and the two
products are fp32 (a few 2^-24 of |a| + |b|), and the result is rounded once to bf16 (2^-8 of
it at most): |got - exact| <= 2^-8 |exact| + 1e-6 (|a| + |b|) |magnitude|.
"""
import math

import numpy as np
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    from kv_cache_block_lowrank_gb300 import _build

    _build.build()
    hss.load()


def turns_table(rot, scaling=0, factor=1.0, ctx=8192.0, low=1.0, high=32.0):
    out = np.zeros(rot // 2, dtype=np.uint64)
    hss.hss_rope_table(hss.hss_rope(rot, scaling, 10000.0, factor, ctx, low, high),
                       out.ctypes.data)
    return out


def exact(x, positions, turns, rot, layout, m):
    """x [n, heads, hd] float64; positions and turns as Python whole numbers."""
    frac = np.array([[(int(p) * int(t)) % 2 ** 64 / 2.0 ** 64 for t in turns] for p in positions])
    ang = torch.from_numpy(2 * math.pi * frac.reshape(len(positions), rot // 2))[:, None]
    first = torch.arange(rot // 2) * (2 if layout else 1)
    second = first + (1 if layout else rot // 2)
    a, b = x[..., first], x[..., second]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., first] = m * (a * ang.cos() - b * ang.sin())
    y[..., second] = m * (b * ang.cos() + a * ang.sin())
    size[..., first] = size[..., second] = (a.abs() + b.abs()) * abs(m)
    return y, size


def check(got, want, size):
    got = got.double().cpu()
    assert got.shape == want.shape
    off = (got - want).abs() - (want.abs() * 2.0 ** -8 + 1e-6 * size)
    assert off.max().item() <= 0, off.max().item()
    still = size == 0
    assert torch.equal(got[still], want[still])  # what is not rotated is copied


CASES = [
    # hd, nq, nkv, bs, rot, layout, tokens
    (128, 32, 8, 16, 128, 0, 1), (128, 32, 8, 16, 128, 1, 1), (128, 8, 8, 16, 64, 0, 3),
    (64, 3, 1, 32, 64, 0, 17), (64, 4, 2, 16, 2, 0, 5), (64, 4, 2, 16, 2, 1, 5),
    (64, 6, 3, 16, 16, 0, 9), (192, 9, 3, 48, 64, 0, 333), (192, 5, 1, 16, 192, 1, 31),
    (192, 4, 4, 16, 190, 0, 12), (256, 16, 2, 256, 256, 0, 65), (256, 7, 7, 16, 74, 0, 20),
    (256, 7, 7, 16, 74, 1, 20), (128, 64, 64, 16, 96, 0, 40), (128, 128, 1, 16, 128, 0, 700),
]


@pytest.mark.parametrize("hd,nq,nkv,bs,rot,layout,n", CASES)
def test_rope_against_64_bits(hd, nq, nkv, bs, rot, layout, n):
    g = torch.Generator().manual_seed(hd + nq + rot + n)
    width = (nq + 2 * nkv) * hd + 8  # a fused projection's rows, and a gap
    qkv = torch.randn(n, width, generator=g).bfloat16()
    pos = torch.randint(0, 1 << 20, (n,), generator=g)
    pos[0] = 0
    if n > 3:
        pos[1], pos[2], pos[3] = -7, (1 << 40) + 3, -(1 << 20)
    blocks = (n + bs - 1) // bs + 1
    slots = torch.randperm(blocks * bs, generator=g)[:n]
    if n > 4:
        slots[4] = -1
    turns = turns_table(rot, 3 if rot > 2 else 0, 4.0)
    m = 1.25
    d = hss.hss_dims(1, nq, nkv, hd, 16, bs, blocks)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    x, kc = qkv.to(DEV), torch.full((blocks, bs, nkv, hd), 7.0, device=DEV).bfloat16()
    vc = kc.clone()
    q_out = torch.empty(n, nq, hd, device=DEV, dtype=torch.bfloat16)
    k_out = torch.empty(n, nkv, hd, device=DEV, dtype=torch.bfloat16)
    call = hss.RopeTokens(d, rot, layout, torch.from_numpy(turns.view(np.int64)).to(DEV), m,
                          pos.to(DEV), slots.to(DEV), n, width, width, width, st)
    at = x.data_ptr()
    call(at, at + 2 * nq * hd, at + 2 * (nq + nkv) * hd, q_out, k_out, kc, vc)
    torch.cuda.synchronize()
    assert st.item() == 0 and hss.hss_read_device_error() == 0

    rows = qkv[:, :width - 8].double().view(n, nq + 2 * nkv, hd)
    want, size = exact(rows[:, :nq + nkv], pos.tolist(), turns.tolist(), rot, layout, m)
    check(q_out, want[:, :nq], size[:, :nq])
    check(k_out, want[:, nq:], size[:, nq:])
    kw = torch.full((blocks * bs, nkv, hd), 7.0, dtype=torch.float64)
    vw, ks = kw.clone(), torch.zeros_like(kw)
    put = slots >= 0
    kw[slots[put]], ks[slots[put]] = want[:, nq:][put], size[:, nq:][put]
    vw[slots[put]] = rows[put][:, nq + nkv:]
    check(kc.view(-1, nkv, hd), kw, ks)
    assert torch.equal(vc.view(-1, nkv, hd).double().cpu(), vw)
    # a second pass over the keys alone writes the same bits
    k2 = torch.empty_like(k_out)
    call(None, at + 2 * nq * hd, None, None, k2, None, None)
    assert torch.equal(k2.view(torch.int16), k_out.view(torch.int16))


def test_rope_turns_back():
    # A rotation by -pos undoes one by pos (up to the two roundings to bf16).
    n, nq, hd = 50, 4, 128
    g = torch.Generator().manual_seed(2)
    x = torch.randn(n, nq, hd, generator=g).bfloat16().to(DEV)
    pos = torch.randint(0, 1 << 17, (n,), generator=g).to(DEV)
    turns = torch.from_numpy(turns_table(hd).view(np.int64)).to(DEV)
    d = hss.hss_dims(1, nq, 1, hd, 16, 16, 4)
    y, z = torch.empty_like(x), torch.empty_like(x)
    hss.RopeTokens(d, hd, 0, turns, 1.0, pos, None, n, nq * hd, hd, hd)(x, None, None, y, None,
                                                                         None, None)
    hss.RopeTokens(d, hd, 0, turns, 1.0, -pos, None, n, nq * hd, hd, hd)(y, None, None, z, None,
                                                                         None, None)
    size = x.float().abs() + x.float().roll(hd // 2, -1).abs()
    assert ((z.float() - x.float()).abs() <= size * 3 * 2.0 ** -8).all()


def test_rope_slot_past_the_pool_is_reported():
    n, nkv, hd, bs = 3, 2, 64, 16
    x = torch.randn(n, nkv, hd).bfloat16().to(DEV)
    turns = torch.from_numpy(turns_table(hd).view(np.int64)).to(DEV)
    slots = torch.tensor([5, 2 * bs, 0]).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    kc = torch.zeros(3, bs, nkv, hd, device=DEV, dtype=torch.bfloat16)  # a block past the pool
    vc = kc.clone()
    hss.hss_read_device_error()
    call = hss.RopeTokens(hss.hss_dims(1, 2, nkv, hd, 16, bs, 2), hd, 1, turns, 1.0,
                          torch.zeros(n, dtype=torch.int64, device=DEV), slots, n, nkv * hd,
                          nkv * hd, nkv * hd, st)
    call(x, x, x, None, None, kc, vc)
    torch.cuda.synchronize()
    assert st.item() == hss.HSS_ERR_OUT_OF_RANGE
    assert hss.hss_read_device_error() == hss.HSS_ERR_OUT_OF_RANGE
    assert torch.equal(vc[0, 5], x[0]) and torch.equal(vc[0, 0], x[2]) and torch.equal(kc, vc)
    assert not vc[2].any() and int((vc != 0).any(-1).any(-1).sum()) == 2


def test_rope_on_another_stream():
    n, nq, nkv, hd, bs = 300, 8, 2, 128, 16
    turns = torch.from_numpy(turns_table(hd).view(np.int64)).to(DEV)
    d = hss.hss_dims(1, nq, nkv, hd, 16, bs, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = torch.randn(n, nq, hd, device=DEV).bfloat16()
        pos = torch.arange(n, device=DEV)
        a, b = torch.empty_like(x), torch.empty_like(x)
        call = hss.RopeTokens(d, hd, 0, turns, 1.0, pos, None, n, nq * hd, nkv * hd, nkv * hd)
        call(x, None, None, a, None, None, None)
    side.synchronize()
    call(x, None, None, b, None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
