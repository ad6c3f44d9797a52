"""hss_norm_rope_tokens against norm and rotation in 64 bits.

Tolerance, from the kernel's arithmetic: the fp32 sum of at most 256 squares is off by up to
256 * 2^-24 of itself, half of that after the root, the reciprocal root and the three products by
a few 2^-23 more, so a normed element by less than 1.2e-5 of itself; the angle by 1e-7 radians; the
result is rounded once to bf16 (2^-8 of it at most):
|got - exact| <= 2^-8 |exact| + 1.5e-5 (|a| + |b|).
"""
import math

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


def turns_of(rot):
    t = [int(round(10000.0 ** (-2 * i / rot) / (2 * math.pi) * 2 ** 64)) for i in range(rot // 2)]
    return t, torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in t], device=DEV)


def exact(x, weight, offset, eps, positions, turns, rot, layout, m):
    """x [n, heads, hd] float64 -> normed and turned, and the sizes of what was added up."""
    y = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * (weight.double().cpu() + offset)
    frac = torch.tensor([[(p * t) % 2 ** 64 / 2.0 ** 64 for t in turns] for p in positions],
                        dtype=torch.float64).reshape(len(positions), -1)
    ang = 2 * math.pi * frac[:, None]
    first = torch.arange(rot // 2) * (2 if layout else 1)
    second = first + (1 if layout else rot // 2)
    z, size = y.clone(), y.abs()
    a, b = y[..., first], y[..., second]
    z[..., first] = m * (a * ang.cos() - b * ang.sin())
    z[..., second] = m * (b * ang.cos() + a * ang.sin())
    size[..., first] = size[..., second] = (a.abs() + b.abs()) * abs(m)
    return z, size


def check(got, want, size):
    off = (got.double().cpu() - want).abs() - (want.abs() * 2.0 ** -8 + 1.5e-5 * size)
    assert off.max().item() <= 0, off.max().item()


CASES = [
    # hd, nq, nkv, bs, rot, layout, tokens, weights ("one", "each", None), offset
    (128, 32, 8, 16, 128, 0, 1, "one", 0.0), (128, 32, 8, 16, 128, 1, 1, "each", 1.0),
    (64, 9, 3, 32, 64, 0, 7, "one", 1.0), (64, 5, 5, 16, 6, 0, 13, "each", 0.0),
    (128, 16, 1, 48, 34, 0, 33, "one", 0.0), (128, 8, 2, 16, 2, 1, 5, None, 5.0),
    (192, 9, 3, 16, 192, 0, 9, "each", 0.0), (192, 4, 4, 64, 64, 1, 17, "one", 1.0),
    (192, 7, 7, 16, 90, 0, 3, "each", 1.0), (256, 6, 2, 128, 256, 1, 11, "one", 0.0),
    (256, 3, 1, 16, 48, 0, 400, "each", 0.0), (128, 64, 8, 16, 128, 0, 700, "one", 0.0),
]


@pytest.mark.parametrize("hd,nq,nkv,bs,rot,layout,tokens,weights,offset", CASES)
def test_against_64_bits(hd, nq, nkv, bs, rot, layout, tokens, weights, offset):
    g = torch.Generator(device=DEV).manual_seed(hd + rot + tokens)
    heads = nq + 2 * nkv
    blocks = tokens // bs + 2
    qkv = torch.randn(tokens, heads * hd + 8, generator=g, device=DEV).mul_(3).bfloat16()
    qkv[::3] *= 100.0
    if tokens > 3:
        qkv[3] = 0.0  # a head of zeros stays zeros
    positions = [(i * 7919 + 3) * (-1 if i % 5 == 4 else 1) for i in range(tokens)]
    slots = torch.randperm(blocks * bs, generator=g, device=DEV)[:tokens]
    pad = torch.zeros(tokens, dtype=torch.bool)
    pad[2::6] = True
    slots[pad.to(DEV)] = -1
    turns, table = turns_of(rot)

    def weight(n):
        shape = {"one": (hd,), "each": (n, hd), None: None}[weights]
        return None if shape is None else torch.randn(shape, generator=g, device=DEV).bfloat16()

    qw, kw = weight(nq), weight(nkv)
    stride = heads * hd + 8
    each = hd if weights == "each" else 0
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = hss.NormRopeTokens(hss.hss_dims(1, nq, nkv, hd, 16, bs, blocks), rot, layout, table,
                              1.25, torch.tensor(positions, device=DEV), slots, tokens, stride,
                              stride, stride, each, each, 1e-5, offset, status)
    q_out = torch.full((tokens, nq, hd), 7.0, device=DEV, dtype=torch.bfloat16)
    k_out = torch.full((tokens, nkv, hd), 7.0, device=DEV, dtype=torch.bfloat16)
    kc, vc = (torch.full((blocks * bs, nkv, hd), 3.0, device=DEV, dtype=torch.bfloat16)
              for _ in range(2))
    at = qkv.data_ptr()
    call(at, at + 2 * nq * hd, at + 2 * (nq + nkv) * hd, qw, kw, q_out, k_out, kc, vc)
    torch.cuda.synchronize()
    assert status.item() == 0
    x = qkv[:, :heads * hd].double().cpu().view(tokens, heads, hd)
    want, size = exact(x[:, :nq], qw, offset, 1e-5, positions, turns, rot, layout, 1.25)
    check(q_out, want, size)
    want, size = exact(x[:, nq:nq + nkv], kw, offset, 1e-5, positions, turns, rot, layout, 1.25)
    check(k_out, want, size)
    real = ~pad
    to = slots.cpu()[real]
    assert torch.equal(kc.cpu()[to], k_out.cpu()[real])
    assert torch.equal(vc.cpu()[to].double(), x[real, nq + nkv:])
    rest = torch.ones(blocks * bs, dtype=torch.bool)
    rest[to] = False
    assert (kc.cpu()[rest] == 3.0).all() and (vc.cpu()[rest] == 3.0).all()


def test_parts_errors_and_another_stream():
    hd, nq, nkv, bs, tokens = 128, 8, 2, 16, 40
    g = torch.Generator(device=DEV).manual_seed(5)
    q = torch.randn(tokens, nq, hd, generator=g, device=DEV).bfloat16()
    k = torch.randn(tokens, nkv, hd, generator=g, device=DEV).bfloat16()
    w = torch.randn(hd, generator=g, device=DEV).bfloat16()
    turns, table = turns_of(hd)
    positions = torch.arange(tokens, device=DEV)
    slots = torch.arange(tokens, device=DEV)
    slots[7] = 3 * bs
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = hss.NormRopeTokens(hss.hss_dims(1, nq, nkv, hd, 16, bs, 3), hd, 0, table, 1.0,
                              positions, slots, tokens, nq * hd, nkv * hd, nkv * hd, 0, 0, 1e-6,
                              0.0, status)
    kc = torch.zeros(3 * bs, nkv, hd, device=DEV, dtype=torch.bfloat16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call(None, k, None, None, w, None, None, kc, None)
    stream.synchronize()
    assert status.item() == hss.HSS_ERR_OUT_OF_RANGE
    assert hss.hss_read_device_error() == hss.HSS_ERR_OUT_OF_RANGE
    want, size = exact(k.double().cpu(), w, 0.0, 1e-6, list(range(tokens)), turns, hd, 0, 1.0)
    real = [i for i in range(tokens) if i != 7]
    check(kc[:tokens][real], want[real], size[real])
    assert (kc[tokens:] == 0).all() and (kc[7] == 0).all()
    # queries alone need no slots; the same bits on every call
    outs = [torch.empty_like(q) for _ in range(2)]
    alone = hss.NormRopeTokens(hss.hss_dims(1, nq, nkv, hd, 16, bs, 3), hd, 0, table, 1.0,
                               positions, None, tokens, nq * hd, nkv * hd, nkv * hd, 0, 0, 1e-6)
    for o in outs:
        alone(q, None, None, w, None, o, None, None, None)
    torch.cuda.synchronize()
    want, size = exact(q.double().cpu(), w, 0.0, 1e-6, list(range(tokens)), turns, hd, 0, 1.0)
    check(outs[0], want, size)
    assert torch.equal(outs[0], outs[1])
