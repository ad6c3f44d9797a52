"""hss_norm_rope_tokens of heads whose squares are below fp32's range, with eps 0 and with an eps that
small, against 64 bits.  (Tolerance as in the operator's own tests: 2^-8 of the result for the rounding
to bf16 and 1.5e-5 of what is added up; below 2^-126 a step of 2^-133.)"""
import pytest
import torch

import kv_cache_block_lowrank_gb300 as hss
from test_gpu_norm_rope import DEV, built, exact, turns_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd,rot,layout,nq,tokens", [
    (64, 64, 0, 3, 5), (128, 128, 0, 8, 3), (128, 64, 1, 9, 40), (128, 34, 0, 2, 7),
    (192, 192, 0, 3, 4), (192, 90, 0, 2, 3), (256, 256, 1, 5, 2), (256, 48, 0, 1, 300)])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -110, 2.0 ** -90, 2.0 ** -70])
def test_small_heads(hd, rot, layout, nq, tokens, eps):
    g = torch.Generator(device=DEV).manual_seed(hd + rot)
    nkv = 1
    # a head of every size from 2^-133 to 2^6, one after another
    heads = nq + 2 * nkv
    power = -133 + (torch.arange(tokens * heads) * 7) % 140
    x = torch.randn(tokens, heads, hd, generator=g, device=DEV).double()
    x = (x * power.view(tokens, heads, 1).double().exp2().to(DEV)).bfloat16()
    x[0, 0] = 0.0
    x[0, 0, hd - 1] = 2.0 ** -133          # the smallest there is, alone in its head
    weight = torch.randn(hd, generator=g, device=DEV).bfloat16()
    positions = [3 * i + 1 for i in range(tokens)]
    turns, table = turns_of(rot)
    blocks = tokens // 16 + 1
    call = hss.NormRopeTokens(hss.hss_dims(1, nq, nkv, hd, 16, 16, blocks), rot, layout, table, 1.0,
                              torch.tensor(positions, device=DEV),
                              torch.arange(tokens, device=DEV), tokens, heads * hd, heads * hd,
                              heads * hd, 0, 0, eps)
    q = torch.empty(tokens, nq, hd, device=DEV, dtype=torch.bfloat16)
    k = torch.empty(tokens, nkv, hd, device=DEV, dtype=torch.bfloat16)
    kc, vc = (torch.zeros(blocks * 16, nkv, hd, device=DEV, dtype=torch.bfloat16)
              for _ in range(2))
    at = x.data_ptr()
    call(at, at + 2 * nq * hd, at + 2 * (nq + nkv) * hd, weight, None, q, k, kc, vc)
    torch.cuda.synchronize()
    exact_x = x.double().cpu()
    for got, part, w in ((q, exact_x[:, :nq], weight), (k, exact_x[:, nq:nq + nkv], None)):
        some = (part != 0).any(-1) | (eps > 0)
        want, size = exact(part, w, 0.0, eps, positions, turns, rot, layout, 1.0)
        got = got.double().cpu()
        assert torch.isfinite(got[some]).all()
        room = want.abs() * 2.0 ** -8 + 1.5e-5 * size + 2.0 ** -133
        assert ((got - want).abs() <= room)[some].all(), (got - want).abs()[some].max()
        assert torch.isnan(got[~some]).all()   # 0 / 0
    assert torch.equal(kc[:tokens], k)
    assert torch.equal(vc[:tokens], x[:, nq + nkv:])   # values as they are, however small


def test_a_head_of_zeros():
    """0 / sqrt(eps) is 0; with eps 0 it is no number, in that head alone."""
    hd, table = 128, turns_of(128)[1]
    x = torch.ones(2, 3, hd, device=DEV, dtype=torch.bfloat16)
    x[0, 1] = 0.0
    for eps in (1e-6, 2.0 ** -149, 0.0):
        out = torch.empty(2, 3, hd, device=DEV, dtype=torch.bfloat16)
        hss.NormRopeTokens(hss.hss_dims(1, 3, 3, hd, 16, 16, 1), hd, 0, table, 1.0,
                           torch.arange(2, device=DEV), None, 2, 3 * hd, 0, 0, 0, 0, eps)(
            x, None, None, None, None, out, None, None, None)
        torch.cuda.synchronize()
        zero = out[0, 1]
        assert (torch.isnan(zero) if eps == 0 else zero == 0).all()
        out[0, 1] = 1.0
        assert torch.isfinite(out).all()
