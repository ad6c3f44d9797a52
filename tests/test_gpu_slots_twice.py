"""Two tokens that name one slot: each 16 bytes of the slot's rows are one token's or the other's,
and the other slots are as if each had been named once."""
import numpy as np
import pytest
import torch
from test_gpu_rope import DEV, built, turns_table  # noqa: F401 (the fixture builds the library)

import kv_cache_block_lowrank_gb300 as hss

pytestmark = pytest.mark.gpu


def vectors(x):
    return x.contiguous().view(torch.int16).view(-1, 8)


def check(cache, rows, slots):
    """cache [slots, ...] holds rows[i] at slots[i], or of two rows with one slot parts of both."""
    at = {}
    for i, s in enumerate(slots):
        at.setdefault(s, []).append(i)
    for s in range(cache.shape[0]):
        mine = at.get(s, [])
        if not mine:
            assert not cache[s].any()
            continue
        got = vectors(cache[s])
        same = torch.stack([(vectors(rows[i]) == got).all(1) for i in mine])
        assert same.any(0).all()


@pytest.mark.parametrize("n", [2, 5, 700])  # (few tokens are split over several CTAs)
def test_rope_tokens_with_one_slot_twice(n):
    nq, nkv, hd, bs = 32, 8, 128, 16
    blocks = n // bs + 1
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(blocks * bs, generator=g)[:n].tolist()
    slots[1] = slots[0]
    q = torch.randn(n, nq, hd, generator=g).bfloat16().to(DEV)
    k = torch.randn(n, nkv, hd, generator=g).bfloat16().to(DEV)
    v = torch.randn(n, nkv, hd, generator=g).bfloat16().to(DEV)
    turns = torch.from_numpy(turns_table(hd).view(np.int64)).to(DEV)
    call = hss.RopeTokens(hss.hss_dims(1, nq, nkv, hd, 16, bs, blocks), hd, 0, turns, 1.0,
                          torch.arange(n, device=DEV), torch.tensor(slots, device=DEV), n,
                          nq * hd, nkv * hd, nkv * hd)
    kc = torch.zeros(blocks * bs, nkv, hd, device=DEV, dtype=torch.bfloat16)
    vc, q_out, k_out = torch.zeros_like(kc), torch.empty_like(q), torch.empty_like(k)
    call(q, k, v, q_out, k_out, kc, vc)
    torch.cuda.synchronize()
    check(kc, k_out, slots)
    check(vc, v, slots)


def test_write_kv_tokens_with_one_slot_twice():
    n, nkv, hd, r, bs, blocks = 300, 8, 128, 32, 16, 20
    g = torch.Generator().manual_seed(1)
    slots = torch.randperm(blocks * bs, generator=g)[:n].tolist()
    slots[150] = slots[0]
    d = hss.hss_dims(1, 8, nkv, hd, r, bs, blocks)
    P = torch.randn(hd, r, generator=g).bfloat16().to(DEV)
    k = torch.randn(n, nkv, hd, generator=g).bfloat16().to(DEV)
    kc = torch.zeros(blocks, bs, nkv, hd, device=DEV, dtype=torch.bfloat16)
    A = torch.zeros(1, blocks, nkv, bs, r, device=DEV, dtype=torch.bfloat16)
    hss.hss_write_kv_tokens(d, P, k, torch.tensor(slots, device=DEV), n, kc, A, 0)
    # each token's row by itself, in a pool where every slot is named once
    own = torch.zeros_like(A)
    alone = list(range(n))
    hss.hss_write_kv_tokens(d, P, k, torch.tensor(alone, device=DEV), n, None, own, 0)
    torch.cuda.synchronize()
    check(kc.view(-1, nkv, hd), k, slots)
    rows = own[0].transpose(1, 2).reshape(-1, nkv, r)
    check(A[0].transpose(1, 2).reshape(-1, nkv, r), rows[:n], slots)
