"""The packed cache's definition (include/hss.h) in plain numpy and torch, in 64 bits."""
import numpy as np
import torch


def bf16_round(x):
    """float64 array -> the nearest bf16, ties to even, after one rounding to fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16().double().numpy()


def tile_bytes(hd):
    return 18 * hd


def quantise(x):
    """[..., hd] float64 (bf16 values) -> codes (int), scales [..., hd / 32] (float64)."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    finite = np.isfinite(g).all(-1)
    most = np.where(finite, np.abs(np.where(np.isfinite(g), g, 0)).max(-1), 0)
    scale = bf16_round((most.astype(np.float32) / np.float32(7)).astype(np.float64))
    some = scale > 0
    ratio = (np.where(np.isfinite(g), g, 0).astype(np.float32)
             / np.where(some, scale, 1).astype(np.float32)[..., None])
    codes = np.where((some & finite)[..., None], np.clip(np.rint(ratio), -7, 7), 0).astype(int)
    return codes.reshape(x.shape), np.where(finite, scale, np.nan)


def key_place(t, d, hd):
    """Byte and nibble of token t's element d of K in a tile."""
    return t * hd // 2 + d % 32 // 8 * (hd // 8) + d // 32 * 4 + d % 8 // 2, d % 2


def value_place(t, d, hd):
    byte = (d // 64 * 32 + d % 8 * 4 + t % 8 // 2) * 16 + d % 64 // 16 * 4 + t % 2 * 2 + t // 8
    return 8 * hd + byte, d % 16 // 8


def scale_place(t, group, hd, value):
    """bf16 index of a group's scale in a tile."""
    return 8 * hd + (16 * (hd // 32) if value else 0) + t * (hd // 32) + group


def read_tokens(cache, nkv, bs, hd, slots):
    """cache: uint8 tensor -> K and V [len(slots), nkv, hd] float64 (numpy)."""
    raw = cache.reshape(-1).cpu()
    data = raw.numpy().astype(int)
    words = raw.view(torch.bfloat16).double().numpy()
    slots = np.asarray(slots)
    t = (slots % bs % 16)[:, None, None]
    h = np.arange(nkv)[None, :, None]
    d = np.arange(hd)[None, None, :]
    start = (((slots // bs)[:, None, None] * nkv + h) * (bs // 16)
             + (slots % bs // 16)[:, None, None]) * tile_bytes(hd)
    out = []
    for value in (False, True):
        byte, half = (value_place if value else key_place)(t, d, hd)
        code = (data[start + byte] >> (4 * half) & 15) - 8
        out.append(code * words[start // 2 + scale_place(t, d // 32, hd, value)])
    return out


def attend(q, cache, nkv, bs, hd, table, ctx, rows, window, sinks, scale, max_blocks):
    """One sequence.  q [rows, nq, hd] float64 -> out, lse, sum p |v| and the largest sum |q k|."""
    nq = q.shape[1]
    g = nq // nkv
    pos = np.arange(min(ctx + rows, len(table) * bs))
    ids = np.asarray(table)[pos // bs] if len(pos) else np.zeros(0, int)
    known = (ids >= 0) & (ids < max_blocks)
    at = ctx + np.arange(rows)[:, None]
    see = (pos <= at) & known
    if window:
        see &= (pos < sinks) | (pos > at - window)
    any_row = see.any(0) if rows else np.zeros(len(pos), bool)
    k, v = np.zeros((len(pos), nkv, hd)), np.zeros((len(pos), nkv, hd))
    if any_row.any():
        k[any_row], v[any_row] = read_tokens(cache, nkv, bs, hd, ids[any_row] * bs
                                             + pos[any_row] % bs)
    out, size = np.zeros((rows, nq, hd)), np.zeros((rows, nq, hd))
    lse, most = np.full((rows, nq), -np.inf), np.zeros((rows, nq))
    for h in range(nq):
        kh, vh = k[:, h // g], v[:, h // g]
        z = np.where(see, q[:, h] @ kh.T * scale, -np.inf)
        mag = np.where(see, np.abs(q[:, h]) @ np.abs(kh).T * abs(scale), 0)
        for i in range(rows):
            if not see[i].any():
                continue
            top = z[i].max()
            p = np.where(see[i], np.exp(z[i] - top), 0)
            lse[i, h] = top + np.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ vh
            size[i, h] = p @ np.abs(vh)
            most[i, h] = mag[i].max()
    return out, lse, size, most
