"""Workloads of the four-bit paged cache and its pages: normed rotary writes, packing, windowed
attention over packed pages, forking and compacting pages.

Each case is one call of one operator (a plan of page copies is followed by the copies) at a size
that a serving loop meets.  ``run`` computes it either through the library (``own`` true) or in
elementary torch operations in 32 bits.
"""
from __future__ import annotations

import math

import torch

own = False

NEG = float("-inf")
GROUP = 32  # elements of a head that share a scale
EPS = 1e-6


# ------------------------------------------------------------------------------------ cases

def _norm(name, tokens, nq, nkv, hd, rot, layout, per_head, plus_one, far, bs):
    return {"name": name, "op": "norm", "tokens": tokens, "nq": nq, "nkv": nkv, "hd": hd,
            "rot": rot, "layout": layout, "per_head": per_head, "plus_one": plus_one, "far": far,
            "bs": bs}


def _pack(name, tokens, nkv, hd, bs, single):
    return {"name": name, "op": "pack", "tokens": tokens, "nkv": nkv, "hd": hd, "bs": bs,
            "single": single}


def _attend(name, seqs, lo, hi, rows_lo, rows_hi, window, sinks, nq, nkv, hd, bs):
    return {"name": name, "op": "attend", "seqs": seqs, "ctx_lo": lo, "ctx_hi": hi,
            "rows_lo": rows_lo, "rows_hi": rows_hi, "window": window, "sinks": sinks, "nq": nq,
            "nkv": nkv, "hd": hd, "bs": bs}


def _fork(name, seqs, new, lo, hi, prefix, bs, nkv, hd, layers):
    return {"name": name, "op": "fork", "seqs": seqs, "new": new, "blocks_lo": lo,
            "blocks_hi": hi, "prefix": prefix, "bs": bs, "nkv": nkv, "hd": hd, "layers": layers}


def _compact(name, seqs, lo, hi, share, moves, bs, nkv, hd, layers):
    return {"name": name, "op": "compact", "seqs": seqs, "blocks_lo": lo, "blocks_hi": hi,
            "share": share, "moves": moves, "bs": bs, "nkv": nkv, "hd": hd, "layers": layers}


def listed():
    return [
        # One new token of each of 16 sequences: a decode step's write, where latency counts.
        _norm("norm_decode_16", 16, 32, 8, 128, 128, "half", False, False, 32768, 16),
        # A whole prefill chunk, with weights for every head.
        _norm("norm_prefill_8192", 8192, 64, 8, 128, 64, "interleaved", True, True, 131072, 16),
        # One new token of each of 64 sequences, packed into their pages.
        _pack("pack_decode_64", 64, 8, 128, 16, True),
        # A ragged prompt of an odd number of tokens.
        _pack("pack_prompt_8191", 8191, 8, 128, 32, False),
        # Single-token decode of one long sequence.
        _attend("decode_1x32768", 1, 32768, 32768, 1, 1, 0, 0, 32, 8, 128, 16),
        # Batched decode at mixed lengths.
        _attend("decode_64_ragged", 64, 1024, 16384, 1, 1, 0, 0, 32, 8, 128, 16),
        # A few drafted tokens over a window and the first tokens, empty and short contexts among
        # long ones, three query heads a kv head.
        _attend("window_16_odd", 16, 0, 100001, 1, 5, 4093, 5, 24, 8, 64, 32),
        # A prompt chunk over a long context.
        _attend("chunk_512x32768", 1, 32768, 32768, 512, 512, 0, 0, 64, 8, 128, 16),
        # Beams of four prompts put in a new order: their last pages part ways.
        _fork("fork_16_beams", 4, 16, 16, 64, 4, 16, 8, 128, 8),
        # A batch after a verified draft: sequences cut back, forked, dropped and grown.
        _fork("fork_256", 256, 256, 16, 128, 8, 16, 8, 128, 4),
        # A few pages moved down between two steps.
        _compact("compact_8_moves", 32, 1, 64, 0.9, 8, 16, 8, 128, 8),
        # A pool half empty, its pages moved to the front.
        _compact("compact_half", 128, 1, 128, 0.5, 1 << 20, 16, 8, 128, 4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "pack", "attend", "attend", "attend", "fork", "compact"])
    bs = rng.choice([16, 16, 32, 48, 64, 128])
    g, nkv = rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([1, 2, 3, 4, 8])
    hd = rng.choice([64, 128, 128, 192, 256])
    if op == "norm":
        tokens = _log_int(rng, 1, 8192)
        rot = 2 * rng.randint(1, hd // 2) if rng.random() < 0.5 else hd
        tokens = min(tokens, 8192 * 80 * 128 // ((g + 2) * nkv * hd))
        c = _norm("", tokens, g * nkv, nkv, hd, rot, rng.choice(["half", "interleaved"]),
                  rng.random() < 0.5, rng.random() < 0.5, _log_int(rng, 128, 1 << 20), bs)
    elif op == "pack":
        single = rng.random() < 0.4
        tokens = _log_int(rng, 1, 256 if single else 8192)
        tokens = max(1, min(tokens, 8191 * 8 * 128 // (nkv * hd)))
        c = _pack("", tokens, nkv, hd, bs, single)
    elif op == "attend":
        seqs, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 131072)
        rows = 1 if rng.random() < 0.4 else _log_int(rng, 2, 512)
        window = 0 if rng.random() < 0.5 else _log_int(rng, 1, 8192)
        sinks = 0 if window == 0 else rng.choice([0, 1, 4, 16, 129])
        # no more work than the largest listed cases: rows times tokens, and bytes of cache
        while (seqs * rows * g * nkv * (hi + rows) * hd > 512 * 64 * 32768 * 128
               or seqs * nkv * (hi + rows) * hd > 64 * 8 * 16384 * 128):
            seqs, hi, rows = max(1, seqs // 2), max(1, hi // 2), max(1, rows * 3 // 4)
        lo = rng.choice([0, hi // 2, hi])
        c = _attend("", seqs, lo, hi, max(1, rows // rng.choice([1, 1, 3])), rows, window, sinks,
                    g * nkv, nkv, hd, bs)
    else:
        bs = rng.choice([16, 16, 32])
        layers, hi = rng.choice([1, 2, 4]), _log_int(rng, 2, 128)
        seqs = _log_int(rng, 1, 256)
        while seqs * hi * layers * bs * nkv * hd > 128 * 64 * 4 * 16 * 8 * 128:
            seqs, hi = max(1, seqs // 2), max(2, hi * 3 // 4)
        lo = rng.choice([1, (hi + 1) // 2, hi])
        if op == "fork":
            c = _fork("", seqs, max(1, rng.choice([seqs, seqs // 2, seqs * 2])), lo, hi,
                      min(lo, rng.choice([0, 1, 8])), bs, nkv, hd, layers)
        else:
            c = _compact("", seqs, lo, hi, rng.choice([0.3, 0.6, 0.95]),
                         rng.choice([1, 16, 1 << 20]), bs, nkv, hd, layers)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs

def _gens(seed):
    host = torch.Generator(device="cpu")
    host.manual_seed(int(seed))
    dev = torch.Generator(device="cuda")
    dev.manual_seed(int(seed) + 1)
    return host, dev


def _bf16(gen, *shape, std=1.0):
    x = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    return x.normal_(0.0, std, generator=gen)


def _ints(gen, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=gen)


def _spread(lo, hi, n, turn=0):
    """n whole numbers spread evenly over [lo, hi], rotated by `turn` places: the same for every
    seed, so that a case's outputs keep their shapes."""
    x = torch.linspace(lo, hi, n, dtype=torch.float64).round().long() if n > 1 \
        else torch.tensor([hi])
    return x.roll(turn)


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])


def _turns(rot):
    """The pairs' frequencies for base 10000 as 64-bit fixed-point fractions of a turn."""
    turns = [int(round(10000.0 ** (-2.0 * i / rot) / (2 * math.pi) * 2.0 ** 64))
             for i in range(rot // 2)]
    return torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns])


def _prepare_norm(case, host, dev):
    n, nq, nkv, hd, bs = (case[k] for k in ("tokens", "nq", "nkv", "hd", "bs"))
    base = 0.0 if case["plus_one"] else 1.0
    shape = (lambda heads: (heads, hd)) if case["per_head"] else (lambda heads: (hd,))
    blocks = (n + bs - 1) // bs + 2
    # the rows of a fused projection: queries, keys and values side by side
    return {"case": case, "qkv": _bf16(dev, n, (nq + 2 * nkv) * hd, std=3.0), "kept": {},
            "positions": _ints(host, 0, case["far"], n).cuda(),
            "slots": torch.randperm(blocks * bs, generator=host)[:n].cuda(),
            "turns": _turns(case["rot"]).cuda(),
            "q_weight": (_bf16(dev, *shape(nq), std=0.2) + base),
            "k_weight": (_bf16(dev, *shape(nkv), std=0.2) + base),
            "q_out": torch.empty(n, nq, hd, device="cuda", dtype=torch.bfloat16),
            "k_cache": _bf16(dev, blocks, bs, nkv, hd), "v_cache": _bf16(dev, blocks, bs, nkv, hd)}


def _tile_bytes(hd):
    """Bytes of 16 tokens of one head: codes of K and V, then their scales."""
    return 2 * 16 * (hd // 2) + 2 * 16 * (hd // GROUP) * 2


def _prepare_pack(case, host, dev):
    n, nkv, hd, bs = (case[k] for k in ("tokens", "nkv", "hd", "bs"))
    if case["single"]:  # a token of each of n sequences, every one in a page of its own
        blocks = n + n // 4 + 1
        slots = torch.randperm(blocks, generator=host)[:n] * bs + _ints(host, 0, bs - 1, n)
    else:  # a prompt's tokens, beginning inside a page
        blocks = (n + bs - 1) // bs + 3
        at = torch.arange(n) + bs // 3
        slots = torch.randperm(blocks, generator=host)[at // bs] * bs + at % bs
    # heads of a wide range of sizes, with the channels that stand out in keys
    size = torch.empty(nkv, hd, device="cuda").log_normal_(0.0, 1.0, generator=dev)
    rows = (_bf16(dev, n, 2, nkv, hd).float() * size).bfloat16()
    cache = torch.randint(0, 256, (blocks, nkv, bs // 16, _tile_bytes(hd)), generator=dev,
                          device="cuda", dtype=torch.uint8)
    return {"case": case, "rows": rows, "slots": slots.cuda(), "cache": cache, "kept": {},
            "seven": torch.full((1,), 7.0, device="cuda")}


def _packed_pages(dev, blocks, nkv, bs, hd):
    """Pages of normal keys and values: codes by the quantiles of a byte, scales around a third."""
    quantile = (torch.arange(256, dtype=torch.float64) + 0.5) / 256
    code = (torch.special.ndtri(quantile) * 2.6).round().clamp(-7, 7).long() + 8
    pair = (code[:, None] * 16 + code[None, :]).flatten().to(torch.uint8).cuda()
    tiles, size = blocks * nkv * (bs // 16), _tile_bytes(hd)
    cache = torch.empty(tiles, size, device="cuda", dtype=torch.uint8)
    codes = 16 * hd
    for first in range(0, tiles, 1 << 16):  # in pieces: the indexes take eight bytes each
        part = cache[first:first + (1 << 16)]
        index = torch.randint(0, 65536, (part.shape[0], codes), generator=dev, device="cuda",
                              dtype=torch.int32)
        part[:, :codes] = pair[index]
        scale = torch.rand(part.shape[0], (size - codes) // 2, generator=dev, device="cuda")
        part[:, codes:] = (0.2 + 0.3 * scale).bfloat16().view(torch.uint8)
    return cache.view(blocks, nkv, bs // 16, size)


def _prepare_attend(case, host, dev):
    nq, nkv, hd, bs, seqs = (case[k] for k in ("nq", "nkv", "hd", "bs", "seqs"))
    # lengths and row counts are paired the same way for every seed; their order is not
    order = torch.randperm(seqs, generator=host)
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], seqs)[order]
    rows = _spread(case["rows_lo"], case["rows_hi"], seqs, seqs // 3)[order]
    blocks = (ctx + rows + bs - 1) // bs
    total_blocks, total_q, max_q = int(blocks.sum()), int(rows.sum()), int(rows.max())
    max_blocks = total_blocks + total_blocks // 8 + 1
    table = torch.randperm(max_blocks, generator=host)[:total_blocks].int()
    return {"case": case, "ctx_len": ctx.int().cuda(), "q_offsets": _offsets(rows).int().cuda(),
            "seq_offsets": _offsets(blocks).int().cuda(), "table": table.cuda(),
            "total_q": total_q, "max_q": max_q, "total_blocks": total_blocks,
            "longest": int((ctx + rows).max()), "max_blocks": max_blocks,
            "q": _bf16(dev, total_q, nq, hd, std=1.5),
            "cache": _packed_pages(dev, max_blocks, nkv, bs, hd),
            "scale": 1.0 / math.sqrt(hd), "kept": {}}


def _prepare_fork(case, host, dev):
    bs, seqs, new = case["bs"], case["seqs"], case["new"]
    order = torch.randperm(seqs, generator=host)
    n = _spread(case["blocks_lo"], case["blocks_hi"], seqs)[order]
    held = n * bs - _ints(host, 0, bs - 1, seqs)                     # tokens of a sequence
    # a few are dropped, some begin anew, and the rest is taken up by one or more
    parents = _ints(host, 0, seqs - 1, new)
    parents[torch.rand(new, generator=host) < 0.05] = -1
    lengths = (held[parents.clamp(min=0)] - _ints(host, 0, 7, new)).clamp(min=0)
    room = _ints(host, 1, 8, new)
    most = int((case["blocks_hi"] * bs + 8 + bs - 1) // bs)
    distinct = int((n - case["prefix"]).clamp(min=0).sum()) + case["prefix"] + 5
    pages = distinct + 2 * new + distinct // 4
    ids = torch.randperm(pages, generator=host)
    # a common prefix, then pages of their own, then pages that a prefix cache alone holds
    own_pages = case["prefix"] + torch.arange(int(n.sum()))
    at = torch.arange(int(n.sum())) - _offsets(n)[:-1].repeat_interleave(n)
    first_own = (at < case["prefix"]).long().cumsum(0)
    index = torch.where(at < case["prefix"], at, own_pages - first_own)
    table = ids[index]
    refs = torch.bincount(table, minlength=pages)
    refs[ids[distinct - 5:distinct]] += 1
    refs[ids[:case["prefix"]]] += 1
    return {"case": case, "table": table.int().cuda(), "seq_offsets": _offsets(n).int().cuda(),
            "total": int(n.sum()), "refs": refs.int().cuda(), "pages": pages,
            "parents": parents.int().cuda(), "lengths": lengths.int().cuda(),
            "room": room.int().cuda(), "table_room": new * most, "kept": {},
            "k_cache": _bf16(dev, case["layers"], pages, bs, case["nkv"], case["hd"]),
            "v_cache": _bf16(dev, case["layers"], pages, bs, case["nkv"], case["hd"])}


def _prepare_compact(case, host, dev):
    bs, seqs = case["bs"], case["seqs"]
    order = torch.randperm(seqs, generator=host)
    n = _spread(case["blocks_lo"], case["blocks_hi"], seqs)[order]
    total = int(n.sum())
    pages = int(total / case["share"]) + 3
    # every eighth page is shared by two sequences
    own_pages = torch.randperm(pages, generator=host)
    again = torch.arange(total) % 8 == 7
    index = torch.arange(total) - again.long().cumsum(0)
    table = own_pages[index]
    refs = torch.bincount(table, minlength=pages)
    return {"case": case, "table": table.int().cuda(), "total": total, "refs": refs.int().cuda(),
            "pages": pages, "move_room": min(case["moves"], pages), "kept": {},
            "k_cache": _bf16(dev, case["layers"], pages, bs, case["nkv"], case["hd"]),
            "v_cache": _bf16(dev, case["layers"], pages, bs, case["nkv"], case["hd"])}


def prepare(case, seed):
    host, dev = _gens(seed)
    return {"norm": _prepare_norm, "pack": _prepare_pack, "attend": _prepare_attend,
            "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](dict(case), host, dev)


# ------------------------------------------------------------------------- the library's calls

def _dims(case, max_blocks):
    import kv_cache_block_lowrank_gb300 as hss

    return hss.hss_dims(case.get("layers", 1), case.get("nq", case["nkv"]), case["nkv"],
                        case["hd"], 16, case["bs"], max_blocks)


def _own_norm(s):
    import kv_cache_block_lowrank_gb300 as hss

    case, kept = s["case"], s["kept"]
    nq, nkv, hd, n = case["nq"], case["nkv"], case["hd"], case["tokens"]
    if "call" not in kept:  # what the layers of a step share
        layout = hss.HSS_ROPE_HALF if case["layout"] == "half" else hss.HSS_ROPE_INTERLEAVED
        stride = (nq + 2 * nkv) * hd
        each = hd if case["per_head"] else 0
        kept["call"] = hss.NormRopeTokens(_dims(case, s["k_cache"].shape[0]), case["rot"], layout,
                                          s["turns"], 1.0, s["positions"], s["slots"], n, stride,
                                          stride, stride, each, each, EPS,
                                          1.0 if case["plus_one"] else 0.0)
    at = s["qkv"].data_ptr()
    kept["call"](at, at + 2 * nq * hd, at + 2 * (nq + nkv) * hd, s["q_weight"], s["k_weight"],
                 s["q_out"], None, s["k_cache"], s["v_cache"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_pack(s):
    import kv_cache_block_lowrank_gb300 as hss

    case, kept = s["case"], s["kept"]
    n, nkv, hd = case["tokens"], case["nkv"], case["hd"]
    if "call" not in kept:
        kept["call"] = hss.PackTokens(_dims(case, s["cache"].shape[0]), s["slots"], n,
                                      2 * nkv * hd, 2 * nkv * hd)
    at = s["rows"].data_ptr()
    kept["call"].pack(at, at + 2 * nkv * hd, s["cache"])
    back = torch.empty_like(s["rows"])
    at = back.data_ptr()
    kept["call"].unpack(s["cache"], at, at + 2 * nkv * hd)
    return {"k": back[:, 0], "v": back[:, 1]}


def _own_attend(s):
    import kv_cache_block_lowrank_gb300 as hss

    case, kept = s["case"], s["kept"]
    if "call" not in kept:  # the layers of a step share tables, lengths and workspace
        dims = _dims(case, s["max_blocks"])
        size = hss.hss_attend_packed_workspace_bytes(dims, case["seqs"], s["max_q"],
                                                     s["total_blocks"], case["window"],
                                                     case["sinks"])
        work = torch.zeros(size, dtype=torch.uint8, device="cuda")
        kept["call"] = hss.AttendPacked(dims, s["q_offsets"], s["total_q"], s["max_q"],
                                        s["table"], s["seq_offsets"], s["ctx_len"], case["seqs"],
                                        s["total_blocks"], case["window"], case["sinks"],
                                        s["scale"], work, size)
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["total_q"], case["nq"], device="cuda")
    kept["call"](s["q"], s["cache"], out, lse)
    return {"out": out, "lse": lse}


def _own_copies(s, src, dst, counts, most):
    import kv_cache_block_lowrank_gb300 as hss

    case = s["case"]
    page = case["bs"] * case["nkv"] * case["hd"] * 2
    hss.hss_copy_pages(src, dst, counts, most, s["k_cache"], s["v_cache"], page, s["pages"],
                       case["layers"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_fork(s):
    import kv_cache_block_lowrank_gb300 as hss

    case, kept = s["case"], s["kept"]
    new, i32 = case["new"], {"dtype": torch.int32, "device": "cuda"}
    if "work" not in kept:
        kept["size"] = hss.hss_fork_pages_workspace_bytes(new, s["pages"])
        kept["work"] = torch.zeros(kept["size"], dtype=torch.uint8, device="cuda")
    table, offsets = torch.empty(s["table_room"], **i32), torch.empty(new + 1, **i32)
    refs, moves, counts = torch.empty_like(s["refs"]), torch.empty(2, new, **i32), \
        torch.empty(4, **i32)
    hss.hss_fork_pages(s["table"], s["seq_offsets"], case["seqs"], s["total"], s["refs"],
                       s["pages"], None, 0, s["parents"], s["lengths"], s["room"], new,
                       case["bs"], s["table_room"], table, offsets, refs, moves[0], moves[1],
                       counts, kept["work"], kept["size"])
    return {"table": table, "offsets": offsets, "refs": refs, "src": moves[0], "dst": moves[1],
            "counts": counts} | _own_copies(s, moves[0], moves[1], counts[1:], new)


def _own_compact(s):
    import kv_cache_block_lowrank_gb300 as hss

    kept, i32 = s["kept"], {"dtype": torch.int32, "device": "cuda"}
    room = s["move_room"]
    if "work" not in kept:
        kept["size"] = hss.hss_compact_pages_workspace_bytes(s["pages"])
        kept["work"] = torch.zeros(kept["size"], dtype=torch.uint8, device="cuda")
    table, refs = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    moves, counts = torch.empty(2, room, **i32), torch.empty(4, **i32)
    hss.hss_compact_pages(s["table"], s["total"], s["refs"], s["pages"], room, table, refs,
                          moves[0], moves[1], counts, kept["work"], kept["size"])
    return {"table": table, "refs": refs, "src": moves[0], "dst": moves[1],
            "counts": counts} | _own_copies(s, moves[0], moves[1], counts, room)


# ----------------------------------------------------------------------------- the plain forms

def _plain_norm(s):
    case = s["case"]
    nq, nkv, hd, rot, n = (case[k] for k in ("nq", "nkv", "hd", "rot", "tokens"))
    # 64-bit products wrap: what is left is the fraction of a turn, signed, in 2^-64
    part = s["positions"][:, None] * s["turns"][None, :]
    angle = (part >> 32).float() * (2.0 * math.pi / 2.0 ** 32)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    x = s["qkv"].view(n, nq + 2 * nkv, hd)
    weight = torch.cat([s["q_weight"].expand(nq, hd), s["k_weight"].expand(nkv, hd)]).float()
    if case["plus_one"]:
        weight = weight + 1.0
    qk = x[:, :nq + nkv].float()
    qk = qk * torch.rsqrt((qk * qk).mean(-1, keepdim=True) + EPS) * weight
    if case["layout"] == "half":
        a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    turned = torch.cat([turned, qk[..., rot:]], -1).bfloat16()
    s["q_out"].copy_(turned[:, :nq])
    s["k_cache"].view(-1, nkv, hd).index_copy_(0, s["slots"], turned[:, nq:])
    s["v_cache"].view(-1, nkv, hd).index_copy_(0, s["slots"], x[:, nq + nkv:])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_pack(s):
    case = s["case"]
    n, nkv, hd = case["tokens"], case["nkv"], case["hd"]
    x = s["rows"].float().view(n, 2, nkv, hd // GROUP, GROUP)
    scale = (x.abs().amax(-1, keepdim=True) / s["seven"]).bfloat16().float()
    some = scale > 0
    code = (x / torch.where(some, scale, torch.ones_like(scale))).round().clamp(-7, 7) * some
    values = (code * scale).bfloat16().view(n, 2, nkv, hd)
    return {"k": values[:, 0], "v": values[:, 1]}


def _plain_values(tiles, hd):
    """K and V, [..., 16, hd] in 32 bits, of tiles of 16 packed tokens [..., bytes]."""
    lead, half = tiles.shape[:-1], 16 * (hd // 2)
    groups = hd // GROUP

    def halves(x):  # the low and the high four bits of each byte
        return torch.stack([x & 15, x >> 4], -1)

    k = halves(tiles[..., :half].view(*lead, 16, 4, groups, 4)).transpose(-4, -3)
    k = k.reshape(*lead, 16, groups, GROUP).float() - 8.0
    # [64 dims, dim % 8, token pair, 16 dims, token % 2, token / 8, half of the 16]
    v = halves(tiles[..., half:2 * half].view(*lead, hd // 64, 8, 4, 4, 2, 2))
    d = len(lead)
    v = v.permute(*range(d), d + 5, d + 2, d + 4, d, d + 3, d + 6, d + 1)
    v = v.reshape(*lead, 16, groups, GROUP).float() - 8.0
    scales = tiles[..., 2 * half:].contiguous().view(torch.bfloat16).float()
    scales = scales.view(*lead, 2, 16, groups, 1)
    k = k * scales[..., 0, :, :, :]
    v = v * scales[..., 1, :, :, :]
    return k.view(*lead, 16, hd), v.view(*lead, 16, hd)


def _plain_attend(s):
    case = s["case"]
    nq, nkv, hd, bs, seqs = (case[k] for k in ("nq", "nkv", "hd", "bs", "seqs"))
    g, rows_max = nq // nkv, s["max_q"]
    window = case["window"] if case["window"] > 0 else 1 << 30
    sinks = case["sinks"]
    offs, q0 = s["seq_offsets"].long(), s["q_offsets"].long()
    rows, ctx = q0[1:] - q0[:-1], s["ctx_len"].long()
    # the tiles of 16 tokens that any row sees: the first tokens', then the window's
    sink_tiles = min((sinks + 15) // 16, (s["longest"] + 15) // 16)
    most = min((s["longest"] + 15) // 16, sink_tiles + (window + rows_max + 29) // 16)
    start = ((ctx + 1 - window).clamp(min=0) // 16).clamp(min=sink_tiles)
    k_at = torch.arange(most, device="cuda")
    tile = torch.where(k_at < sink_tiles, k_at, start[:, None] + k_at - sink_tiles)
    pos = (tile[..., None] * 16 + torch.arange(16, device="cuda")).view(seqs, -1)
    entry = (offs[:-1, None] + tile * 16 // bs).clamp(max=s["total_blocks"] - 1)
    tiles = s["cache"][s["table"].long()[entry], :, tile * 16 % bs // 16]
    row = (q0[:-1, None] + torch.arange(rows_max, device="cuda")).clamp(max=s["total_q"] - 1)
    q = s["q"][row].float().view(seqs, rows_max, nkv, g, hd).permute(0, 2, 1, 3, 4)
    k, v = _plain_values(tiles.transpose(1, 2), hd)   # [seqs, nkv, most, 16, hd]
    del tiles
    score = q.reshape(seqs, nkv, rows_max * g, hd) @ k.view(seqs, nkv, most * 16, hd).mT
    score = score.mul_(s["scale"])
    del k
    i = torch.arange(rows_max, device="cuda")
    at = (ctx[:, None] + i)[:, :, None]                # a row's own position
    p = pos[:, None, :]
    see = (p <= at) & ((p < sinks) | (p > at - window)) & (i < rows[:, None])[:, :, None]
    score = score.view(seqs, nkv, rows_max, g, -1).masked_fill_(~see[:, None, :, None], NEG)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = weight.view(seqs, nkv, rows_max * g, -1) @ v.reshape(seqs, nkv, most * 16, hd)
    out = out.view(seqs, nkv, rows_max, g, hd) / torch.where(total > 0, total,
                                                             torch.ones_like(total))
    lse = (top + total.log()).view(seqs, nkv, rows_max, g)
    # back to the rows as they are packed
    seq_of = torch.repeat_interleave(torch.arange(seqs, device="cuda"), rows,
                                     output_size=s["total_q"])
    row_of = torch.arange(s["total_q"], device="cuda") - q0[seq_of]
    out = out.permute(0, 2, 1, 3, 4)[seq_of, row_of].reshape(s["total_q"], nq, hd).bfloat16()
    return {"out": out, "lse": lse.permute(0, 2, 1, 3)[seq_of, row_of].reshape(s["total_q"], nq)}


def _plain_copies(s, src, dst):
    there = (src >= 0) & (dst >= 0)
    a, b = src[there].long(), dst[there].long()
    for name in ("k_cache", "v_cache"):
        s[name][:, b] = s[name][:, a]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_fork(s):
    case, dev = s["case"], "cuda"
    bs, new, room_all, pages = case["bs"], case["new"], s["table_room"], s["pages"]
    offs, parents = s["seq_offsets"].long(), s["parents"].long()
    some, p = parents >= 0, parents.clamp(min=0)
    has = torch.where(some, offs[p + 1] - offs[p], torch.zeros_like(p))
    length = torch.minimum(s["lengths"].long().clamp(min=0), has * bs)
    kept = (length + bs - 1) // bs
    room = s["room"].long().clamp(min=0)
    n = (length + room + bs - 1) // bs
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    new_offs = torch.cat([zero, n.cumsum(0)])
    at = torch.arange(room_all, device=dev)
    owner = torch.searchsorted(new_offs[1:].contiguous(), at, right=True).clamp(max=new - 1)
    j = at - new_offs[owner]
    real = at < new_offs[-1]
    stays = real & (j < kept[owner])
    old = s["table"].long()
    ids = old[(offs[p[owner]] + j).clamp(0, s["total"] - 1)]
    refs = s["refs"].clone()
    refs.index_add_(0, old, torch.full_like(s["table"], -1))
    refs.index_add_(0, ids, stays.int())
    # a page that is written from its middle on goes on belonging to one sequence only
    writer = (length % bs != 0) & (room > 0)
    page = old[(offs[p] + kept - 1).clamp(0, s["total"] - 1)]
    number = torch.arange(new, dtype=torch.int32, device=dev)
    writers = torch.zeros(pages, dtype=torch.int32, device=dev).index_add_(0, page, writer.int())
    first = torch.full((pages,), new, dtype=torch.int32, device=dev).scatter_reduce_(
        0, page, torch.where(writer, number, torch.full_like(number, new)), "amin")
    keeps = (refs[page] == writers[page]) & (first[page] == number)
    copies = writer & ~keeps
    refs.index_add_(0, page, -copies.int())
    fresh = real & ((j >= kept[owner]) | (copies[owner] & (j == kept[owner] - 1)))
    rank = fresh.cumsum(0) - 1
    free = (refs != 0).to(torch.int8).argsort(stable=True)
    count = (refs == 0).sum()
    got = fresh & (rank < count)
    taken = torch.where(got, free[rank.clamp(0, pages - 1)], torch.full_like(rank, -1))
    table = torch.where(fresh, taken, torch.where(stays, ids, torch.full_like(ids, -1))).int()
    spare = torch.cat([refs, torch.zeros(1, dtype=torch.int32, device=dev)])
    spare[torch.where(got, taken, torch.full_like(taken, pages))] = 1
    refs = spare[:pages]
    to = torch.where(copies, copies.cumsum(0) - 1, torch.full_like(p, new))
    src, dst = (torch.full((new + 1,), -1, dtype=torch.int32, device=dev) for _ in range(2))
    src[to] = page.int()
    dst[to] = table[(new_offs[:-1] + kept - 1).clamp(0, room_all - 1)]
    counts = torch.stack([new_offs[-1], copies.sum(), (refs != 0).sum(),
                          (fresh & ~got).sum()]).int()
    return {"table": table, "offsets": new_offs.int(), "refs": refs, "src": src[:new],
            "dst": dst[:new], "counts": counts} | _plain_copies(s, src[:new], dst[:new])


def _plain_compact(s):
    pages, most, dev = s["pages"], s["move_room"], "cuda"
    used = s["refs"] != 0
    count = used.sum()
    page = torch.arange(pages, device=dev)
    hole = ~used & (page < count)
    above = used & (page >= count)
    # the lowest hole takes the highest page, and so on
    holes = torch.where(hole, page, torch.full_like(page, pages)).sort().values[:most]
    tops = torch.where(above, page, torch.full_like(page, -1)).sort(descending=True).values
    made = torch.arange(most, device=dev) < above.sum()
    src = torch.where(made, tops[:most], torch.full_like(holes, -1))
    dst = torch.where(made, holes, torch.full_like(holes, -1))
    goes = torch.cat([page, page[:1]])
    goes[torch.where(made, src, torch.full_like(src, pages))] = dst
    refs = torch.cat([s["refs"], s["refs"][:1]])
    refs[torch.where(made, dst, torch.full_like(dst, pages))] = s["refs"][src.clamp(min=0)]
    refs[torch.where(made, src, torch.full_like(src, pages))] = 0
    refs = refs[:pages]
    table = goes[s["table"].long()].int()
    last = torch.where(refs != 0, page + 1, torch.zeros_like(page)).max()
    counts = torch.stack([made.sum(), count, last, above.sum() - made.sum()]).int()
    src, dst = src.int(), dst.int()
    return {"table": table, "refs": refs, "src": src, "dst": dst,
            "counts": counts} | _plain_copies(s, src, dst)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "pack": _own_pack, "attend": _own_attend, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"norm": _plain_norm, "pack": _plain_pack, "attend": _plain_attend,
            "fork": _plain_fork, "compact": _plain_compact}[op](state)


# ------------------------------------------------------------------------------- work, 64 bits

def _seen(case):
    """Tokens that any row of a sequence sees, and pairs of a row and a token it sees, over all
    sequences."""
    seqs = case["seqs"]
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], seqs).tolist()
    rows = _spread(case["rows_lo"], case["rows_hi"], seqs, seqs // 3).tolist()
    window, sinks = case["window"] or 1 << 30, case["sinks"]
    tokens = pairs = 0
    for c, t in zip(ctx, rows):
        first = max(0, c + 1 - window)
        tokens += c + t - first + min(sinks, first)
        for at in range(c, c + t):
            first = max(0, at + 1 - window)
            pairs += at + 1 - first + min(sinks, first)
    return tokens, pairs, sum(rows)


def work(case):
    if case["op"] == "norm":
        heads = case["nq"] + 2 * case["nkv"]
        turned = case["nq"] + case["nkv"]
        # every row read and written, and a position, a slot and (once) weights and frequencies
        data = case["tokens"] * (heads * case["hd"] * 4 + 16) + case["rot"] // 2 * 8
        data += (turned if case["per_head"] else 2) * case["hd"] * 2
        return {"bytes": data,
                "flops": case["tokens"] * turned * (case["hd"] * 4 + case["rot"] * 3)}
    if case["op"] == "pack":
        # rows read, packed, and read back
        each = case["tokens"] * 2 * case["nkv"]
        packed = case["hd"] // 2 + case["hd"] // GROUP * 2
        return {"bytes": each * (2 * case["hd"] * 2 + 2 * packed) + case["tokens"] * 16,
                "flops": each * case["hd"] * 5}
    if case["op"] == "attend":
        tokens, pairs, rows = _seen(case)
        data = tokens * case["nkv"] * _tile_bytes(case["hd"]) / 16
        data += rows * case["nq"] * (case["hd"] * 4 + 4) + tokens / case["bs"] * 4
        return {"bytes": int(data), "flops": int(4 * pairs * case["nq"] * case["hd"])}
    page = case["bs"] * case["nkv"] * case["hd"] * 2 * 2 * case["layers"]
    entries = int(_spread(case["blocks_lo"], case["blocks_hi"], case["seqs"]).sum())
    if case["op"] == "fork":
        # about as many last pages are copied as sequences have a sibling
        new, seqs = case["new"], case["seqs"]
        apart = max(0, int(new - seqs * (1.0 - (1.0 - 1.0 / seqs) ** new)))
        return {"bytes": int(apart * page * 2 + entries * (4 + 8) + new * 24), "flops": entries}
    used = entries - entries // 8
    pages = int(entries / case["share"]) + 3
    moves = min(int(used * (1.0 - used / pages)), case["moves"])
    return {"bytes": int(moves * page * 2 + entries * 8 + pages * 8), "flops": entries}


def _exact_norm(case, seed):
    s = prepare(case, seed)
    nq, nkv, hd, rot, n = (case[k] for k in ("nq", "nkv", "hd", "rot", "tokens"))
    half, bs = rot // 2, case["bs"]
    turns = [t % (1 << 64) for t in s["turns"].tolist()]
    positions = torch.tensor(s["positions"].tolist(), dtype=torch.int64)
    # fractions of a turn from whole numbers, 32 bits at a time, so that nothing is rounded
    low = torch.tensor([t & 0xFFFFFFFF for t in turns])
    high = torch.tensor([t >> 32 for t in turns])
    frac = ((positions[:, None] * high) % (1 << 32)).double() / 2.0 ** 32 \
        + (positions[:, None] * low).double() / 2.0 ** 64
    angle = (2 * math.pi * (frac % 1.0)).cuda()
    c, d = angle.cos()[:, None], angle.sin()[:, None]
    rows = s["qkv"].double().view(n, nq + 2 * nkv, hd)
    y = rows.clone()
    add = 1.0 if case["plus_one"] else 0.0
    for lo, hi, w in ((0, nq, s["q_weight"]), (nq, nq + nkv, s["k_weight"])):
        part = rows[:, lo:hi]
        length = (part.pow(2).sum(-1, keepdim=True) / hd + EPS).sqrt()
        y[:, lo:hi] = part / length * (w.double() + add)
    first = torch.arange(half, device="cuda") * (1 if case["layout"] == "half" else 2)
    second = first + (half if case["layout"] == "half" else 1)
    u, w = y[:, :nq + nkv, first], y[:, :nq + nkv, second]
    y[:, :nq + nkv, first], y[:, :nq + nkv, second] = u * c - w * d, u * d + w * c
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    kc[s["slots"] // bs, s["slots"] % bs] = y[:, nq:nq + nkv]
    vc[s["slots"] // bs, s["slots"] % bs] = rows[:, nq + nkv:]
    return {"q": y[:, :nq].contiguous(), "k_cache": kc, "v_cache": vc}


def _exact_pack(case, seed):
    s = prepare(case, seed)
    got = []
    for i in range(2):
        x = s["rows"][:, i].double()
        groups = x.unflatten(-1, (-1, GROUP))
        # the scale is part of the format: a seventh of the largest, rounded to 32 bits and to bf16
        scale = (groups.abs().max(-1).values / 7.0).float().bfloat16().double()[..., None]
        steps = torch.where(scale == 0, torch.zeros_like(groups), groups / scale)
        got.append((steps.round().clamp(-7, 7) * scale).flatten(-2))
    return {"k": got[0], "v": got[1]}


def _exact_head(s, pages, h, count, hd, bs):
    """K and V of the first `count` tokens of a table, head h, element by element."""
    t = torch.arange(count, device="cuda")[:, None]
    d = torch.arange(hd, device="cuda")[None]
    size = _tile_bytes(hd)
    flat = s["cache"].view(-1)
    nkv = s["cache"].shape[1]
    start = ((pages[t // bs] * nkv + h) * (bs // 16) + t % bs // 16) * size
    r = t % 16
    at = start + r * (hd // 2) + (d % 32 // 8) * (hd // 8) + d // 32 * 4 + d % 8 // 2
    k = (flat[at].long() >> (4 * (d % 2))) & 15
    lane = 4 * (d % 8) + r % 8 // 2
    at = start + 8 * hd + (d // 64 * 32 + lane) * 16 + d // 16 % 4 * 4 + r % 2 * 2 + r // 8
    v = (flat[at].long() >> (4 * (d // 8 % 2))) & 15
    words = flat.view(torch.bfloat16)
    at = (start + 16 * hd) // 2 + r * (hd // 32) + d // 32
    return ((k - 8).double() * words[at].double(),
            (v - 8).double() * words[at + 16 * (hd // 32)].double())


def _exact_attend(case, seed):
    tokens, pairs, _ = _seen(case)
    if pairs * case["nq"] * case["hd"] > 1 << 41:
        return None
    s = prepare(case, seed)
    nq, nkv, hd, bs = case["nq"], case["nkv"], case["hd"], case["bs"]
    g, window, sinks = nq // nkv, case["window"] or 1 << 30, case["sinks"]
    out = torch.zeros(s["total_q"], nq, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((s["total_q"], nq), NEG, dtype=torch.float64, device="cuda")
    for b in range(case["seqs"]):
        e0, e1 = s["seq_offsets"][b].item(), s["seq_offsets"][b + 1].item()
        r0, r1 = s["q_offsets"][b].item(), s["q_offsets"][b + 1].item()
        c, t = s["ctx_len"][b].item(), r1 - r0
        own_at = torch.arange(c, c + t, device="cuda")[:, None]
        at = torch.arange(c + t, device="cuda")[None]
        hidden = (at > own_at) | ((at >= sinks) & (at <= own_at - window))
        for h in range(nkv):
            k, v = _exact_head(s, s["table"][e0:e1].long(), h, c + t, hd, bs)
            for first in range(h * g, h * g + g):  # one head at a time bounds the memory
                z = s["q"][r0:r1, first].double() @ k.T * s["scale"]
                z[hidden] = NEG
                ln = torch.logsumexp(z, 1)
                out[r0:r1, first] = (z - ln[:, None]).exp() @ v
                lse[r0:r1, first] = ln
    return {"out": out, "lse": lse}


def exact(case, seed):
    # (pages are counted and copied: nothing there is a computed number)
    if case["op"] in ("fork", "compact"):
        return None
    return {"norm": _exact_norm, "pack": _exact_pack, "attend": _exact_attend}[case["op"]](
        dict(case), seed)
