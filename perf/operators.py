"""Workloads of the paged-cache operators: rotary cache writes, tree attention, eviction.

Each case is one call of one operator at a size that a serving loop meets.  ``run`` computes
it either through the library (``own`` true) or in elementary torch operations in 32 bits.
"""
from __future__ import annotations

import math

import torch

own = False

NEG = float("-inf")


# ------------------------------------------------------------------------------------ cases

def _rope(name, tokens, nq, nkv, hd, rot, layout, scaling, far, bs):
    return {"name": name, "op": "rope", "tokens": tokens, "nq": nq, "nkv": nkv, "hd": hd,
            "rot": rot, "layout": layout, "scaling": scaling, "far": far, "bs": bs}


def _attend(name, seqs, lo, hi, nodes_lo, nodes_hi, mask, nq, nkv, hd, bs, weights):
    return {"name": name, "op": "attend", "seqs": seqs, "ctx_lo": lo, "ctx_hi": hi,
            "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "mask": mask, "nq": nq, "nkv": nkv,
            "hd": hd, "bs": bs, "weights": weights}


def _evict(name, seqs, lo, hi, bs, share):
    return {"name": name, "op": "evict", "seqs": seqs, "blocks_lo": lo, "blocks_hi": hi,
            "bs": bs, "share": share}


def listed():
    return [
        # One new token of one sequence: a decode step's write, where only latency counts.
        _rope("rope_decode_1", 1, 32, 8, 128, 128, "half", "plain", 32768, 16),
        # One token for each of 64 sequences at long positions, a quarter of the head rotated.
        _rope("rope_batch_64", 64, 32, 8, 128, 32, "interleaved", "ramp", 131072, 16),
        # A ragged prompt piece: an odd number of tokens, three query heads a kv head, wide heads.
        _rope("rope_odd_333", 333, 9, 3, 192, 64, "half", "linear", 16384, 48),
        # A whole prefill chunk.
        _rope("rope_prefill_8192", 8192, 64, 8, 128, 128, "interleaved", "base", 131072, 16),
        # Single-token decode of one long sequence; its blocks' weights feed the eviction.
        _attend("decode_1x32768", 1, 32768, 32768, 1, 1, "chain", 32, 8, 128, 16, True),
        # Batched decode at mixed lengths.
        _attend("decode_64_ragged", 64, 1024, 16384, 1, 1, "chain", 32, 8, 128, 16, True),
        # Short, odd and empty contexts, small trees, three query heads a kv head.
        _attend("tree_short_odd", 5, 0, 300, 1, 7, "tree", 9, 3, 64, 32, True),
        # Drafted trees of tens of nodes, verified in one pass.
        _attend("tree_8x61", 8, 4096, 32768, 61, 61, "tree", 64, 8, 128, 16, False),
        # A chunk of 512 rows (a chain of nodes) over a long context.
        _attend("chunk_512x131072", 1, 131072, 131072, 512, 512, "chain", 64, 8, 128, 16, False),
        # One sequence's cache cut to its budget.
        _evict("evict_1x2048", 1, 2048, 2048, 16, 0.9),
        # A batch of short and ordinary sequences, some below their budget.
        _evict("evict_64_ragged", 64, 64, 1024, 16, 0.8),
        # Very long sequences.
        _evict("evict_8x65536", 8, 65536, 65536, 16, 0.5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "evict"])
    bs = rng.choice([16, 16, 32, 48, 64, 128])
    g, nkv = rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), rng.choice([1, 2, 3, 4, 8])
    hd = rng.choice([64, 128, 128, 192, 256])
    if op == "rope":
        tokens = _log_int(rng, 1, 8192)
        rot = 2 * rng.randint(1, hd // 2) if rng.random() < 0.5 else hd
        c = _rope("", tokens, g * nkv, nkv, hd, rot, rng.choice(["half", "interleaved"]),
                  rng.choice(["plain", "linear", "base", "ramp"]), _log_int(rng, 128, 1 << 20), bs)
        if tokens * (g + 2) * nkv * hd > 8192 * 80 * 128:
            c["tokens"] = 8192 * 80 * 128 // ((g + 2) * nkv * hd)
    elif op == "attend":
        seqs, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 131072)
        nodes = 1 if rng.random() < 0.4 else _log_int(rng, 2, 256)
        # no more work than the largest listed cases: rows times tokens, and bytes of cache
        while (seqs * nodes * g * nkv * (hi + nodes) * hd > (1 << 36)
               or seqs * nkv * (hi + nodes) * hd > 64 * 8 * 16384 * 128):
            seqs, hi = max(1, seqs // 2), max(1, hi // 2)
        lo = rng.choice([0, hi // 2, hi])
        c = _attend("", seqs, lo, hi, max(1, nodes // rng.choice([1, 1, 3])), nodes,
                    rng.choice(["tree", "chain"]), g * nkv, nkv, hd, bs, rng.random() < 0.5)
    else:
        seqs, hi = _log_int(rng, 1, 64), _log_int(rng, 8, 65536)
        hi = max(8, min(hi, (8 * 65536) // seqs))
        c = _evict("", seqs, rng.choice([1, hi // 2, hi]), hi, bs, rng.choice([0.3, 0.7, 0.95]))
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


def _rope_frequencies(case):
    """Radians a position, in double: base 10000, the context stretched by four where scaled."""
    rot, base, factor, original = case["rot"], 10000.0, 4.0, 8192.0
    i = torch.arange(rot // 2, dtype=torch.float64)
    if case["scaling"] == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "ramp":
        keep = ((original * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f / factor * (1.0 - keep) + f * keep
    return f


def _prepare_rope(case, host, dev):
    n, nq, nkv, hd, bs = (case[k] for k in ("tokens", "nq", "nkv", "hd", "bs"))
    # turns: the frequencies as 64-bit fixed-point fractions of a turn, the library's table
    turns = [int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in _rope_frequencies(case).tolist()]
    turns = torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns])
    # the rows of a fused projection: queries, keys and values side by side
    qkv = _bf16(dev, n, (nq + 2 * nkv) * hd)
    blocks = (n + bs - 1) // bs + 2
    slots = torch.randperm(blocks * bs, generator=host)[:n]
    return {"case": case, "qkv": qkv, "positions": _ints(host, 0, case["far"], n).cuda(),
            "slots": slots.cuda(), "turns": turns.cuda(),
            "kept": {}, "magnitude": 0.1 * math.log(4.0) + 1.0 if case["scaling"] == "ramp" else 1.0,
            "q_out": torch.empty(n, nq, hd, device="cuda", dtype=torch.bfloat16),
            "k_cache": _bf16(dev, blocks, bs, nkv, hd), "v_cache": _bf16(dev, blocks, bs, nkv, hd)}


def _tree_words(host, counts, words):
    """Visibility words of random trees: node j's parent is a random earlier node or the root."""
    total = int(counts.sum())
    rows = []
    for n in counts.tolist():
        see = torch.zeros(n, 64 * words, dtype=torch.bool)
        parent = (torch.rand(n, generator=host) * torch.arange(n)).long().tolist()
        for j in range(n):
            if j > 0 and j % 4 != 3:
                see[j] = see[parent[j]]
            see[j, j] = True
        rows.append(see)
    bits = torch.cat(rows).view(total, words, 64).long()
    return (bits << torch.arange(64)).sum(-1)


def _prepare_attend(case, host, dev):
    nq, nkv, hd, bs, seqs = (case[k] for k in ("nq", "nkv", "hd", "bs", "seqs"))
    # lengths and tree sizes are paired the same way for every seed; their order is not
    order = torch.randperm(seqs, generator=host)
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], seqs)[order]
    nodes = _spread(case["nodes_lo"], case["nodes_hi"], seqs, seqs // 3)[order]
    blocks = (ctx + nodes + bs - 1) // bs
    total_blocks, total_q, max_q = int(blocks.sum()), int(nodes.sum()), int(nodes.max())
    max_blocks = total_blocks + total_blocks // 8 + 1
    table = torch.randperm(max_blocks, generator=host)[:total_blocks].int()
    state = {"case": case, "ctx_len": ctx.int().cuda(), "q_offsets": _offsets(nodes).int().cuda(),
             "seq_offsets": _offsets(blocks).int().cuda(), "table": table.cuda(),
             "total_q": total_q, "max_q": max_q, "total_blocks": total_blocks,
             "max_table": int(blocks.max()), "max_blocks": max_blocks,
             "q": _bf16(dev, total_q, nq, hd, std=2.0),
             "k_cache": _bf16(dev, max_blocks, bs, nkv, hd),
             "v_cache": _bf16(dev, max_blocks, bs, nkv, hd),
             "words": (max_q + 63) // 64, "mask": None, "weights_in": None, "decay": 0.97,
             "scale": 1.0 / math.sqrt(hd), "kept": {}}
    if case["mask"] == "tree":
        state["mask"] = _tree_words(host, nodes, state["words"]).cuda()
    if case["weights"]:
        # what some thirty steps leave, each sharing out nq of attention a row over the blocks
        each = 30.0 * nq * total_q / total_blocks
        state["weights_in"] = torch.rand(total_blocks, generator=dev, device="cuda") * each
    return state


def _prepare_evict(case, host, dev):
    order = torch.randperm(case["seqs"], generator=host)
    n = _spread(case["blocks_lo"], case["blocks_hi"], case["seqs"])[order]
    total = int(n.sum())
    # log-normal weights, as sums of attention are, with the ties of blocks never looked at
    w = torch.empty(total, device="cuda").log_normal_(0.0, 2.0, generator=dev)
    w = w * (torch.rand(total, generator=dev, device="cuda") > 0.05)
    filled = n * case["bs"] - _ints(host, 0, case["bs"] - 1, case["seqs"])
    budget = (n.double() * case["share"]).long().clamp(min=1)
    budget[::3] = int(case["blocks_hi"] * case["share"])
    return {"case": case, "weights": w, "total": total,
            "table": torch.randperm(total + 7, generator=host)[:total].int().cuda(),
            "seq_offsets": _offsets(n).int().cuda(), "ctx_len": filled.int().cuda(),
            "budgets": budget.int().cuda(), "keep_first": 1, "keep_last": 2}


def prepare(case, seed):
    host, dev = _gens(seed)
    return {"rope": _prepare_rope, "attend": _prepare_attend,
            "evict": _prepare_evict}[case["op"]](dict(case), host, dev)


# ------------------------------------------------------------------------- the library's calls

def _dims(case, max_blocks):
    import kv_cache_block_lowrank_gb300 as hss

    return hss.hss_dims(1, case["nq"], case["nkv"], case["hd"], 16, case["bs"], max_blocks)


def _own_rope(s):
    import kv_cache_block_lowrank_gb300 as hss

    case = s["case"]
    nq, nkv, hd, n = case["nq"], case["nkv"], case["hd"], case["tokens"]
    kept = s["kept"]
    if "call" not in kept:  # the layers of a step share positions, slots and table: bound once
        layout = hss.HSS_ROPE_HALF if case["layout"] == "half" else hss.HSS_ROPE_INTERLEAVED
        stride = (nq + 2 * nkv) * hd
        kept["call"] = hss.RopeTokens(_dims(case, s["k_cache"].shape[0]), case["rot"], layout,
                                      s["turns"], s["magnitude"], s["positions"], s["slots"], n,
                                      stride, stride, stride)
    qkv = s["qkv"]
    at = qkv.data_ptr()
    kept["call"](at, at + 2 * nq * hd, at + 2 * (nq + nkv) * hd, s["q_out"], None, s["k_cache"],
              s["v_cache"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    import kv_cache_block_lowrank_gb300 as hss

    case = s["case"]
    kept = s["kept"]
    if "call" not in kept:  # the layers of a step share tables, lengths, masks and workspace
        dims = _dims(case, s["max_blocks"])
        size = hss.hss_attend_tree_workspace_bytes(dims, case["seqs"], s["max_q"],
                                                   s["total_blocks"], case["weights"])
        work = torch.zeros(size, dtype=torch.uint8, device="cuda")
        kept["call"] = hss.AttendTree(dims, s["q_offsets"], s["total_q"], s["max_q"], s["mask"],
                                      s["words"] if s["mask"] is not None else 0, s["table"],
                                      s["seq_offsets"], s["ctx_len"], case["seqs"],
                                      s["total_blocks"], s["scale"], s["decay"], work, size)
    out = torch.empty_like(s["q"])
    lse = torch.empty(s["total_q"], case["nq"], device="cuda")
    weights = torch.empty(s["total_blocks"], device="cuda") if case["weights"] else None
    kept["call"](s["q"], s["k_cache"], s["v_cache"], out, lse, s["weights_in"], weights)
    return {"out": out, "lse": lse} | ({"weights": weights} if case["weights"] else {})


def _own_evict(s):
    import kv_cache_block_lowrank_gb300 as hss

    seqs, total = s["case"]["seqs"], s["total"]
    table, freed = torch.empty_like(s["table"]), torch.empty_like(s["table"])
    weights, ctx = torch.empty_like(s["weights"]), torch.empty_like(s["ctx_len"])
    offs, freed_offs = torch.empty_like(s["seq_offsets"]), torch.empty_like(s["seq_offsets"])
    hss.hss_evict_blocks(s["weights"], s["table"], s["seq_offsets"], s["ctx_len"], s["budgets"],
                         seqs, total, s["case"]["bs"], s["keep_first"], s["keep_last"], table,
                         offs, weights, ctx, freed, freed_offs)
    return {"table": table, "seq_offsets": offs, "weights": weights, "ctx_len": ctx,
            "freed": freed, "freed_offsets": freed_offs}


# ----------------------------------------------------------------------------- the plain forms

def _plain_rope(s):
    case = s["case"]
    nq, nkv, hd, rot, n = (case[k] for k in ("nq", "nkv", "hd", "rot", "tokens"))
    # 64-bit products wrap: what is left is the fraction of a turn, signed, in 2^-64
    part = s["positions"][:, None] * s["turns"][None, :]
    angle = (part >> 32).float() * (2.0 * math.pi / 2.0 ** 32)
    cos, sin = angle.cos()[:, None] * s["magnitude"], angle.sin()[:, None] * s["magnitude"]
    x = s["qkv"].view(n, nq + 2 * nkv, hd)
    qk = x[:, :nq + nkv].float()
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


def _plain_attend(s):
    case = s["case"]
    nq, nkv, hd, bs, seqs = (case[k] for k in ("nq", "nkv", "hd", "bs", "seqs"))
    g, most, nodes_max = nq // nkv, s["max_table"], s["max_q"]
    length = most * bs
    offs, q0 = s["seq_offsets"].long(), s["q_offsets"].long()
    nodes, ctx = q0[1:] - q0[:-1], s["ctx_len"].long()
    # every sequence padded to the longest
    entry = (offs[:-1, None] + torch.arange(most, device="cuda")).clamp(max=s["total_blocks"] - 1)
    ids = s["table"].long()[entry]
    row = (q0[:-1, None] + torch.arange(nodes_max, device="cuda")).clamp(max=s["total_q"] - 1)
    q = s["q"][row].float().view(seqs, nodes_max, nkv, g, hd).permute(0, 2, 1, 3, 4)
    k = s["k_cache"][ids].view(seqs, length, nkv, hd).permute(0, 2, 3, 1).float()
    score = (q.reshape(seqs, nkv, nodes_max * g, hd) @ k).mul_(s["scale"])
    del k
    i = torch.arange(nodes_max, device="cuda")
    j = torch.arange(length, device="cuda")[None] - ctx[:, None]          # node index of a token
    if s["mask"] is None:
        see = j[:, None, :] <= i[None, :, None]
    else:
        at = j.clamp(0, 64 * s["words"] - 1)
        words = s["mask"].view(-1, s["words"])[row]                       # [seqs, nodes, words]
        word = words.gather(2, (at // 64)[:, None, :].expand(-1, nodes_max, -1))
        see = (((word >> (at % 64)[:, None, :]) & 1) > 0) | (j < 0)[:, None, :]
    see = see & (j < nodes[:, None])[:, None, :] & (i < nodes[:, None])[:, :, None]
    score = score.view(seqs, nkv, nodes_max, g, length).masked_fill_(~see[:, None, :, None], NEG)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    v = s["v_cache"][ids].view(seqs, length, nkv, hd).permute(0, 2, 1, 3).float()
    out = (p.view(seqs, nkv, nodes_max * g, length) @ v).view(seqs, nkv, nodes_max, g, hd)
    lse = (top + total.log()).view(seqs, nkv, nodes_max, g)
    # back to the rows as they are packed
    seq_of = torch.repeat_interleave(torch.arange(seqs, device="cuda"), nodes,
                                     output_size=s["total_q"])
    node_of = torch.arange(s["total_q"], device="cuda") - q0[seq_of]
    out = out.permute(0, 2, 1, 3, 4)[seq_of, node_of].reshape(s["total_q"], nq, hd).bfloat16()
    lse = lse.permute(0, 2, 1, 3)[seq_of, node_of].reshape(s["total_q"], nq)
    got = {"out": out, "lse": lse}
    if case["weights"]:
        mass = p.sum((1, 2, 3)).view(seqs, most, bs).sum(-1)
        owner = torch.repeat_interleave(torch.arange(seqs, device="cuda"), offs[1:] - offs[:-1],
                                        output_size=s["total_blocks"])
        place = torch.arange(s["total_blocks"], device="cuda") - offs[owner]
        got["weights"] = s["decay"] * s["weights_in"] + mass[owner, place]
    return got


def _plain_evict(s):
    seqs, total, dev = s["case"]["seqs"], s["total"], "cuda"
    offs, ctx = s["seq_offsets"].long(), s["ctx_len"].long()
    n = offs[1:] - offs[:-1]
    last = torch.minimum(n - s["keep_last"], ctx // s["case"]["bs"])
    candidates = (last - s["keep_first"]).clamp(min=0)
    evict = torch.minimum((n - s["budgets"]).clamp(min=0), candidates)
    owner = torch.repeat_interleave(torch.arange(seqs, device=dev), n, output_size=total)
    j = torch.arange(total, device=dev) - offs[owner]
    candidate = (j >= s["keep_first"]) & (j < last[owner])
    w = s["weights"] + 0.0
    w = torch.where(w.isnan(), torch.full_like(w, math.inf), w)
    by_weight = w.argsort(stable=True)
    order = by_weight[(owner * 2 + ~candidate)[by_weight].argsort(stable=True)]
    rank = torch.empty(total, dtype=torch.int64, device=dev)
    rank[order] = torch.arange(total, device=dev) - offs[owner[order]]
    gone = candidate & (rank < evict[owner])
    spare = torch.full((1,), total, device=dev)

    def packed(source, taken, fill):
        to = torch.where(taken, taken.cumsum(0) - 1, spare)
        whole = torch.full((total + 1,), fill, dtype=source.dtype, device=dev)
        whole[to] = source
        return whole[:total]

    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    return {"table": packed(s["table"], ~gone, -1), "weights": packed(s["weights"], ~gone, 0.0),
            "seq_offsets": torch.cat([zero, (n - evict).cumsum(0)]).int(),
            "ctx_len": (ctx - evict * s["case"]["bs"]).int(), "freed": packed(s["table"], gone, -1),
            "freed_offsets": torch.cat([zero, evict.cumsum(0)]).int()}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "attend": _own_attend, "evict": _own_evict}[op](state)
    return {"rope": _plain_rope, "attend": _plain_attend, "evict": _plain_evict}[op](state)


# ------------------------------------------------------------------------------- work, 64 bits

def work(case):
    if case["op"] == "rope":
        heads = case["nq"] + 2 * case["nkv"]
        # every row read and written, and a position, a slot and (once) the frequencies
        data = case["tokens"] * (heads * case["hd"] * 4 + 16) + case["rot"] // 2 * 8
        return {"bytes": data, "flops": case["tokens"] * (case["nq"] + case["nkv"]) * case["rot"] * 3}
    if case["op"] == "attend":
        ctx = case["seqs"] * (case["ctx_lo"] + case["ctx_hi"]) / 2
        rows = case["seqs"] * (case["nodes_lo"] + case["nodes_hi"]) / 2
        tokens = ctx + rows
        data = tokens * case["nkv"] * case["hd"] * 4 + rows * case["nq"] * (case["hd"] * 4 + 4)
        data += tokens / case["bs"] * (4 + (8 if case["weights"] else 0))
        seen = (rows / case["seqs"]) * (tokens / case["seqs"]) * case["seqs"]
        return {"bytes": int(data), "flops": int(4 * seen * case["nq"] * case["hd"])}
    entries = case["seqs"] * (case["blocks_lo"] + case["blocks_hi"]) / 2
    return {"bytes": int(entries * 20 + case["seqs"] * 20), "flops": int(entries * 2)}


def _exact_rope(case, seed):
    s = prepare(case, seed)
    nq, nkv, hd, rot, n = (case[k] for k in ("nq", "nkv", "hd", "rot", "tokens"))
    half = rot // 2
    turns = [t % (1 << 64) for t in s["turns"].tolist()]
    positions = torch.tensor(s["positions"].tolist(), dtype=torch.int64)
    # fractions of a turn from whole numbers, 32 bits at a time, so that nothing is rounded
    low = torch.tensor([t & 0xFFFFFFFF for t in turns])
    high = torch.tensor([t >> 32 for t in turns])
    lo_part = positions[:, None] * low
    frac = ((positions[:, None] * high) % (1 << 32)).double() / 2.0 ** 32 + lo_part.double() / 2.0 ** 64
    angle = (2 * math.pi * (frac % 1.0)).cuda()
    c, d = angle.cos() * s["magnitude"], angle.sin() * s["magnitude"]
    rows = s["qkv"].double().view(n, nq + 2 * nkv, hd)
    y = rows.clone()
    first = torch.arange(half, device="cuda") * (1 if case["layout"] == "half" else 2)
    second = first + (half if case["layout"] == "half" else 1)
    u, w = rows[..., first], rows[..., second]
    y[..., first] = u * c[:, None] - w * d[:, None]
    y[..., second] = u * d[:, None] + w * c[:, None]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    bs = case["bs"]
    kc[s["slots"] // bs, s["slots"] % bs] = y[:, nq:nq + nkv]
    vc[s["slots"] // bs, s["slots"] % bs] = rows[:, nq + nkv:]
    return {"q": y[:, :nq].contiguous(), "k_cache": kc, "v_cache": vc}


def _exact_attend(case, seed):
    s = prepare(case, seed)
    nq, nkv, hd, bs = case["nq"], case["nkv"], case["hd"], case["bs"]
    g = nq // nkv
    out = torch.zeros(s["total_q"], nq, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((s["total_q"], nq), NEG, dtype=torch.float64, device="cuda")
    weights = s["weights_in"].double() * s["decay"] if case["weights"] else None
    for b in range(case["seqs"]):
        e0, e1 = s["seq_offsets"][b].item(), s["seq_offsets"][b + 1].item()
        r0, r1 = s["q_offsets"][b].item(), s["q_offsets"][b + 1].item()
        c, t = s["ctx_len"][b].item(), r1 - r0
        see = torch.ones(t, c + t, dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            see[:, c:] = torch.ones(t, t, device="cuda").tril().bool()
        else:
            node = torch.arange(t, device="cuda")
            see[:, c:] = (s["mask"].view(-1, s["words"])[r0:r1][:, node // 64] >> (node % 64)) & 1 == 1
        for h in range(nkv):
            k = s["k_cache"][s["table"][e0:e1].long(), :, h].reshape(-1, hd)[:c + t].double()
            v = s["v_cache"][s["table"][e0:e1].long(), :, h].reshape(-1, hd)[:c + t].double()
            for first in range(0, g):  # one head at a time bounds the memory
                z = s["q"][r0:r1, h * g + first].double() @ k.T * s["scale"]
                z = torch.where(see, z, torch.full((), NEG, dtype=torch.float64, device="cuda"))
                some = see.any(1)
                ln = torch.logsumexp(z, 1)
                w = torch.where(some[:, None], (z - ln[:, None]).exp(), torch.zeros_like(z))
                out[r0:r1, h * g + first] = w @ v
                lse[r0:r1, h * g + first] = ln
                if weights is not None:
                    m = torch.zeros((e1 - e0) * bs, dtype=torch.float64, device="cuda")
                    m[:c + t] = w.sum(0)
                    weights[e0:e1] += m.view(-1, bs).sum(1)
    return {"out": out, "lse": lse} | ({"weights": weights} if case["weights"] else {})


def _exact_evict(case, seed):
    import numpy as np

    s = prepare(case, seed)
    w, table = s["weights"].cpu().numpy(), s["table"].cpu().numpy()
    offs, ctx, budget = (s[k].cpu().numpy().astype(np.int64)
                         for k in ("seq_offsets", "ctx_len", "budgets"))
    left = np.zeros(len(w))
    count = 0
    for b in range(case["seqs"]):
        n = int(offs[b + 1] - offs[b])
        lo, hi = s["keep_first"], min(n - s["keep_last"], int(ctx[b]) // case["bs"])
        part = w[offs[b]:offs[b + 1]].astype(np.float64)
        inside = np.arange(lo, max(lo, hi))
        gone = inside[np.argsort(part[inside], kind="stable")][:max(0, n - int(budget[b]))]
        stay = np.delete(part, gone)
        left[count:count + len(stay)] = stay
        count += len(stay)
    # the whole-number outputs have no counterpart in 64 bits: they are compared as they are
    return {"table": None, "weights": torch.from_numpy(left), "seq_offsets": None, "ctx_len": None,
            "freed": None, "freed_offsets": None}


def exact(case, seed):
    return {"rope": _exact_rope, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](
        dict(case), seed)
