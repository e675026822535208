"""The operators of a decode loop over a paged key-value cache, as cases to be timed: appending
rotated keys and values, the attention of one new token per sequence, beam search's selection,
and the reordering of the sequences' states that follows it.

``run`` computes a case in its plain form (elementary torch operations) or, with ``own`` set,
through the library.  ``exact`` computes the same outputs in 64 bits, written apart.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one request's decode step: a single token, rotated and stored
        {"name": "append_1_token_d128", "op": "append", "seqs": 1, "new": 1, "past": 1000,
         "kv_heads": 4, "group": 4, "d": 128, "page": 16, "rot": 128, "interleaved": False},
        # a serving batch's decode step, neighbours rotated, part of the head only, odd pages
        {"name": "append_256x1_d64_page20", "op": "append", "seqs": 256, "new": 1, "past": 700,
         "kv_heads": 8, "group": 2, "d": 64, "page": 20, "rot": 32, "interleaved": True},
        # prompts of several requests at once, ragged, behind cached prefixes
        {"name": "append_9_prompts_d128", "op": "append", "seqs": 9, "new": 4001, "past": 333,
         "kv_heads": 4, "group": 4, "d": 128, "page": 64, "rot": 128, "interleaved": False},
        # one request with a short context, where launches and latency count
        {"name": "attention_1x1000_16q2_d128", "op": "attention", "seqs": 1, "len": 1000,
         "spread": 1, "idle": 0, "kv_heads": 2, "group": 8, "d": 128, "page": 16},
        # one request with a long context: the length has to be split
        {"name": "attention_1x131072_16q2_d128", "op": "attention", "seqs": 1, "len": 131072,
         "spread": 1, "idle": 0, "kv_heads": 2, "group": 8, "d": 128, "page": 64},
        # a serving batch whose lengths differ 32-fold, some of its places idle, odd pages
        {"name": "attention_61x8191_ragged_16q4_d128", "op": "attention", "seqs": 61, "len": 8191,
         "spread": 32, "idle": 3, "kv_heads": 4, "group": 4, "d": 128, "page": 20},
        # small heads, one query head for each key head
        {"name": "attention_128x2000_16q16_d64", "op": "attention", "seqs": 128, "len": 2000,
         "spread": 4, "idle": 0, "kv_heads": 16, "group": 1, "d": 64, "page": 16},
        # the benchmark's 16 heads and 4096 tokens for 64 sequences, the largest amount of work
        {"name": "attention_64x4096_16q16_d128", "op": "attention", "seqs": 64, "len": 4096,
         "spread": 1, "idle": 0, "kv_heads": 16, "group": 1, "d": 128, "page": 128},
        # one request searched with four beams
        {"name": "select_1x4x50257_f32", "op": "select", "groups": 1, "beams": 4, "cols": 50257,
         "K": 4, "dtype": "f32", "ended": 0},
        # a serving batch of eight beams that asks for twice as many candidates, some beams ended
        {"name": "select_32x8x128256_bf16_K16", "op": "select", "groups": 32, "beams": 8,
         "cols": 128256, "K": 16, "dtype": "bf16", "ended": 1},
        # states of one request's beams, one layer at a time
        {"name": "reorder_1x4_1_layer", "op": "reorder", "groups": 1, "beams": 4, "layers": 1,
         "len": 1003, "kv_heads": 4, "d": 128, "page": 16},
        # states of a batch of beams over all of a model's layers
        {"name": "reorder_32x8_16_layers", "op": "reorder", "groups": 32, "beams": 8,
         "layers": 16, "len": 500, "kv_heads": 4, "d": 128, "page": 64},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_PAGES = [1, 8, 16, 16, 20, 32, 64, 100, 128, 256]


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "select", "reorder"])
    d = rng.choice([64, 128])
    if op == "append":
        kv_heads, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 1, 2, 4, 6, 8])
        new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 8000)
        most = max(1, 9 * 4001 * 24 * 128 // (new * kv_heads * (group + 2) * d))
        return {"op": op, "seqs": min(_log_int(rng, 1, 512), most), "new": new,
                "past": rng.choice([0, _log_int(rng, 1, 3000)]), "kv_heads": kv_heads,
                "group": group, "d": d, "page": rng.choice(_PAGES),
                "rot": rng.choice([0, 32, d, d]), "interleaved": rng.random() < 0.4}
    if op == "attention":
        kv_heads = rng.choice([1, 2, 4, 5, 8, 16])
        group = rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16])
        length = _log_int(rng, 1, 131072)
        most = max(1, 64 * 4096 * 16 * 128 // (length * kv_heads * d))
        seqs = min(_log_int(rng, 1, 300), most)
        return {"op": op, "seqs": seqs, "len": length, "spread": rng.choice([1, 1, 4, 32]),
                "idle": rng.choice([0, 0, seqs // 8]), "kv_heads": kv_heads, "group": group,
                "d": d, "page": rng.choice(_PAGES)}
    beams = rng.randint(1, 12)
    if op == "select":
        cols = _log_int(rng, 500, 160000)
        groups = min(_log_int(rng, 1, 64), max(1, 32 * 8 * 128256 // (beams * cols)))
        return {"op": op, "groups": groups, "beams": beams, "cols": cols,
                "K": rng.randint(1, 2 * beams), "dtype": rng.choice(["f32", "bf16"]),
                "ended": rng.choice([0, 0, beams // 3])}
    page, kv_heads = rng.choice(_PAGES), rng.choice([1, 2, 4, 5, 8, 16])
    layers, length = _log_int(rng, 1, 32), _log_int(rng, 1, 1000)
    # pages of one group: shared ones, and two of each beam's own
    per_group = (2 * beams + -(-(length + 12 * 64) // page)) * layers * kv_heads * page * d
    return {"op": op, "groups": max(1, min(_log_int(rng, 1, 64), (1 << 29) // per_group)),
            "beams": beams, "layers": layers, "len": length, "kv_heads": kv_heads, "d": d,
            "page": page}


_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _lengths(case):
    """The sequences' lengths of an attention case, in no order: from len / spread to len, evenly
    over the logarithm, and the idle places with none."""
    n = case["seqs"]
    out = [max(1, round(case["len"] * case["spread"] ** -(i / max(n - 1, 1)))) for i in range(n)]
    for i in range(case["idle"]):
        out[n - 1 - i] = 0
    return out


def _new_tokens(case):
    """The number of new tokens of each sequence of an append case: one each, or about the case's
    number, no two alike."""
    if case["new"] == 1:
        return [1] * case["seqs"]
    return [max(1, case["new"] - 37 * (i % 50)) for i in range(case["seqs"])]


def _group_lengths(case):
    """The length of each group of a reorder case: its beams' part-filled pages differ."""
    return [case["len"] + 11 * g for g in range(case["groups"])]


def _survivors(case):
    return max(1, math.ceil(case["beams"] * 0.6))


def work(case):
    if case["op"] == "append":
        tokens = sum(_new_tokens(case))
        heads = case["kv_heads"] * (case["group"] + 2)
        # queries, keys and values in, rotated queries and the cache's places out
        return {"bytes": 2 * tokens * heads * case["d"] * 2 + case["seqs"] * 8 + case["rot"] * 2,
                "flops": tokens * (heads - case["kv_heads"]) * case["rot"] * 3}
    if case["op"] == "attention":
        keys, heads = sum(_lengths(case)), case["kv_heads"] * case["group"]
        rows = case["seqs"] * heads
        return {"bytes": keys * case["kv_heads"] * case["d"] * 4 + rows * (case["d"] * 4 + 4) +
                4 * (case["seqs"] + keys // case["page"]),
                "flops": 4 * keys * heads * case["d"]}
    if case["op"] == "select":
        # beams that have ended bring their score alone
        cells = case["groups"] * (case["beams"] - case["ended"]) * case["cols"]
        return {"bytes": cells * (4 if case["dtype"] == "f32" else 2) +
                case["groups"] * (case["beams"] * 5 + case["K"] * 12), "flops": 4 * cells}
    row = case["layers"] * case["kv_heads"] * case["d"] * 4
    rest = sum(n % case["page"] for n in _group_lengths(case))
    entries = sum(n // case["page"] for n in _group_lengths(case))
    # the part-filled pages of the beams that live on in, one for every beam out
    return {"bytes": (row * rest + 4 * entries) * (_survivors(case) + case["beams"]) +
            case["groups"] * case["beams"] * 12, "flops": 0}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEVICE)

    def order(n):
        return torch.rand(n, generator=g, device=DEVICE).argsort()

    def table_of(lengths, width, ids):
        """Pages taken from `ids` in turn, as many as each length needs; -1 behind them."""
        need = (lengths + case["page"] - 1) // case["page"]
        first = need.cumsum(0) - need
        at = torch.arange(width, device=DEVICE)[None, :]
        used = at < need[:, None]
        flat = (first[:, None] + at).masked_fill(~used, 0)
        return ids[flat].masked_fill(~used, -1).int().contiguous()

    def ints(values):
        return torch.tensor(values, dtype=torch.int64, device=DEVICE)

    state = {"case": case}
    if case["op"] == "append":
        new = ints(_new_tokens(case))[order(case["seqs"])]
        past = (rand(case["seqs"]) * (case["past"] + 1)).long()
        lengths = past + new
        # what the tables have room for does not depend on the seed
        width = -(-(case["past"] + max(_new_tokens(case))) // case["page"])
        pages = case["seqs"] * width + 3
        shape = (pages, case["kv_heads"], case["page"], case["d"])
        tokens = sum(_new_tokens(case))
        heads = case["kv_heads"] * (case["group"] + 2)
        # one matrix product made queries, keys and values of every token
        qkv = randn(tokens, heads, case["d"], dtype=torch.bfloat16)
        hq, hkv = case["kv_heads"] * case["group"], case["kv_heads"]
        half = case["rot"] // 2
        state.update(
            k_cache=randn(*shape, dtype=torch.bfloat16),
            v_cache=randn(*shape, dtype=torch.bfloat16),
            table=table_of(lengths, width, order(pages)), lengths=lengths.int(),
            q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:],
            starts=None if case["new"] == 1 else
            torch.cat([new.new_zeros(1), new.cumsum(0)]).int(),
            inv_freq=None if half == 0 else
            (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().to(DEVICE))
    elif case["op"] == "attention":
        lengths = ints(_lengths(case))[order(case["seqs"])]
        need = sum(-(-n // case["page"]) for n in _lengths(case))
        width = -(-case["len"] // case["page"])
        shape = (need + 3, case["kv_heads"], case["page"], case["d"])
        state.update(
            k_cache=randn(*shape, dtype=torch.bfloat16),
            v_cache=randn(*shape, dtype=torch.bfloat16),
            table=table_of(lengths, width, order(need + 3)), lengths=lengths.int(),
            # queries that look for some keys more than for others
            q=(2 * randn(case["seqs"], case["kv_heads"] * case["group"], case["d"])).bfloat16())
    elif case["op"] == "select":
        groups, beams, cols = case["groups"], case["beams"], case["cols"]
        x = randn(groups * beams, cols) * 2.5
        x += 4.0 * (rand(groups * beams, 1) * 2 - 1)
        # a few likely tokens stand out, and a grammar forbids some
        at = torch.randint(0, cols, (groups * beams, 6), generator=g, device=DEVICE)
        x.scatter_add_(1, at, 9.0 + 2.0 * randn(groups * beams, 6))
        x = x.to(_DTYPES[case["dtype"]])
        x.masked_fill_(rand(groups * beams, cols) < 0.01, float("-inf"))
        scores = -(20.0 + 3.0 * rand(groups, beams))
        ended = None
        if case["ended"]:
            ended = rand(groups, beams).argsort(1) < case["ended"]
        state.update(x=x, scores=scores, ended=ended)
    else:
        groups, beams, page = case["groups"], case["beams"], case["page"]
        seqs = groups * beams
        per_group = ints(_group_lengths(case))[order(groups)]
        lengths = per_group[:, None].expand(groups, beams).reshape(-1)
        width = -(-(max(_group_lengths(case)) + 1) // page)
        # every beam has a page of its own to fill, before and after; the full ones are shared
        pages = 2 * seqs + groups * width + 3
        ids = order(pages).int()
        shared = ids[2 * seqs:2 * seqs + groups * width].view(groups, 1, width)
        table = shared.expand(groups, beams, width).reshape(seqs, width).clone()
        out_table = torch.full_like(table, -1)
        at = (lengths // page)[:, None]
        table.scatter_(1, at, ids[:seqs, None])
        out_table.scatter_(1, at, ids[seqs:2 * seqs, None])
        shape = (case["layers"], pages, case["kv_heads"], page, case["d"])
        # some beams die, the others live on once or more often
        alive = rand(groups, beams).argsort(1)[:, :_survivors(case)]
        pick = (torch.arange(beams, device=DEVICE) % _survivors(case)).expand(groups, beams)
        pick = pick.gather(1, rand(groups, beams).argsort(1))
        state.update(
            k_cache=randn(*shape, dtype=torch.bfloat16),
            v_cache=randn(*shape, dtype=torch.bfloat16),
            table=table, lengths=lengths.int(), parents=alive.gather(1, pick).int().contiguous(),
            out_table=out_table, out_lengths=torch.zeros_like(lengths).int())
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"append": _plain_append, "attention": _plain_attention, "select": _plain_select,
            "reorder": _plain_reorder}[state["case"]["op"]](state)


def _run_own(state):
    import softmax_topk_gb300 as st
    case = state["case"]
    if case["op"] == "append":
        q = st.paged_append(state["k_cache"], state["v_cache"], state["table"], state["lengths"],
                            state["k"], state["v"], q=state["q"], starts=state["starts"],
                            inv_freq=state["inv_freq"], interleaved=case["interleaved"])
        return state["k_cache"], state["v_cache"], q
    if case["op"] == "attention":
        return st.paged_attention(state["q"], state["k_cache"], state["v_cache"], state["table"],
                                  state["lengths"])
    if case["op"] == "select":
        return st.beam_select(state["x"], state["scores"], case["K"], ended=state["ended"], pad=0)
    table, lengths = st.paged_reorder(state["k_cache"], state["v_cache"], state["table"],
                                      state["lengths"], state["parents"], state["out_table"],
                                      out_lengths=state["out_lengths"])
    return state["k_cache"], state["v_cache"], table, lengths


def _places(state):
    """The page and the slot of every new token, and its position."""
    lengths, starts = state["lengths"].long(), state["starts"]
    tokens = state["k"].shape[0]
    if starts is None:
        seq = torch.arange(tokens, device=DEVICE)
        pos = lengths - 1
    else:
        first = starts.long()
        seq = torch.repeat_interleave(torch.arange(len(lengths), device=DEVICE),
                                      first[1:] - first[:-1], output_size=tokens)
        pos = lengths[seq] - first[seq + 1] + torch.arange(tokens, device=DEVICE)
    page = state["case"]["page"]
    return state["table"].long()[seq, pos // page], pos % page, pos


def _rotate(x, cos, sin, interleaved):
    half = cos.shape[-1]
    out = x.float()
    if interleaved:
        a, b = out[..., 0:2 * half:2].clone(), out[..., 1:2 * half:2].clone()
        out[..., 0:2 * half:2] = a * cos - b * sin
        out[..., 1:2 * half:2] = b * cos + a * sin
    else:
        a, b = out[..., :half].clone(), out[..., half:2 * half].clone()
        out[..., :half] = a * cos - b * sin
        out[..., half:2 * half] = b * cos + a * sin
    return out.bfloat16()


def _plain_append(state):
    page, slot, pos = _places(state)
    q, k = state["q"], state["k"]
    if state["inv_freq"] is not None:
        # angles of far positions need 64 bits
        angle = pos.double()[:, None, None] * state["inv_freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()
        q = _rotate(q, cos, sin, state["case"]["interleaved"])
        k = _rotate(k, cos, sin, state["case"]["interleaved"])
    else:
        q = q.clone(memory_format=torch.contiguous_format)
    state["k_cache"][page, :, slot] = k
    state["v_cache"][page, :, slot] = state["v"]
    return state["k_cache"], state["v_cache"], q


def _plain_attention(state):
    case, q = state["case"], state["q"]
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device=DEVICE)
    lse = torch.full(q.shape[:2], float("-inf"), device=DEVICE)
    kv, group, d, width = case["kv_heads"], case["group"], case["d"], state["table"].shape[1]
    scale = 1.0 / math.sqrt(d)
    # as many sequences at once as a gigabyte of keys in 32 bits allows
    step = max(1, (1 << 28) // (width * case["page"] * kv * d))
    for b in range(0, case["seqs"], step):
        lengths, table = state["lengths"][b:b + step].long(), state["table"][b:b + step].long()
        n = len(lengths)
        at = torch.arange(width * case["page"], device=DEVICE)
        hidden = (at >= lengths[:, None])[:, None, None, :]

        def rows(cache):
            got = cache[table.clamp(min=0)].transpose(1, 2)  # [n, heads, width, page, d]
            return got.reshape(n, kv, width * case["page"], d).float()

        s = q[b:b + step].float().view(n, kv, group, d) @ rows(state["k_cache"]).transpose(-1, -2)
        s = (s * scale).masked_fill(hidden, float("-inf"))
        m = s.amax(-1, keepdim=True).clamp(min=-3e38)
        e = (s - m).exp()
        total = e.sum(-1, keepdim=True)
        v = rows(state["v_cache"]).masked_fill(hidden.view(n, 1, -1, 1), 0.0)
        o = e @ v / total.clamp(min=1e-30)
        out[b:b + step] = o.view(n, kv * group, d).bfloat16()
        lse[b:b + step] = (m + total.log()).view(n, kv * group)
    return out, lse


def _plain_select(state):
    case, x = state["case"], state["x"]
    groups, beams, cols, K = case["groups"], case["beams"], case["cols"], case["K"]
    # candidates of different beams lie next to one another: 64 bits for their values
    wide = x.double()
    m = wide.amax(1, keepdim=True)
    lse = m + (wide - m).exp().sum(1, keepdim=True).log()
    # within a beam the logits themselves give the order, ties to the lower column
    best = torch.sort(x, dim=1, descending=True, stable=True)
    values = best.values[:, :K].double() - lse + state["scores"].double().view(-1, 1)
    tokens = best.indices[:, :K]
    if state["ended"] is not None:
        ended = state["ended"].view(-1)
        values[ended] = float("-inf")
        values[ended, 0] = state["scores"].double().view(-1)[ended]
        tokens = tokens.masked_fill(ended[:, None], 0)
    top = torch.sort(values.view(groups, -1), dim=1, descending=True, stable=True)
    at = top.indices[:, :K]
    return (top.values[:, :K].float(), (at // values.shape[1]).int(),
            tokens.reshape(groups, -1).gather(1, at).int())


def _plain_reorder(state):
    case, page = state["case"], state["case"]["page"]
    seqs = case["groups"] * case["beams"]
    first = torch.arange(seqs, device=DEVICE) // case["beams"] * case["beams"]
    source = first + state["parents"].view(-1).long()
    lengths = state["lengths"][source]
    full, rest = (lengths // page).long(), (lengths % page).long()
    width = state["table"].shape[1]
    at = torch.arange(width, device=DEVICE)[None, :]
    state["out_table"].copy_(torch.where(at < full[:, None], state["table"][source],
                                         state["out_table"]))
    state["out_lengths"].copy_(lengths)
    last = full.clamp(max=width - 1)[:, None]
    here = state["table"][source].gather(1, last).long().view(-1)
    there = state["out_table"].gather(1, last).long().view(-1)
    keep = (torch.arange(page, device=DEVICE) < rest[:, None])[:, None, :, None]
    copied = rest > 0
    here, there, keep = here[copied], there[copied], keep[copied]
    for cache in (state["k_cache"], state["v_cache"]):
        for layer in cache:
            layer[there] = torch.where(keep, layer[here], layer[there])
    return state["k_cache"], state["v_cache"], state["out_table"], state["out_lengths"]


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "select": _exact_select,
            "reorder": _exact_reorder}[case["op"]](state)


def _host(t):
    return None if t is None else t.cpu().tolist()


def _exact_append(state):
    """Sequence by sequence: each token's pairs as complex numbers, turned by its position."""
    case = state["case"]
    k_cache, v_cache = state["k_cache"].double(), state["v_cache"].double()
    q, k, v = (state[name].double() for name in ("q", "k", "v"))
    half, page = case["rot"] // 2, case["page"]

    def turned(x, positions):
        if half == 0:
            return x
        angle = positions.double()[:, None] * state["inv_freq"].double()[None, :]
        turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
        part = x[..., :2 * half]
        if case["interleaved"]:
            z = torch.complex(part[..., 0::2].contiguous(), part[..., 1::2].contiguous()) * turn
            part = torch.stack([z.real, z.imag], dim=-1).flatten(-2)
        else:
            z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * turn
            part = torch.cat([z.real, z.imag], dim=-1)
        return torch.cat([part, x[..., 2 * half:]], dim=-1)

    starts = _host(state["starts"]) or list(range(case["seqs"] + 1))
    q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    for b, length in enumerate(_host(state["lengths"])):
        lo, hi = starts[b], starts[b + 1]
        pos = torch.arange(length - (hi - lo), length, device=DEVICE)
        where = state["table"][b].long()[pos // page]
        k_cache[where, :, pos % page] = turned(k[lo:hi], pos)
        v_cache[where, :, pos % page] = v[lo:hi]
        q_out[lo:hi] = turned(q[lo:hi], pos)
    return k_cache, v_cache, q_out


def _exact_attention(state):
    """One sequence and one key head at a time, over its own keys only."""
    case = state["case"]
    q = state["q"].double()
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=DEVICE)
    for b, length in enumerate(_host(state["lengths"])):
        if length == 0:
            continue
        ids = state["table"][b, :-(-length // case["page"])].long()
        for h in range(case["kv_heads"]):
            heads = slice(h * case["group"], (h + 1) * case["group"])
            k, v = (state[name][ids, h].reshape(-1, case["d"])[:length].double()
                    for name in ("k_cache", "v_cache"))
            log_w = torch.einsum("gd,nd->gn", q[b, heads], k) * case["d"] ** -0.5
            lse[b, heads] = torch.logsumexp(log_w, 1)
            out[b, heads] = torch.einsum("gn,nd->gd", torch.softmax(log_w, 1), v)
    return out, lse


def _exact_select(state):
    """Group by group over all beams' log-probabilities, the best of what is left in turn."""
    case = state["case"]
    groups, beams, cols, K = case["groups"], case["beams"], case["cols"], case["K"]
    values = torch.empty(groups, K, dtype=torch.float64)
    parents, tokens = (torch.empty(groups, K, dtype=torch.int32) for _ in range(2))
    for b in range(groups):
        c = torch.log_softmax(state["x"].view(groups, beams, cols)[b].double(), 1)
        c += state["scores"][b].double()[:, None]
        if state["ended"] is not None:
            for i in torch.nonzero(state["ended"][b]).flatten().tolist():
                c[i] = float("-inf")
                c[i, 0] = state["scores"][b, i].double()
        c = c.view(-1)
        for j in range(K):
            best = c.max()
            at = int(torch.nonzero(c == best)[0])
            values[b, j], parents[b, j], tokens[b, j] = float(best), at // cols, at % cols
            c[at] = float("-inf")
    return values, parents, tokens


def _exact_reorder(state):
    """Beam by beam: the parent's full pages are shared, its part-filled page copied.  Nothing is
    computed, so this too has every output, in 64 bits."""
    case, page, beams = state["case"], state["case"]["page"], state["case"]["beams"]
    old, table = _host(state["table"]), _host(state["out_table"])
    lengths, parents = _host(state["lengths"]), _host(state["parents"].view(-1))
    k_cache, v_cache, out_lengths = state["k_cache"].double(), state["v_cache"].double(), []
    for j, parent in enumerate(parents):
        p = j // beams * beams + parent
        full, rest = divmod(lengths[p], page)
        table[j][:full] = old[p][:full]
        out_lengths.append(lengths[p])
        if rest:
            for new, cache in ((k_cache, state["k_cache"]), (v_cache, state["v_cache"])):
                new[:, table[j][full], :, :rest] = cache[:, old[p][full], :, :rest].double()
    return (k_cache, v_cache, torch.tensor(table, dtype=torch.int32),
            torch.tensor(out_lengths, dtype=torch.int32))
