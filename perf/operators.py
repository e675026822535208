"""The operators that a model's training and decoding loops call beside softmax, TopK and the
attention forward, as cases to be timed: the attention's gradient, the router over experts with
its gradient, and the sampler.

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
        # attention's gradient: a short causal sequence, where launches and latency count
        {"name": "attn_bwd_2x300_d64_causal", "op": "attention_bwd", "bh": 2, "n": 300, "d": 64,
         "causal": True, "dlse": True},
        # an encoder's odd length, no mask
        {"name": "attn_bwd_16x1001_d128", "op": "attention_bwd", "bh": 16, "n": 1001, "d": 128,
         "causal": False, "dlse": False},
        # training on a long context with small heads
        {"name": "attn_bwd_16x16384_d64_causal", "op": "attention_bwd", "bh": 16, "n": 16384,
         "d": 64, "causal": True, "dlse": False},
        # the benchmark's attention (batch 4, 16 heads), the largest amount of work
        {"name": "attn_bwd_64x4096_d128", "op": "attention_bwd", "bh": 64, "n": 4096, "d": 128,
         "causal": False, "dlse": False},
        # routing of a decode step: eight tokens, groups of experts, a balance bias
        {"name": "route_8x256_f32_sigmoid_groups", "op": "route", "rows": 8, "experts": 256,
         "K": 8, "dtype": "f32", "score": "sigmoid", "bias": True, "groups": 8, "topk_groups": 4,
         "group_top": 2, "renorm": True, "scale": 2.5},
        # routing of a training batch with bf16 logits, softmax scores
        {"name": "route_8191x60_bf16_softmax", "op": "route", "rows": 8191, "experts": 60, "K": 4,
         "dtype": "bf16", "score": "softmax", "bias": False, "groups": 1, "topk_groups": 1,
         "group_top": 1, "renorm": False, "scale": 1.0},
        # routing of a large batch
        {"name": "route_65536x256_f32_sigmoid_groups", "op": "route", "rows": 65536,
         "experts": 256, "K": 8, "dtype": "f32", "score": "sigmoid", "bias": True, "groups": 8,
         "topk_groups": 4, "group_top": 2, "renorm": True, "scale": 2.5},
        # the router's gradient: all of the softmax's logits get one
        {"name": "route_bwd_8191x60_bf16_softmax", "op": "route_bwd", "rows": 8191, "experts": 60,
         "K": 4, "dtype": "bf16", "score": "softmax", "renorm": False, "scale": 1.0},
        # the router's gradient of a large batch, renormalised weights
        {"name": "route_bwd_65536x256_f32_sigmoid", "op": "route_bwd", "rows": 65536,
         "experts": 256, "K": 8, "dtype": "f32", "score": "sigmoid", "renorm": True, "scale": 2.5},
        # one request's next token
        {"name": "sample_1x128256_bf16_top_p", "op": "sample", "rows": 1, "cols": 128256,
         "dtype": "bf16", "mode": "top_p"},
        # a serving batch in which every request has settings of its own
        {"name": "sample_256x50257_f32_mixed", "op": "sample", "rows": 256, "cols": 50257,
         "dtype": "f32", "mode": "mixed"},
        # a large batch drawn from the whole vocabulary at one temperature
        {"name": "sample_256x128256_bf16_temperature", "op": "sample", "rows": 256,
         "cols": 128256, "dtype": "bf16", "mode": "temperature"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention_bwd", "route", "route_bwd", "sample"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "attention_bwd":
        d = rng.choice([64, 128])
        n = _log_int(rng, 1, 16384)
        most = max(1, 64 * 4096 * 4096 * 128 // (n * n * d))
        return {"op": op, "bh": min(_log_int(rng, 1, 64), most), "n": n, "d": d,
                "causal": rng.random() < 0.6, "dlse": rng.random() < 0.3}
    if op in ("route", "route_bwd"):
        experts = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 256, 384, 512])
        case = {"op": op, "rows": _log_int(rng, 1, 65536 * 256 // max(experts, 256)),
                "experts": experts, "dtype": dtype, "score": rng.choice(["softmax", "sigmoid"]),
                "K": rng.randint(1, min(12, experts)), "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5])}
        if op == "route":
            groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0])
            size = experts // groups
            least = -(-case["K"] // size)
            case["bias"] = rng.random() < 0.6
            case["groups"] = groups
            case["topk_groups"] = rng.randint(least, groups)
            case["group_top"] = rng.choice([1, 2]) if size > 1 else 1
        return case
    cols = _log_int(rng, 500, 160000)
    return {"op": op, "rows": min(_log_int(rng, 1, 512), 256 * 128256 // cols), "cols": cols,
            "dtype": dtype, "mode": rng.choice(["temperature", "top_k", "top_p", "min_p", "mixed"])}


_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    if case["op"] == "attention_bwd":
        bh, n, d = case["bh"], case["n"], case["d"]
        pairs = n * (n + 1) // 2 if case["causal"] else n * n
        # q, k, v, o, do in, dq, dk, dv out; the logsumexp (and its gradient) in; five products
        return {"bytes": 8 * bh * n * d * 2 + bh * n * 4 * (2 if case["dlse"] else 1),
                "flops": 5 * 2 * bh * pairs * d}
    if case["op"] == "route":
        cells = case["rows"] * case["experts"]
        return {"bytes": cells * _size(case) + case["rows"] * case["K"] * 8 +
                (case["experts"] * 4 if case["bias"] else 0), "flops": 4 * cells}
    if case["op"] == "route_bwd":
        cells = case["rows"] * case["experts"]
        # where only the chosen experts' logits have a gradient the others need not be read
        read = cells if case["score"] == "softmax" and not case["renorm"] else \
            case["rows"] * case["K"]
        return {"bytes": (read + cells) * _size(case) + case["rows"] * case["K"] * 8,
                "flops": 4 * read}
    cells = case["rows"] * case["cols"]
    return {"bytes": cells * _size(case) + case["rows"] * 12, "flops": 4 * cells}


# ------------------------------------------------------------------ inputs
def _scores(q, k, scale, causal):
    s = (q @ k.transpose(-1, -2)) * scale
    if causal:
        n = s.shape[-1]
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=s.device).triu(1),
                          float("-inf"))
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=DEVICE)

    state = {"case": case}
    if case["op"] == "attention_bwd":
        shape = (case["bh"], case["n"], case["d"])
        q, k, v, do = (randn(*shape).bfloat16() for _ in range(4))
        scale = 1.0 / math.sqrt(case["d"])
        # what the forward pass left behind: its output and the rows' logsumexp
        o = torch.empty_like(q)
        lse = torch.empty(shape[:2], device=DEVICE)
        for b in range(case["bh"]):
            s = _scores(q[b].float(), k[b].float(), scale, case["causal"])
            m = s.amax(-1, keepdim=True)
            e = (s - m).exp()
            total = e.sum(-1, keepdim=True)
            o[b] = (e @ v[b].float() / total).bfloat16()
            lse[b] = (m + total.log()).squeeze(-1)
        state.update(q=q, k=k, v=v, o=o, lse=lse, do=do, scale=scale,
                     dlse=randn(*shape[:2]) if case["dlse"] else None)
    elif case["op"] == "route":
        state["x"] = randn(case["rows"], case["experts"]).to(_DTYPES[case["dtype"]])
        state["bias"] = randn(case["experts"]) * 0.1 if case["bias"] else None
    elif case["op"] == "route_bwd":
        x = randn(case["rows"], case["experts"]).to(_DTYPES[case["dtype"]])
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        state.update(x=x, idx=order[:, :case["K"]].int().contiguous(),
                     dw=randn(case["rows"], case["K"]))
    else:
        rows, cols = case["rows"], case["cols"]
        x = randn(rows, cols) * 2.5
        x += 4.0 * (rand(rows, 1) * 2 - 1)
        # a few likely tokens stand out, and a grammar forbids some
        at = torch.randint(0, cols, (rows, 6), generator=g, device=DEVICE)
        x.scatter_add_(1, at, 9.0 + 2.0 * randn(rows, 6))
        x = x.to(_DTYPES[case["dtype"]])
        x.masked_fill_(rand(rows, cols) < 0.01, float("-inf"))
        settings = {}
        if case["mode"] == "mixed":
            settings["temperature"] = 0.3 + 1.2 * rand(rows)
            settings["temperature"].masked_fill_(rand(rows) < 0.1, 0.0)
            top_k = torch.randint(1, 101, (rows,), generator=g, device=DEVICE, dtype=torch.int32)
            settings["top_k"] = top_k.masked_fill_(rand(rows) < 0.4, 0)
            settings["top_p"] = (0.5 + 0.5 * rand(rows)).masked_fill_(rand(rows) < 0.4, 1.0)
            settings["min_p"] = (0.1 * rand(rows)).masked_fill_(rand(rows) < 0.5, 0.0)
        else:
            settings["temperature"] = 0.8
            if case["mode"] == "top_k":
                settings["top_k"] = min(50, cols)
            elif case["mode"] == "top_p":
                settings["top_p"] = 0.95
            elif case["mode"] == "min_p":
                settings["min_p"] = 0.05
        state.update(x=x, u=rand(rows), settings=settings)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"attention_bwd": _plain_attention_bwd, "route": _plain_route,
            "route_bwd": _plain_route_bwd, "sample": _plain_sample}[state["case"]["op"]](state)


def _run_own(state):
    import softmax_topk_gb300 as st
    case = state["case"]
    if case["op"] == "attention_bwd":
        return st.attention_backward(state["q"], state["k"], state["v"], state["o"], state["lse"],
                                     state["do"], causal=case["causal"], scale=state["scale"],
                                     dlse=state["dlse"])
    if case["op"] == "route":
        return st.route(state["x"], case["K"], score=case["score"], bias=state["bias"],
                        groups=case["groups"], topk_groups=case["topk_groups"],
                        group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
    if case["op"] == "route_bwd":
        return st.route_backward(state["x"], state["idx"], state["dw"], score=case["score"],
                                 renorm=case["renorm"], scale=case["scale"])
    return st.sample(state["x"], state["u"], **state["settings"])


def _plain_attention_bwd(state):
    case = state["case"]
    q, k, v, o, do = (state[t].float() for t in ("q", "k", "v", "o", "do"))
    delta = (o * do).sum(-1)
    if state["dlse"] is not None:
        delta = delta - state["dlse"]
    dq, dk, dv = (torch.empty_like(state["q"]) for _ in range(3))
    step = max(1, (1 << 28) // (case["n"] * case["n"]))
    for b in range(0, case["bh"], step):
        e = slice(b, b + step)
        p = (_scores(q[e], k[e], state["scale"], case["causal"]) - state["lse"][e, :, None]).exp()
        dv[e] = (p.transpose(-1, -2) @ do[e]).bfloat16()
        ds = p * (do[e] @ v[e].transpose(-1, -2) - delta[e, :, None])
        dq[e] = (ds @ k[e] * state["scale"]).bfloat16()
        dk[e] = (ds.transpose(-1, -2) @ q[e] * state["scale"]).bfloat16()
    return dq, dk, dv


def _plain_route(state):
    case, x = state["case"], state["x"].double()  # choices next to a border need 64 bits
    if case["score"] == "softmax":
        e = (x - x.amax(1, keepdim=True)).exp()
        s = e / e.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + (-x).exp())
    choice = s if state["bias"] is None else s + state["bias"].double()
    # without a bias the logits themselves give the scores' order
    key = x if state["bias"] is None and case["groups"] == 1 else choice
    if case["groups"] > 1:
        grouped = choice.view(case["rows"], case["groups"], -1)
        best = torch.sort(grouped, dim=2, descending=True).values[:, :, :case["group_top"]].sum(2)
        top = torch.sort(best, dim=1, descending=True, stable=True).indices
        keep = torch.zeros_like(best, dtype=torch.bool)
        keep.scatter_(1, top[:, :case["topk_groups"]], True)
        key = grouped.masked_fill(~keep[:, :, None], float("-inf")).view_as(choice)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :case["K"]]
    w = s.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return (w * case["scale"]).float(), idx.int()


def _plain_route_bwd(state):
    case, x, idx = state["case"], state["x"].float(), state["idx"].long()
    dw = state["dw"] * case["scale"]
    if case["score"] == "softmax":
        e = (x - x.amax(1, keepdim=True)).exp()
        s = e / e.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + (-x).exp())
    sk = s.gather(1, idx)
    if case["renorm"]:
        total = sk.sum(1, keepdim=True)
        dw = (dw - (dw * sk / total).sum(1, keepdim=True)) / total
    ds = torch.zeros_like(s).scatter_(1, idx, dw)
    if case["score"] == "softmax":
        dx = s * (ds - (dw * sk).sum(1, keepdim=True))
        if case["renorm"]:  # the chosen experts' weights depend on their own logits only
            dx = dx * torch.zeros_like(s).scatter_(1, idx, 1.0)
    else:
        dx = ds * s * (1.0 - s)
    return dx.to(state["x"].dtype)


def _column(value, rows):
    if isinstance(value, torch.Tensor):
        return value.double()[:, None]
    return torch.full((rows, 1), float(value), dtype=torch.float64, device=DEVICE)


def _plain_sample(state):
    # cuts and draws lie next to borders, and the running sums are long: 64 bits
    x, u, s = state["x"].double(), state["u"].double()[:, None], state["settings"]
    rows, cols = x.shape
    t = _column(s.get("temperature", 1.0), rows)
    k = _column(s.get("top_k", 0), rows)
    p = _column(s.get("top_p", 1.0), rows).float().double()
    min_p = _column(s.get("min_p", 0.0), rows).float().double()
    t = t.float().double()
    greedy = t <= 0
    m = x.amax(1, keepdim=True)
    w = ((x - m) / torch.where(greedy, torch.ones_like(t), t)).exp()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(cols, device=x.device)[None, :]
    keep = (rank < k) | (k <= 0)
    wk = ws * keep
    cum = wk.cumsum(1)
    total = wk.sum(1, keepdim=True)
    keep &= (rank <= (cum < p * total).sum(1, keepdim=True)) | (p >= 1)
    keep &= ws >= min_p
    keep = torch.where(greedy, rank == 0, keep)
    kept = torch.zeros_like(w).scatter_(1, order, ws * keep)
    cum = kept.cumsum(1)
    total = cum[:, -1:]
    pick = (cum <= u * total).sum(1, keepdim=True)
    return pick.squeeze(1).int(), (kept.gather(1, pick) / total).squeeze(1).float()


# ------------------------------------------------------------------ in 64 bits, from the definitions
def exact(case, seed):
    state = prepare(case, seed)
    return {"attention_bwd": _exact_attention_bwd, "route": _exact_route,
            "route_bwd": _exact_route_bwd, "sample": _exact_sample}[case["op"]](state)


def _exact_attention_bwd(state):
    """One slice at a time, queries in blocks: dS_ij = P_ij (dO_i . (v_j) - dO_i . o_i + dL_i)."""
    case, scale = state["case"], state["scale"]
    n, d = case["n"], case["d"]
    out = [torch.zeros(case["bh"], n, d, dtype=torch.float64, device=DEVICE) for _ in range(3)]
    dq, dk, dv = out
    for b in range(case["bh"]):
        k, v = state["k"][b].double(), state["v"][b].double()
        for i in range(0, n, 2048):
            rows = slice(i, min(n, i + 2048))
            cols = slice(0, rows.stop if case["causal"] else n)
            q, o, do = (state[t][b, rows].double() for t in ("q", "o", "do"))
            logits = torch.einsum("id,jd->ij", q, k[cols]).mul_(scale)
            logits -= state["lse"][b, rows, None].double()
            p = logits.exp_()
            if case["causal"]:
                at = torch.arange(rows.start, rows.stop, device=DEVICE)
                p *= torch.arange(cols.stop, device=DEVICE)[None, :] <= at[:, None]
            shift = torch.einsum("id,id->i", do, o)
            if state["dlse"] is not None:
                shift = shift - state["dlse"][b, rows].double()
            ds = torch.einsum("id,jd->ij", do, v[cols]).sub_(shift[:, None]).mul_(p)
            dq[b, rows] = torch.einsum("ij,jd->id", ds, k[cols]) * scale
            dk[b, cols] += torch.einsum("ij,id->jd", ds, q) * scale
            dv[b, cols] += torch.einsum("ij,id->jd", p, do)
    return tuple(out)


def _numpy(t):
    return t.cpu().double().numpy()


def _exact_route(state):
    import numpy as np
    case, x = state["case"], _numpy(state["x"])
    rows, experts = x.shape
    if case["score"] == "softmax":
        s = np.exp(x - x.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    else:
        s = np.exp(np.minimum(x, 0)) / (1 + np.exp(-np.abs(x)))
    if state["bias"] is None:
        choice = s
    else:
        choice = s + _numpy(state["bias"])
    alive = np.ones((rows, experts), dtype=bool)
    if case["groups"] > 1:
        parts = choice.reshape(rows, case["groups"], -1)
        value = parts.max(2)
        if case["group_top"] == 2:
            value = value + np.partition(parts, -2, axis=2)[:, :, -2]
        best = np.argsort(-value, axis=1, kind="stable")[:, :case["topk_groups"]]
        chosen = np.zeros((rows, case["groups"]), dtype=bool)
        np.put_along_axis(chosen, best, True, axis=1)
        alive = np.repeat(chosen, experts // case["groups"], axis=1)
    key = np.where(alive, choice if state["bias"] is not None else x, -np.inf)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :case["K"]]
    w = np.take_along_axis(s, idx, axis=1)
    if case["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return torch.from_numpy(w * case["scale"]), torch.from_numpy(idx.astype(np.int32))


def _exact_route_bwd(state):
    """The gradient by differentiating the definition, in 64 bits."""
    case = state["case"]
    x = state["x"].double().requires_grad_(True)
    with torch.enable_grad():
        if case["score"] == "softmax":
            log_s = x - x.logsumexp(1, keepdim=True)
        else:
            log_s = -torch.log1p((-x).exp())
        log_w = log_s.gather(1, state["idx"].long())
        if case["renorm"]:
            log_w = log_w - log_w.logsumexp(1, keepdim=True)
        total = (log_w.exp() * state["dw"].double()).sum() * case["scale"]
    return torch.autograd.grad(total, x)[0]


def _exact_sample(state):
    """Row by row: the descending prefix that the filters leave, then the draw in column order."""
    import numpy as np
    x, u, settings = _numpy(state["x"]), _numpy(state["u"]), state["settings"]
    rows, cols = x.shape

    def setting(name, default):
        value = settings.get(name, default)
        if isinstance(value, torch.Tensor):
            return _numpy(value)
        return np.full(rows, float(np.float32(value)))

    t, k, p, min_p = (setting(*a) for a in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0),
                                            ("min_p", 0.0)))
    picks, probs = np.empty(rows, dtype=np.int32), np.empty(rows)
    for r in range(rows):
        if t[r] <= 0:
            picks[r], probs[r] = int(np.argmax(x[r])), 1.0
            continue
        w = np.exp((x[r] - x[r].max()) / t[r])
        if k[r] > 0 or p[r] < 1 or min_p[r] > 0:
            order = np.argsort(-x[r], kind="stable")
            left = int(min(k[r], cols)) if k[r] > 0 else cols
            run_sum = np.cumsum(w[order[:left]])
            if p[r] < 1:
                left = min(left, int(np.searchsorted(run_sum, p[r] * run_sum[-1], "left")) + 1)
            if min_p[r] > 0:
                left = min(left, int(np.count_nonzero(w >= min_p[r])))
            columns = np.sort(order[:left])
        else:
            columns = np.arange(cols)
        run_sum = np.cumsum(w[columns])
        at = int(np.searchsorted(run_sum, u[r] * run_sum[-1], "right"))
        picks[r], probs[r] = columns[at], w[columns[at]] / run_sum[-1]
    return torch.from_numpy(picks), torch.from_numpy(probs)
