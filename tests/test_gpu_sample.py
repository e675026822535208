"""The sampler on the GPU against the float64 oracle: the drawn columns exactly, their
probabilities within 2^-22 relative (weights and sums are good to about 2^-38; the quotient is
rounded to fp32 once, 2^-24)."""
import numpy as np
import pytest
import torch

from oracle import operators as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
INF = float("inf")


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def logits(rows, cols, dtype, seed, spread=2.5, holes=0.01):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * spread
    if holes:
        hole = torch.rand(rows, cols, generator=g, device="cuda") < holes
        hole[:, 0] = False
        x.masked_fill_(hole, -INF)
    return x.to(DT[dtype]), torch.rand(rows, generator=g, device="cuda")


def check(st, x, u, label="", **kw):
    out, prob = st.sample(x, u, **kw)
    torch.cuda.synchronize()
    okw = {k: (v.cpu().numpy() if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    want, want_p = ref.sample(x, u, **okw)
    got = out.cpu().numpy()
    bad = np.flatnonzero(got != want)
    assert bad.size == 0, f"{label} {kw}: rows {bad[:5]}: {got[bad[:5]]} for {want[bad[:5]]}"
    p = prob.double().cpu().numpy()
    off = np.abs(p - want_p) - 2.0 ** -22 * want_p
    assert off.max() <= 1e-37, f"{label} {kw}: probabilities off by {off.max():.3e}"
    return out, prob


COLS = [1, 2, 3, 31, 33, 100, 513, 1000, 4099, 32000, 50257, 128256]
FILTERS = [{}, {"temperature": 0.7}, {"top_k": 1}, {"top_k": 5}, {"top_k": 50}, {"top_p": 0.9},
           {"top_p": 0.0}, {"top_p": 0.999}, {"min_p": 0.05}, {"min_p": 1.0},
           {"temperature": 1.3, "top_k": 40, "top_p": 0.8, "min_p": 0.02}]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", COLS)
def test_one_setting_for_all_rows(st, cols, dtype):
    x, u = logits(9, cols, dtype, seed=cols)
    for kw in FILTERS:
        check(st, x, u, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(64, 257), (300, 5003), (40, 50257)])
def test_a_setting_per_row(st, rows, cols, dtype):
    x, u = logits(rows, cols, dtype, seed=rows)
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + 1)

    def rand():
        return torch.rand(rows, generator=g, device="cuda")

    t = rand() * 2
    t[rand() < 0.2] = 0
    k = torch.randint(0, 2 * cols, (rows,), generator=g, device="cuda", dtype=torch.int32)
    k = torch.where(rand() < 0.5, k % 60, k)
    p = torch.where(rand() < 0.4, torch.ones_like(u), rand())
    mp = torch.where(rand() < 0.5, torch.zeros_like(u), rand() * 0.2)
    check(st, x, u, temperature=t, top_k=k, top_p=p, min_p=mp)
    check(st, x, u, temperature=0.9, top_k=k)
    check(st, x, u, temperature=t, min_p=0.03)
    check(st, x, u, top_p=p)


def test_per_row_values_outside_their_range(st):
    """Taken as the nearest inside; NaN as 0 (temperature) or off."""
    x, u = logits(12, 300, "f32", seed=5)
    nan = float("nan")
    t = torch.tensor([nan, -1.0, 0.0, -INF, 1, 1, 1, 1, 1, 1, 1, INF], device="cuda")
    k = torch.tensor([0, 0, 0, 0, -5, 2 ** 31 - 1, -2 ** 31, 300, 0, 0, 0, 0], dtype=torch.int32,
                     device="cuda")
    p = torch.tensor([1.0] * 8 + [nan, 7.0, -3.0, 1.0], device="cuda")
    mp = torch.tensor([0.0] * 8 + [nan, -1.0, 0.0, 0.0], device="cuda")
    out, prob = st.sample(x, u, temperature=t, top_k=k, top_p=p, min_p=mp)
    best = x.argmax(1).int()
    assert torch.equal(out[:4], best[:4]) and (prob[:4] == 1).all()
    plain, _ = st.sample(x, u)
    assert torch.equal(out[4:10], plain[4:10])
    assert out[10] == best[10] and prob[10] == 1          # top_p below 0 keeps the best
    live = torch.isfinite(x[11]).nonzero().flatten()      # an infinite temperature: all alike
    assert out[11] == live[int(float(u[11].double()) * len(live))]
    big, _ = st.sample(x, u, min_p=torch.full((12,), 9.0, device="cuda"))
    assert torch.equal(big, best)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties(st, dtype):
    """Equal logits: the lower columns stay, and sums of equal weights meet the border exactly."""
    x = torch.zeros(8, 1000, device="cuda")
    x[1, ::3] = 1.0
    x[2] = torch.arange(1000, device="cuda") % 7
    x[3, 500:] = -0.0
    x[4] = -5.0
    x[5, 10:] = -INF
    x[6] = torch.arange(1000, device="cuda") // 100
    x = x.to(DT[dtype])
    for value in (0.0, 0.25, 0.5, 0.75, 0.9999999):
        u = torch.full((8,), value, device="cuda")
        for kw in ({}, {"top_k": 4}, {"top_k": 333}, {"top_k": 7, "top_p": 0.5}, {"top_p": 0.5},
                   {"top_p": 0.25}, {"min_p": 0.5}, {"top_k": 600, "top_p": 0.75, "min_p": 0.1}):
            check(st, x, u, label=f"u={value}", **kw)


def test_masked_rows(st):
    x, u = logits(7, 5000, "f32", seed=6)
    x[0] = -INF
    x[1] = -INF
    x[1, 4321] = -3e38
    x[2, :4999] = -INF
    x[3] = float("nan")
    x[4, 7] = float("nan")
    x[5] = torch.finfo(torch.float32).min
    out, prob = st.sample(x, u)
    assert out[0] == -1 and prob[0] == 0 and out[3] == -1
    for kw in ({}, {"top_k": 3}, {"top_p": 0.5}, {"min_p": 0.1}, {"temperature": 0.0},
               {"top_k": 10, "top_p": 0.9, "min_p": 0.01}):
        check(st, x, u, **kw)


def test_ends_of_u(st):
    x, _ = logits(6, 777, "f32", seed=7)
    x[0, :100] = -60.0  # weights far below the sums' last bit: u = 0 still takes the first column
    for value in (0.0, -1.0, 1 - 2.0 ** -24, 1.0, 5.0, float("nan"), 2.0 ** -30):
        u = torch.full((6,), value, device="cuda")
        for kw in ({}, {"top_k": 20}, {"top_p": 0.7}):
            if value == 2.0 ** -30 and not kw:
                continue  # a draw this close to 0 may fall on either side of tiny weights
            check(st, x, u, label=f"u={value}", **kw)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.1, 30.0, 1e4, 1e38])
def test_spreads_and_temperatures(st, spread):
    x, u = logits(8, 3001, "f32", seed=8, spread=spread, holes=0)
    for t in (1e-6, 0.01, 1.0, 50.0, 1e6):
        for kw in ({}, {"top_p": 0.9}, {"top_k": 30, "top_p": 0.5}, {"min_p": 0.3}):
            check(st, x, u, temperature=t, label=f"spread={spread}", **kw)


def test_peaked_logits(st):
    """A few likely columns and a long tail, as a model's answers have."""
    x, u = logits(64, 50257, "f32", seed=9)
    x.scatter_add_(1, torch.randint(0, 50257, (64, 5), device="cuda"),
                   torch.rand(64, 5, device="cuda") * 15)
    for kw in FILTERS:
        check(st, x, u, **kw)


@pytest.mark.parametrize("rows", [3, 40, 150])
@pytest.mark.parametrize("left", [1, 7, 100, 1500, 2500, 9000])
def test_masks_that_leave_few_columns(st, left, rows):
    """Fewer columns than top-k keeps, or too few in some part of the row, in rows that one to
    eight CTAs share; scattered, and all at the row's end."""
    x, u = logits(rows, 50257, "f32", seed=left, holes=0)
    g = torch.Generator(device="cuda")
    g.manual_seed(left + 1)
    order = torch.rand(x.shape, generator=g, device="cuda")
    order[::2] += torch.arange(50257, device="cuda") * 1e-5
    kept = torch.zeros_like(x, dtype=torch.bool).scatter_(1, order.topk(left, 1)[1], True)
    x.masked_fill_(~kept, -INF)
    for kw in ({"top_k": 50}, {"top_k": 1000, "top_p": 0.9}, {"top_k": 3, "min_p": 0.2},
               {"top_p": 0.8}, {"temperature": 0.5}):
        check(st, x, u, **kw)


def test_ends_of_the_temperature(st):
    """Infinite, large and tiny temperatures under every filter, with masked columns; those below
    5e-29 act as that, which between logits of this size leaves the largest alone."""
    x, u = logits(6, 9001, "f32", seed=13, holes=0.3)
    for value in (INF, 3e38, 1e30, 5e-29, 1e-30, 1e-45):
        t = torch.full((6,), value, device="cuda")
        for kw in ({}, {"top_p": 0.5}, {"top_p": 0.999, "min_p": 0.5}, {"top_k": 40},
                   {"top_k": 2000, "top_p": 0.7}, {"min_p": 0.5}):
            check(st, x, u, temperature=t, **kw)


@pytest.mark.parametrize("rows", [1, 30, 100, 400])
def test_many_columns_at_the_border(st, rows):
    """Top-p whose border lies among thousands of small weights, which are divided again: rows of
    one to eight CTAs, many of them."""
    for cols, spread, p in ((128256, 2.5, 0.999), (50257, 0.3, 0.97), (20011, 0.01, 0.5)):
        x, u = logits(min(rows, 20), cols, "f32", seed=rows, spread=spread, holes=0)
        want, want_p = check(st, x, u, top_p=p)
        x = x.repeat((rows + 19) // 20, 1)[:rows].contiguous()
        u = u.repeat((rows + 19) // 20)[:rows].contiguous()
        for _ in range(20):
            out, prob = st.sample(x, u, top_p=p)
            at = torch.arange(rows, device="cuda") % 20
            assert torch.equal(out, want[at]) and torch.equal(prob, want_p[at])


def test_draws_follow_the_distribution(st):
    """Evenly spaced u: every column comes as often as its probability says, within one draw."""
    x, _ = logits(1, 40, "f32", seed=10)
    n = 1 << 14
    u = (torch.arange(n, device="cuda") + 0.5) / n
    out, prob = st.sample(x.expand(n, 40).contiguous(), u, top_p=0.9)
    count = torch.bincount(out.long(), minlength=40)
    _, _, kept = ref.sample_row(x[0].double().cpu().numpy(), 0.5, top_p=0.9)
    w = x[0].double().softmax(0)[kept]
    share = torch.zeros(40, dtype=torch.float64, device="cuda")
    share[kept] = w / w.sum()
    assert (count - share * n).abs().max() <= 1.0 + 1e-6


def test_unaligned_base_guards_graph_and_streams(st):
    for dtype in ("f32", "bf16"):
        flat, _ = logits(1, 20 * 3001 + 1, dtype, seed=11)
        x = flat[0, 1:].view(20, 3001)
        u = torch.rand(20, device="cuda")
        raw_o = torch.full((22,), 7, dtype=torch.int32, device="cuda")
        raw_p = torch.full((22,), 7.0, device="cuda")
        kw = dict(temperature=0.8, top_k=100, top_p=0.95)
        want = [t.clone() for t in check(st, x, u, **kw)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            st.sample(x, u, out=raw_o[1:21], prob=raw_p[1:21], **kw)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(raw_o[1:21], want[0]) and torch.equal(raw_p[1:21], want[1])
        assert raw_o[0] == 7 and raw_o[21] == 7 and raw_p[0] == 7 and raw_p[21] == 7
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            again = st.sample(x, u, **kw)
        side.synchronize()
        assert torch.equal(again[0], want[0])


def test_refusals(st):
    x, u = logits(4, 100, "f32", seed=1)
    for kw in (dict(temperature=-1.0), dict(top_k=-1), dict(top_p=1.5), dict(min_p=float("nan"))):
        with pytest.raises(st.OsError):
            st.sample(x, u, **kw)
    with pytest.raises(ValueError):
        st.sample(x, u[:3])
    with pytest.raises(ValueError):
        st.sample(x, u.double())
    with pytest.raises(ValueError):
        st.sample(x, u, top_k=torch.ones(4, device="cuda"))
    with pytest.raises(TypeError):
        st.sample(x.half(), u)
    assert torch.equal(st.sample(x, u, top_k=2 ** 32 + 1)[0], st.sample(x, u)[0])  # off, not 1
    out, prob = st.sample(x[:0], u[:0])
    assert out.shape == (0,) and prob.shape == (0,)
