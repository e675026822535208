"""The router over experts and its gradient on the GPU against the float64 oracle: chosen experts
exactly, weights and gradients element by element.

Tolerance (u = 2^-24, the fp32 half step): a score is an exponential (2u) of a difference rounded
once (|z| u with |z| the spread of the row's logits), divided by a sum of such (as much again, and
one rounding per addition: 5 in a lane's run and 5 over the warp, 64 terms at most in a run), so it
is within (2 spread + 80) u relative; a renormalised weight is a quotient of such, twice that; the
scale and the store round once each.  A gradient is a product of three such factors, one of them
a difference g - D whose error is (2 spread + 80) u of |g| + |D|.  bf16 gradients round by 2^-8.
"""
import numpy as np
import pytest
import torch

from oracle import operators as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def logits(rows, experts, dtype, seed, spread=1.0, holes=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, experts, generator=g, device="cuda") * spread
    if holes:
        x.masked_fill_(torch.rand(rows, experts, generator=g, device="cuda") < holes, float("-inf"))
    return x.to(DT[dtype])


def spread_of(x):
    x = x.double()
    low = x.masked_fill(x == float("-inf"), float("inf")).amin()
    return float(x.amax() - low.clamp(max=1e9)) if x.isfinite().any() else 0.0


def check(st, x, K, label="", groups_tied=None, **kw):
    w, idx = st.route(x, K, **kw)
    torch.cuda.synchronize()
    okw = dict(kw)
    if okw.get("bias") is not None:
        okw["bias"] = okw["bias"].cpu().numpy().astype(np.float64)
    want_w, want_idx = ref.route(x, K, **okw)
    got = idx.cpu().numpy()
    bad = np.argwhere((got != want_idx).any(1))
    if groups_tied is not None:
        bad = np.array([b for b in bad if not groups_tied(x[int(b[0])], okw)])
    assert bad.size == 0, f"{label}: {len(bad)} rows differ, row {bad[0]}: {got[bad[0, 0]]} " \
                          f"for {want_idx[bad[0, 0]]}"
    rel = (4 * spread_of(x) + 170) * U
    off = np.abs(w.double().cpu().numpy() - want_w) - rel * np.abs(want_w)
    assert off.max() <= 1e-37 * abs(kw.get("scale", 1.0)), f"{label}: weights off by {off.max():.3e}"
    return w, idx


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,K", [(1, 1), (2, 2), (7, 3), (8, 2), (32, 32), (33, 5), (60, 4),
                                       (64, 6), (127, 8), (128, 1), (256, 8), (384, 8), (512, 10),
                                       (1000, 32), (1024, 8)])
def test_plain(st, experts, K, dtype, score, renorm):
    x = logits(37, experts, dtype, seed=experts)
    check(st, x, K, score=score, renorm=renorm, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,K,groups,topk_groups,group_top", [
    (256, 8, 8, 4, 2), (64, 6, 8, 3, 1), (60, 4, 3, 2, 2), (160, 6, 8, 3, 1), (35, 5, 5, 2, 2),
    (96, 4, 12, 5, 2), (17, 3, 17, 9, 1), (1024, 8, 32, 4, 2), (1020, 8, 17, 4, 2), (24, 4, 2, 1, 2),
    (1023, 12, 3, 1, 2), (990, 12, 11, 3, 1), (32, 1, 32, 1, 1)])
def test_groups(st, experts, K, groups, topk_groups, group_top, dtype, score):
    x = logits(41, experts, dtype, seed=experts + groups)
    bias = torch.randn(experts, device="cuda") * 0.1
    for b in (None, bias):
        check(st, x, K, label=f"bias={b is not None}", score=score, bias=b, groups=groups,
              topk_groups=topk_groups, group_top=group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,K,groups,topk_groups,group_top", [
    (64, 1, 1, 1, 1), (64, 4, 8, 3, 2), (128, 3, 1, 1, 1), (128, 8, 4, 2, 2), (256, 8, 1, 1, 1),
    (256, 6, 8, 4, 2), (320, 5, 5, 2, 1), (384, 9, 3, 2, 2), (512, 16, 1, 1, 1), (512, 10, 16, 7, 2),
    (256, 1, 1, 1, 1), (256, 4, 32, 9, 2), (1024, 8, 1, 1, 1), (960, 12, 15, 4, 1)])
def test_batches_of_a_thread_per_row(st, experts, K, groups, topk_groups, group_top, dtype, score):
    """Rows enough for the kernel with a thread per row, the last tile ragged; with and without
    a bias, missing experts and empty rows among them."""
    x = logits(2457, experts, dtype, seed=experts + K, holes=0.2 if experts == 128 else 0.0)
    x[5] = float("-inf")
    x[2456, 1:] = float("-inf")
    x[7] = 1.0
    bias = torch.randn(experts, device="cuda") * 0.1
    for b in (None, bias, bias * 0):
        check(st, x, K, label=f"bias={b is not None}", score=score, bias=b, groups=groups,
              topk_groups=topk_groups, group_top=group_top, renorm=K != 5, scale=1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties_in_a_large_batch(st, score):
    g = torch.Generator(device="cuda")
    g.manual_seed(19)
    base = torch.randn(2500, 1, generator=g, device="cuda")
    x = base + torch.randint(-3, 4, (2500, 256), generator=g, device="cuda") * 2.0 ** -24 * base.abs()
    bias = torch.randint(-2, 3, (256,), generator=g, device="cuda").float() * 2.0 ** -25
    for b in (None, bias, bias + 1.0, bias * 0):
        check(st, x, 7, score=score, bias=b)


def near_runs(rows, experts, g, values):
    """Normal logits, in row r 2 + r % 19 of them at random places replaced by values(n)."""
    x = torch.randn(rows, experts, generator=g)
    for r in range(rows):
        n = 2 + r % 19
        x[r, torch.randperm(experts, generator=g)[:n]] = values(n)
    return x


def check_some(st, x, K, rows=2500, **kw):
    """x, and rows of it again up to `rows` in all (a large batch), against the oracle of x."""
    big = x.repeat((rows + len(x) - 1) // len(x), 1)[:rows]
    w, idx = st.route(big, K, **kw)
    idx = idx.cpu().numpy()
    okw = dict(kw)
    if okw.get("bias") is not None:
        okw["bias"] = okw["bias"].cpu().numpy().astype(np.float64)
    _, want = ref.route(x, K, **okw)
    tied = okw.get("groups", 1) > 1 and okw["group_top"] == 2
    for r in range(len(x)):
        if (idx[r::len(x)] != want[r]).any() and not (tied and _border_below_64_bits(x[r], okw)):
            raise AssertionError(f"row {r}: {idx[r]} for {want[r]}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,K,groups", [(256, 2, 1), (256, 4, 1), (256, 6, 1), (256, 8, 1),
                                              (512, 12, 1), (512, 16, 1), (256, 8, 8), (1024, 8, 4)])
def test_runs_of_near_choices(st, experts, K, groups, dtype):
    """Runs of 2 to 20 saturated scores (1 - e^-x, x from 14 to 22: hardly two apart in fp32, all
    in 64 bits) in orders of every kind, below and across the border of the choice, with one bias
    for all and with biases that differ in the last bits."""
    g = torch.Generator().manual_seed(experts + K + groups)
    x = near_runs(190, experts, g, lambda n: 14 + 8 * torch.rand(n, generator=g)).to("cuda", DT[dtype])
    fine = (torch.randint(-3, 4, (experts,), generator=g).float() * 2.0 ** -24).cuda()
    coarse = (torch.randint(0, 3, (experts,), generator=g).float() * 2.0 ** -12).cuda()
    for b in (fine * 0, fine, fine + 0.5, coarse):
        check_some(st, x, K, score="sigmoid", bias=b, groups=groups, topk_groups=max(1, groups // 2),
                   group_top=2 if groups > 1 else 1)


@pytest.mark.parametrize("K", [4, 5, 8, 16])
def test_runs_of_near_logits(st, K):
    """Logits that differ in their last bits only, in random order of the experts."""
    g = torch.Generator().manual_seed(K)
    x = near_runs(190, 1024, g, lambda n: 5 + torch.arange(n) * 2.0 ** -21).cuda()
    for score in ("softmax", "sigmoid"):
        check_some(st, x, K, score=score)
        check_some(st, x, K, score=score, bias=torch.zeros(1024, device="cuda"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_large_batches(st, score):
    """Many rows: choices that turn on the last bits of fp32 come up and are settled in 64 bits."""
    for dtype in ("f32", "bf16"):
        x = logits(6000, 256, dtype, seed=3)
        bias = torch.randn(256, device="cuda") * 0.1
        check(st, x, 8, label=dtype, score=score, bias=bias, groups=8, topk_groups=4, group_top=2,
              scale=2.5)


def _border_below_64_bits(row, kw):
    """Whether the values of the last group taken and the first left out are closer than 64-bit
    arithmetic orders.  Two scores that each carry up to 2 ulp (of at most 2^-53) in either
    library and a sum that rounds once more give values within 5 * 2^-53 each of the true ones:
    borders under 2^-49 = 16 * 2^-53 are not decided.  Sums such as s(x + 3h) + s(x + h) and
    2 s(x + 2h), h = 2^-24 |x|, differ by h^2 s'' < 2^-48 |s''|, so they come up here."""
    s = ref.route_scores(row[None], kw["score"])[0]
    c = s + (0 if kw.get("bias") is None else kw["bias"])
    best = np.sort(c.reshape(kw["groups"], -1), axis=1)[:, ::-1][:, :kw["group_top"]].sum(1)
    best = np.sort(best)[::-1]
    return best[kw["topk_groups"] - 1] - best[kw["topk_groups"]] < 2.0 ** -49


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties(st, score):
    """Logits a few fp32 steps apart, so that scores plus bias collide in fp32 in every row, and
    the bias alone decides or undoes the order."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    base = torch.randn(300, 1, generator=g, device="cuda")
    steps = torch.randint(-3, 4, (300, 64), generator=g, device="cuda").float()
    x = base + steps * 2.0 ** -24 * base.abs()
    bias = torch.randint(-2, 3, (64,), generator=g, device="cuda").float() * 2.0 ** -25
    for b in (None, bias, bias + 1.0, bias * 0):
        check(st, x, 8, score=score, bias=b, groups=8, topk_groups=3, group_top=2,
              groups_tied=_border_below_64_bits)
        check(st, x, 8, score=score, bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_exact_ties_go_to_the_lower_expert(st, score):
    x = torch.zeros(5, 48, device="cuda")
    x[1] = torch.tensor([1.0, 2.0, 0.0] * 16)
    x[2, 10:] = -0.0
    x[3] = 3.0
    zero = torch.zeros(48, device="cuda")
    for b in (None, zero, zero + 7):
        for kw in ({}, {"groups": 6, "topk_groups": 2, "group_top": 2}):
            check(st, x, 6, score=score, bias=b, **kw)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_missing_experts_and_empty_rows(st, score, renorm):
    x = logits(64, 40, "f32", seed=4, holes=0.5)
    x[0] = float("-inf")
    x[1, 1:] = float("-inf")
    x[2, :39] = float("-inf")
    bias = torch.randn(40, device="cuda")
    for b in (None, bias):
        for kw in ({}, {"groups": 4, "topk_groups": 2, "group_top": 2}):
            w, _ = check(st, x, 5, score=score, bias=b, renorm=renorm, **kw)
            assert not w[0].any() and w.isfinite().all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_apart_logits(st, score):
    """Scores that underflow: renormalised weights are still ratios of them."""
    x = torch.tensor([[-200.0, -201.0, -199.0, -300.0], [90.0, 80.0, -90.0, 0.0],
                      [-1000.0, -1000.5, -3e38, -1001.0], [1e30, 1e30, -1e30, 0.0]], device="cuda")
    w, idx = st.route(x, 2, score=score)
    want, want_idx = ref.route(x, 2, score=score)
    assert (idx.cpu().numpy() == want_idx).all()
    assert np.abs(w.cpu().numpy() - want).max() <= 300 * U


def test_strided_base_and_unaligned_rows(st):
    """Rows that start anywhere, and a base one element past a 16-byte boundary."""
    for dtype in ("f32", "bf16"):
        flat = logits(1, 50 * 256 + 1, dtype, seed=6)[0]
        x = flat[1:].view(50, 256)
        bias = torch.randn(257, device="cuda")[1:]
        check(st, x, 8, score="sigmoid", bias=bias)
        _, idx = st.route(x, 8)
        dw = torch.randn(50, 8, device="cuda")
        check_bwd(st, x, idx, dw, "softmax", False)


def check_bwd(st, x, idx, dw, score, renorm, scale=1.5, dx=None):
    dx = st.route_backward(x, idx, dw, score=score, renorm=renorm, scale=scale, dx=dx)
    torch.cuda.synchronize()
    assert dx.dtype == x.dtype and dx.shape == x.shape
    want = ref.route_backward(x, idx, dw, score=score, renorm=renorm, scale=scale)
    # error: rel of what each element is made of: s (|g| + sum |g s|) scaled, slots added up
    size = np.zeros_like(want)
    g = np.abs(dw.double().cpu().numpy()) * abs(scale)
    ii = idx.cpu().numpy()
    s = ref.route_scores(x, score)
    for r in range(len(want)):
        top = g[r].sum()
        for k, e in enumerate(ii[r]):
            if 0 <= e < want.shape[1]:
                size[r, e] += (g[r, k] + top) * (1.0 if renorm else s[r, e])
        if score == "softmax" and not renorm:
            size[r] += s[r] * top
    rel = (4 * spread_of(x) + 170) * U
    tol = rel * size + (2.0 ** -8 * np.abs(want) if x.dtype == torch.bfloat16 else 0) + 1e-37
    off = np.abs(dx.double().cpu().numpy() - want) - tol
    assert off.max() <= 0, f"{score} renorm={renorm}: off by {off.max():.3e} over the bound"
    return dx


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,K", [(1, 1), (3, 2), (8, 8), (32, 4), (60, 4), (64, 6), (129, 7),
                                       (256, 8), (511, 32), (1024, 8)])
def test_gradient(st, experts, K, dtype, score, renorm):
    x = logits(29, experts, dtype, seed=experts + 1)
    _, idx = st.route(x, K, score=score)
    dw = torch.randn(29, K, device="cuda")
    check_bwd(st, x, idx, dw, score, renorm)


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_odd_indices_and_missing_experts(st, score, renorm):
    """Experts named twice count twice, those outside the row take no part, a missing expert
    (-inf) and an empty row get no gradient."""
    x = logits(40, 24, "f32", seed=8, holes=0.3)
    x[0] = float("-inf")
    idx = torch.randint(-3, 30, (40, 6), dtype=torch.int32, device="cuda")
    idx[5] = 2
    idx[6] = -1
    idx[7] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1, 2, 3])
    dx = check_bwd(st, x, idx, torch.randn(40, 6, device="cuda"), score, renorm)
    assert not dx[0].any() and not dx[6].any() and dx.isfinite().all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_differences(st, score, renorm):
    x = logits(16, 32, "f32", seed=10)
    w, idx = st.route(x, 4, score=score, renorm=renorm)
    dw = torch.randn(16, 4, device="cuda")
    dx = st.route_backward(x, idx, dw, score=score, renorm=renorm).double().cpu().numpy()
    way = np.random.default_rng(0).standard_normal(x.shape)
    x64, at, g = x.double().cpu().numpy(), idx.cpu().numpy().astype(np.int64), dw.double().cpu().numpy()

    def loss(a):
        t = np.take_along_axis(ref.route_scores(a, score), at, 1)
        return ((t / t.sum(1, keepdims=True) if renorm else t) * g).sum()

    numeric = (loss(x64 + 1e-6 * way) - loss(x64 - 1e-6 * way)) / 2e-6
    tol = 200 * U * (np.abs(way).max() * np.abs(g).sum() * 8) + 1e-7 * abs(numeric)
    assert abs((dx * way).sum() - numeric) <= tol


def test_graph_streams_and_guards(st):
    x = logits(1000, 256, "f32", seed=12)
    bias = torch.randn(256, device="cuda") * 0.1
    kw = dict(score="sigmoid", bias=bias, groups=8, topk_groups=4, group_top=2, scale=2.5)
    raw_w = torch.full((1002, 8), 7.0, device="cuda")
    raw_i = torch.full((1002, 8), 7, dtype=torch.int32, device="cuda")
    raw_d = torch.full((1002, 256), 7.0, device="cuda")
    w, idx, dx = raw_w[1:1001], raw_i[1:1001], raw_d[1:1001]
    dw = torch.randn(1000, 8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.route(x, 8, weights=w, idx=idx, **kw)
        st.route_backward(x, idx, dw, score="sigmoid", scale=2.5, dx=dx)
    for seed in (1, 2):
        x.copy_(logits(1000, 256, "f32", seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want_w, want_i = st.route(x, 8, **kw)
            want_d = st.route_backward(x, want_i, dw, score="sigmoid", scale=2.5)
        side.synchronize()
        assert torch.equal(w, want_w) and torch.equal(idx, want_i) and torch.equal(dx, want_d)
    for raw in (raw_w, raw_i, raw_d):
        assert (raw[0] == 7).all() and (raw[1001] == 7).all()


def test_refusals(st):
    x = logits(4, 16, "f32", seed=1)
    for kw in (dict(K=0), dict(K=17), dict(K=2, groups=3), dict(K=2, score=5),
               dict(K=2, scale=float("nan")), dict(K=9, groups=2, topk_groups=1)):
        with pytest.raises(st.OsError):
            st.route(x, **kw)
    with pytest.raises(ValueError):
        st.route(x, 2, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        st.route(x.t(), 2)
    with pytest.raises(TypeError):
        st.route(x.half(), 2)
    with pytest.raises(ValueError):
        st.route_backward(x, torch.zeros(4, 2, dtype=torch.int64, device="cuda"),
                          torch.zeros(4, 2, device="cuda"))
    w, i = st.route(x[:0], 2)
    assert w.shape == (0, 2) and st.route_backward(x[:0], i, w).shape == (0, 16)
