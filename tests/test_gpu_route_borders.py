"""The router's choice of groups against the float64 oracle where a group's two best choice values
are large and of opposite sign: their sum is small, but each of them was rounded as what it is
(|c| 2^-24)."""
import numpy as np
import pytest
import torch

from oracle import operators as ref

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LARGE = 5000  # rows of a large batch


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def logit_of(s, score):
    """The logit whose sigmoid is s, or whose exponential is s."""
    return np.log(s / (1 - s)) if score == "sigmoid" else np.log(s)


def opposite_groups(rows, experts, groups, large, score, dtype, seed):
    """Logits and biases of groups whose best two carry the biases B and -B (B up to `large`, one
    per group) and scores that add up to nearly the same in every group: apart by about the fp32
    step of B, or in bf16 by what its logits' steps make of it."""
    rng = np.random.default_rng(seed)
    size = experts // groups
    x = rng.normal(-3, 0.3, (rows, groups, size))
    bias = rng.uniform(-4, -3, (groups, size)) * large
    for g in range(groups):
        p, q = rng.choice(size, 2, replace=False)
        bias[g, p] = np.float32(rng.uniform(0.5, 1) * large)
        bias[g, q] = -bias[g, p]
        a = rng.uniform(0.2, 0.8, rows)
        x[:, g, p] = logit_of(a, score)
        x[:, g, q] = logit_of(1 - a + rng.normal(0, large * 2.0 ** -24, rows).clip(-0.1, 0.1), score)
    return (torch.tensor(x.reshape(rows, experts), device="cuda").to(DT[dtype]),
            torch.tensor(bias.reshape(experts), dtype=torch.float32, device="cuda"))


def decided(x, bias, score, groups, topk_groups):
    """Rows whose border between groups 64-bit arithmetic decides.  A choice value carries |c| 2^-53
    from its addition and up to 4 2^-53 from its score, a group's value twice that, so the
    difference of two, in either library, is off by less than 8 (|c| + 4) 2^-53."""
    c = ref.route_scores(x, score) + bias.double().cpu().numpy()
    best = np.sort(c.reshape(len(c), groups, -1), axis=2)[:, :, ::-1][:, :, :2]
    value = np.sort(best.sum(2), axis=1)[:, ::-1]
    return value[:, topk_groups - 1] - value[:, topk_groups] > 2.0 ** -50 * (np.abs(best).max() + 4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("large", [100.0, 1000.0, 2.0 ** 17])
@pytest.mark.parametrize("experts,groups", [(4, 2), (34, 17), (60, 15), (64, 32), (96, 3), (256, 32),
                                            (256, 8), (512, 16), (1024, 32), (1020, 17)])
def test_groups_of_large_opposite_biases(st, experts, groups, large, dtype, score):
    topk_groups = max(1, groups // 2)
    K = min(8, topk_groups * (experts // groups))
    x, bias = opposite_groups(125, experts, groups, large, score, dtype, seed=experts + groups)
    _, want = ref.route(x, K, score=score, bias=bias.cpu().numpy(), groups=groups,
                        topk_groups=topk_groups, group_top=2)
    sure = decided(x, bias, score, groups, topk_groups)
    if dtype == "f32":
        assert sure.mean() > 0.9
    for times in (1, LARGE // 125):
        _, idx = st.route(x.repeat(times, 1), K, score=score, bias=bias, groups=groups,
                          topk_groups=topk_groups, group_top=2)
        got = idx.cpu().numpy().reshape(times, 125, K)
        for t in range(times):
            bad = np.flatnonzero((got[t] != want).any(1) & sure)
            assert bad.size == 0, f"{times} x 125 rows: {len(bad)} differ, row {bad[0]}: " \
                                  f"{got[t, bad[0]]} for {want[bad[0]]}"


def test_groups_one_step_apart(st):
    """Two groups of true value 1 + 0.8 h and 1 + 0.6 h (h = 2^-14, the fp32 step of 1000 +
    score), which fp32 makes 1 and 1 + h of."""
    h = 2.0 ** -14
    s = np.array([[0.5 + 0.4 * h, 0.5 + 0.4 * h, 0.5 + 0.6 * h, 0.5]])
    x = torch.tensor(np.log(s / (1 - s)), dtype=torch.float32, device="cuda")
    bias = torch.tensor([1000.0, -1000.0, 1000.0, -1000.0], device="cuda")
    _, idx = st.route(x, 2, score="sigmoid", bias=bias, groups=2, topk_groups=1, group_top=2)
    assert idx.tolist() == [[0, 1]]


def test_groups_switched_off_by_their_bias(st):
    """Biases of -1e9 keep groups out, and the others' choice is still the exact one."""
    rng = np.random.default_rng(3)
    for rows in (50, LARGE):
        x = torch.tensor(rng.normal(0, 1, (rows, 256)), dtype=torch.float32, device="cuda")
        bias = torch.tensor(rng.normal(0, 0.1, 256), dtype=torch.float32, device="cuda")
        bias[64:128] = bias[192:] = -1e9
        for score in ("softmax", "sigmoid"):
            kw = dict(score=score, groups=8, topk_groups=3, group_top=2)
            _, want = ref.route(x, 8, bias=bias.cpu().numpy(), **kw)
            assert (st.route(x, 8, bias=bias, **kw)[1].cpu().numpy() == want).all()
