"""Choices by softmax scores under a bias in rows of many experts, where the denominator is a sum of
as many terms, against the float64 oracle."""
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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,groups", [(1024, 1), (1024, 4), (960, 1), (1020, 17), (1008, 21)])
def test_softmax_of_many_experts_beside_one(st, experts, groups, dtype):
    """One logit `spread` above the others, all equal (or nearly): the others' exponentials are
    small steps of the sum beside the first, and biases leave 1e-7 to 2e-6 between the first
    expert's choice value and another's.  The oracle's 64 bits decide all of these (1e-15)."""
    rng = np.random.default_rng(experts + groups)
    first, other = 0, experts - 1
    for spread in (16.0, 16.7, 17.25, 17.75, 18.0625, 18.5):
        x = torch.full((5, experts), 0.25)
        x[1:] += torch.tensor(rng.normal(0, 0.05, (4, experts)), dtype=torch.float32)
        x[:, first] = x[:, other] + spread
        x = x.to("cuda", DT[dtype])
        s = ref.route_scores(x, "softmax")
        for row in (0, 1 + int(rng.integers(4))):
            for gap in (1e-7, 3e-7, 6e-7, 1e-6, 1.5e-6, 2e-6):
                for sign in (1, -1):
                    bias = torch.full((experts,), -1.0)
                    bias[first] = -0.9
                    bias[other] = float(s[row, first] - 0.9 + sign * gap - s[row, other])
                    _, want = ref.route(x[row:row + 1], 2, bias=bias.numpy(), groups=groups,
                                        topk_groups=groups)
                    one = x[row:row + 1].contiguous()
                    bias = bias.cuda()
                    for rows in (1, LARGE):
                        _, idx = st.route(one.repeat(rows, 1), 2, bias=bias, groups=groups,
                                          topk_groups=groups)
                        assert (idx == torch.tensor(want, device="cuda")).all(), \
                            (spread, row, sign * gap, rows)
