"""The sampler at the ends of fp32's range: logits whose difference to the row's maximum is no
fp32 number, at temperatures that make ordinary weights of them.  Against the float64 oracle, as in the
sampler's other tests."""
import pytest
import torch

from .test_gpu_sample import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(3, 40), (3, 9001), (200, 1000), (20, 50257)])
def test_differences_past_the_largest_number(st, rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = (torch.rand(rows, cols, generator=g, device="cuda") * 2 - 1) * 3.38e38
    x[0, :cols // 2] = -3.38e38  # half the row as far away as can be
    x[0, cols // 2:] = 3.38e38
    x[1, ::7] = float("-inf")
    x = x.to(dtype)
    u = torch.rand(rows, generator=g, device="cuda")
    for t in (3e37, 1e38, 3.4e38):
        for kw in ({}, {"top_k": 30}, {"top_k": cols - 1}, {"top_p": 0.9}, {"top_p": 0.3},
                   {"min_p": 0.05}, {"top_k": 25, "top_p": 0.8, "min_p": 0.01}):
            check(st, x, u, temperature=t, **kw)
