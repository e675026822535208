"""Batches of the router that are large under every rule (5000 rows, the last tile ragged), against
the float64 oracle: shapes, scores, biases, missing experts, and runs of near choices."""
import pytest
import torch

from .test_gpu_route import check, check_some, logits, near_runs

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ROWS = 5003


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,K,groups,topk_groups,group_top", [
    (64, 4, 8, 3, 2), (128, 3, 1, 1, 1), (160, 6, 8, 3, 1), (192, 8, 4, 2, 2), (224, 16, 1, 1, 1),
    (256, 8, 1, 1, 1), (256, 1, 1, 1, 1), (256, 6, 8, 4, 2), (320, 5, 5, 2, 1), (384, 9, 3, 2, 2),
    (512, 16, 1, 1, 1), (640, 8, 1, 1, 1), (768, 10, 16, 7, 2), (960, 12, 15, 4, 1), (1024, 4, 1, 1, 1)])
def test_shapes(st, experts, K, groups, topk_groups, group_top, dtype, score):
    x = logits(600, experts, dtype, seed=experts + K, holes=0.2 if experts == 128 else 0.0)
    x[5] = float("-inf")
    x[599, 1:] = float("-inf")
    x[7] = 1.0
    bias = torch.randn(experts, device="cuda") * 0.1
    for b in (None, bias, bias * 0):
        kw = dict(score=score, bias=b, groups=groups, topk_groups=topk_groups, group_top=group_top,
                  renorm=K != 5, scale=1.5)
        w, idx = check(st, x, K, label=f"bias={b is not None}", **kw)
        times = ROWS // 600 + 1
        big_w, big_idx = st.route(x.repeat(times, 1)[:ROWS], K, **kw)
        at = torch.arange(ROWS, device="cuda") % 600
        assert torch.equal(big_idx, idx[at]) and torch.equal(big_w, w[at])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts", [192, 256, 512, 768, 1024])
@pytest.mark.parametrize("K", [4, 5, 8, 16])
def test_runs_of_near_choices(st, K, experts, dtype):
    """Logits that differ in their last bits only, or are equal, in random order of the experts;
    with biases that undo the order or tell equal logits apart."""
    g = torch.Generator().manual_seed(K + experts)
    x = near_runs(190, experts, g, lambda n: 5 + torch.arange(n) * 2.0 ** -21).to("cuda", DT[dtype])
    fine = (torch.randint(-3, 4, (experts,), generator=g).float() * 2.0 ** -26).cuda()
    for score in ("softmax", "sigmoid"):
        for b in (None, fine * 0, fine, fine + 0.5):
            check_some(st, x, K, rows=ROWS, score=score, bias=b)
