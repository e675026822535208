"""What the router gives a token does not depend on how many are routed with it, to the bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("experts,K,groups", [(64, 4, 1), (192, 6, 4), (256, 8, 1), (256, 8, 8),
                                              (320, 6, 5), (384, 12, 3), (512, 4, 1), (1024, 16, 1),
                                              (1024, 8, 32)])
def test_weights_do_not_depend_on_the_batch(st, experts, K, groups, dtype):
    """The same bits for a token alone, among a few and among thousands."""
    g = torch.Generator(device="cuda").manual_seed(experts + K)
    x = (torch.randn(5000, experts, generator=g, device="cuda") * 2).to(DT[dtype])
    bias = torch.randn(experts, generator=g, device="cuda") * 0.1
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            for b in (None, bias):
                kw = dict(score=score, renorm=renorm, bias=b, groups=groups,
                          topk_groups=max(1, groups // 2), group_top=min(2, groups))
                w, idx = st.route(x, K, **kw)
                for lo, hi in ((0, 1), (1, 400), (400, 2431), (17, 4950)):
                    part_w, part_i = st.route(x[lo:hi].contiguous(), K, **kw)
                    assert torch.equal(part_i, idx[lo:hi])
                    assert torch.equal(part_w, w[lo:hi]), (score, renorm, lo, hi)
