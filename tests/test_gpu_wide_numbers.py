"""Numbers that 32 bits do not hold, as arguments of the router and the sampler: refused, or taken
for what they are, never for their low bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
WIDE = 2 ** 32


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def test_route(st):
    x = torch.randn(4, 64, device="cuda")
    for kw in (dict(groups=WIDE + 1), dict(groups=8, topk_groups=WIDE + 2),
               dict(groups=8, group_top=WIDE + 1), dict(score=WIDE)):
        with pytest.raises(st.OsError):
            st.route(x, 2, **kw)
    for K in (WIDE + 4, 2 ** 31):
        with pytest.raises(st.OsError):
            st.route(x[:0], K)
    w, idx = st.route(x, 4)
    with pytest.raises(st.OsError):
        st.route_backward(x, idx, w, score=WIDE)


def test_top_k(st):
    """Refused below 0, off above a row's length."""
    x = torch.randn(3, 100, device="cuda")
    u = torch.rand(3, device="cuda")
    for k in (-1, -2 ** 31, -2 ** 31 - 1, -WIDE, -WIDE + 5, -2 ** 40):
        with pytest.raises(st.OsError):
            st.sample(x, u, top_k=k)
    for k in (100, 2 ** 31, WIDE, 2 ** 40 + 1):
        assert torch.equal(st.sample(x, u, top_k=k)[0], st.sample(x, u)[0])
