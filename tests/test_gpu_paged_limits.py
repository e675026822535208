"""The paged cache's operators at the largest sizes that their checks let through."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def test_append_to_as_many_sequences_as_there_can_be(st):
    """2^31 - 1 sequences, nearly all of them idle: the tokens are the last two's."""
    seqs = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GB")
    k, v = (torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((seqs, 1), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    starts = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    table[-2], table[-1] = 1, 3
    lengths[-2], lengths[-1] = 2, 9
    starts[-2], starts[-1] = 2, 5
    new_k, new_v = torch.randn(2, 7, 1, 64, device="cuda").bfloat16()
    st.paged_append(k, v, table, lengths, new_k, new_v, starts=starts)
    for pool, new in ((k, new_k), (v, new_v)):
        want = torch.zeros_like(pool)
        want[1, 0, :2] = new[:2, 0]
        want[3, 0, 6:9] = new[2:5, 0]
        assert torch.equal(pool, want)
