"""The attention gradient beside query rows without keys (L = -inf), whose output and whose
gradient of L are NaN or infinite, as the derivative of a -inf logsumexp is: such a row takes no
part, so its dQ is 0 and nothing of it reaches another row."""
import math

import pytest
import torch

from .test_gpu_attention_bwd import bounds, check, make

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


@pytest.mark.parametrize("rough", [NAN, INF, -INF])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 150, 300])
def test_rows_without_keys_hold_anything(st, n, d, causal, rough):
    q, k, v, do = make(3, n, d, seed=n + d)
    o, lse = st.attention(q, k, v, causal=causal)
    dlse = torch.randn_like(lse)
    empty = torch.zeros(3, n, dtype=torch.bool, device="cuda")
    empty[0, 0] = empty[1, n - 1] = empty[1, n // 2] = True
    empty[2] = True  # a slice of nothing else
    lse[empty] = -INF
    o[empty], dlse[empty] = 0, 0
    want, err = bounds(q, k, v, o, lse, do, 1 / math.sqrt(d), causal, dlse)
    for what in ("o", "dlse", "both"):
        oo, dl = o.clone(), dlse.clone()
        if what != "dlse":
            oo[empty] = rough
        if what != "o":
            dl[empty] = rough
        got = st.attention_backward(q, k, v, oo, lse, do, causal=causal, dlse=dl)
        check(got, want, err, f"n={n} d={d} causal={causal} {what}")
        assert not got[0][empty].any() and not got[1][2].any() and not got[2][2].any()
