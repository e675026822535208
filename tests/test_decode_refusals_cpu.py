"""Refusals of the paged cache's entry points that tests/test_decode_cpu.py does not make.  No kernel
is launched here."""
import pytest

from tests.test_decode_cpu import NULL, VALUE, at, cache


@pytest.fixture(scope="module")
def st():
    import __graft_entry__
    __graft_entry__._builder().build()
    import softmax_topk_gb300
    return softmax_topk_gb300


def test_scales_whose_base_2_form_is_not_finite(st):
    """Scores are formed with scale log2 e: beyond 2^128 / log2 e a score of 0 would be NaN."""
    def call(scale):  # without a workspace, so that no accepted call runs
        return st._lib.os_paged_attention(cache(st), at(10), 256, at(11), at(12), None, 4, scale,
                                          None)

    for scale in (2.36e38, 3e38, 3.4e38):
        assert call(scale) == VALUE
    for scale in (1e-45, 1.0, 2.35e38):
        assert call(scale) == NULL
