"""The append's search for a token's sequence (sequence_of in csrc/kernels/paged_kernels.cuh) at the
largest number of sequences: its 32-bit expressions restated on the host, with unsigned places
modulo 2^32, for tokens of the first, the last and sequences between; every entry of `starts` that
a lane reads is one of the tensor's, and the sequence found is the token's."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "softmax_topk_gb300", "csrc", "kernels", "paged_kernels.cuh")
MOST = 2 ** 31 - 1


def sequence_type():
    """The type that the kernel counts places in."""
    body = open(SOURCE).read().split("int sequence_of(", 1)[1].split("\n}", 1)[0]
    return re.search(r"^\s*(\w+) lo = 0, hi = seqs;", body, re.M)[1]


def wrapped(v, kind):
    v &= 2 ** 32 - 1
    return v if kind == "unsigned" or v < 2 ** 31 else v - 2 ** 32


def find(target, seqs, kind, read):
    """The search for sequence `target` of one token each: starts[i] <= t exactly for i <= target."""
    lo, hi = 0, seqs
    for _ in range(40):
        if wrapped(hi - lo, kind) <= 1:
            return lo
        step = wrapped(hi - lo + 31, kind) // 32
        below = 0
        for lane in range(32):
            at = wrapped(lo + (lane + 1) * step, kind)
            if at < hi:
                read(at)
                below += at <= target
        lo, was = wrapped(lo + below * step, kind), lo
        hi = min(hi, wrapped(lo + step, kind))
        assert lo >= was
    raise AssertionError("does not end")


@pytest.mark.parametrize("seqs", [1, 2, 31, 32, 33, 1025, 2 ** 24 + 1, MOST - 40, MOST - 31, MOST])
def test_every_place_is_one_of_starts(seqs):
    def read(at):
        assert 0 <= at <= seqs, at

    for target in {t for t in (0, 1, seqs // 3, seqs // 2, seqs - 2, seqs - 1) if 0 <= t < seqs}:
        assert find(target, seqs, sequence_type(), read) == target
