"""Beam search's selection where its fp32 sums are at their worst: rows whose mass lies before
values that each pass the running reference by just over 1, and long rows.

Values are compared to the bound that the kernels go by (csrc/beam_error.h, worked out in
tests/test_beam_error_cpu.py), with the largest share of columns that a thread can have, and half
a step of the output; choices exactly."""
import math

import numpy as np
import pytest
import torch

from oracle import decode as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -23


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def bound(cols, share):
    return U * (0.612 * (3 + math.log(cols)) + 20.25 + 1.25 * (math.log(share) + 0.6) +
                share * share * 2.0 ** -26)


def rising(rows, tiles, last, step):
    """fp32 rows of `tiles` tiles (256 threads, 16 columns each) of zeros, the last ones with one
    value per thread that is `step` above the one before it."""
    x = torch.zeros(rows, tiles, 4, 256, 4, device="cuda")
    x[:, tiles - last:] = -60.0
    for j in range(last):
        x[:, tiles - last + j, 0, :, 0] = (j + 1) * step
    return x.view(rows, -1)


@pytest.mark.parametrize("step", [1.32122802734375, 1.72967529296875])
@pytest.mark.parametrize("tiles", [125, 1000])
def test_values_of_rising_rows(st, step, tiles):
    """One beam a group, so that no row is summed again; more rows than CTAs, so that each is one
    run."""
    for last in (0, 1, 4, 6, 8):
        x = rising(460, tiles, last, step)
        row = x[0].double()
        c = float(row.max() - torch.logsumexp(row, 0))
        scores = torch.full((460, 1), -c, device="cuda")
        got = st.beam_select(x, scores, 1)[0].double()
        want = float(scores[0, 0].double()) + c
        cols = x.shape[1]
        assert float((got - want).abs().max()) <= bound(cols, cols // 256) + 2.0 ** -24 * abs(want)


def test_choices_between_rising_and_falling_rows(st):
    """A row and the same values backwards: equal sums whose fp32 errors differ, and scores a unit in
    the last place apart, in either order."""
    x = rising(460, 125, 6, 1.32122802734375)
    x[1::2] = x[0].flip(0)
    scores = torch.full((230, 2), -2.0, device="cuda")
    up = torch.arange(230, device="cuda") % 3
    near = torch.nextafter(scores[0, 0], torch.zeros((), device="cuda"))
    scores[up == 1, 0] = near
    scores[up == 2, 1] = near
    _, parents, _ = st.beam_select(x, scores, 2)
    top = int((x[0] == x[0].max()).sum())
    assert top >= 2  # both places of a group are its better beam's
    want = (up == 2).int()
    assert torch.equal(parents[:, 0], want) and torch.equal(parents[:, 1], want)


@pytest.mark.parametrize("base", [2.0 ** 24, -2.0 ** 26, 2.0 ** 27, 2.0 ** 29])
def test_rows_far_from_zero(st, base):
    """Maxima beyond 2^24, whose products with log2 e are rounded to whole numbers."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    gap = max(1.0, abs(base) * 2.0 ** -23)
    x = base - gap * torch.randint(0, 12, (10, 30011), generator=g, device="cuda").double()
    x = x.float()
    s = -torch.rand(10, 1, generator=g, device="cuda")
    got = st.beam_select(x, s, 20)
    values, parents, tokens = ref.beam_select(x, s, 20)
    assert np.array_equal(got[1].cpu().numpy(), parents)
    assert np.array_equal(got[2].cpu().numpy(), tokens)
    err = np.abs(got[0].cpu().double().numpy() - values)
    assert np.all(err <= bound(30011, 128) + 5.5 * U + 2.0 ** -24 * np.abs(values))
    # beams that differ by little, and equal rows
    x[1], x[6] = x[0].flip(0), x[5]
    s = torch.full((2, 5), -1.0, device="cuda")
    s[0, 1] = torch.nextafter(s[0, 0], torch.zeros((), device="cuda"))
    s[:, 2:] = -9.0
    got = st.beam_select(x, s, 12)
    values, parents, tokens = ref.beam_select(x, s, 12)
    assert np.array_equal(got[1].cpu().numpy(), parents)
    assert np.array_equal(got[2].cpu().numpy(), tokens)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_rows_in_full(st, dtype):
    """Every value, beam and column of rows of five million, two of them equal."""
    cols = 5_000_011
    g = torch.Generator(device="cuda")
    g.manual_seed(22)
    x = (torch.randn(1, cols, generator=g, device="cuda") * 2.5).to(dtype)
    x = torch.cat([x, x.flip(1), x])
    s = torch.tensor([[-3.0, -3.25, -3.0]], device="cuda")
    got = st.beam_select(x, s, 9)
    values, parents, tokens = ref.beam_select(x, s, 9)
    assert np.array_equal(got[1].cpu().numpy(), parents)
    assert np.array_equal(got[2].cpu().numpy(), tokens)
    err = np.abs(got[0].cpu().double().numpy() - values)
    # (one run in 32 of the row, by 256 threads, in tiles of up to 32 columns a thread)
    assert np.all(err <= bound(cols, cols // 32 // 256 + 64) + 2.0 ** -24 * np.abs(values))
