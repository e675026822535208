"""Beam search's selection on the GPU against the float64 oracle.

Beams and columns are those of real arithmetic, so they are compared exactly; the inputs are drawn
so that distinct values of different beams differ by more than 2^-30, or are equal throughout.
Values are good to their rounding (2^-24 of the value) and the sums' error of lse, which is below
40 units of 2^-23 (120 are allowed)."""
import numpy as np
import pytest
import torch

from oracle import decode as ref

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def check(st, x, scores, K, ended=None, pad=0, **kw):
    got = st.beam_select(x, scores, K, ended=ended, pad=pad, **kw)
    values, parents, tokens = ref.beam_select(x, scores, K, ended, pad)
    assert np.array_equal(got[1].cpu().numpy(), parents)
    assert np.array_equal(got[2].cpu().numpy(), tokens)
    v = got[0].cpu().double().numpy()
    there = values > -np.inf
    assert np.array_equal(v > -np.inf, there)
    err = np.abs(v[there] - values[there])
    assert np.all(err <= 120 * 2.0 ** -23 + 2.0 ** -24 * np.abs(values[there]))
    return got


def logits(rows, cols, seed, dtype=torch.float32, scale=2.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * scale
    x += 3 * torch.randn(rows, 1, generator=g, device="cuda")
    return x.to(dtype), torch.randn(rows, generator=g, device="cuda") * 2 - 15


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups,beams,cols,K", [
    (1, 1, 1, 1), (1, 1, 5, 8), (3, 2, 7, 4), (2, 4, 1000, 4), (1, 4, 50257, 8), (5, 3, 4097, 6),
    (2, 64, 333, 64), (1, 1, 40000, 64), (33, 5, 2000, 10), (2, 8, 32000, 16), (70, 12, 515, 24),
    (1, 6, 128256, 12), (1, 2, 262145, 33)])
def test_select(st, dtype, groups, beams, cols, K):
    x, s = logits(groups * beams, cols, seed=cols + K, dtype=dtype)
    check(st, x, s.view(groups, beams), K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_at_every_alignment(st, dtype):
    for shift in range(9):
        flat, s = logits(1, 6 * 5003 + 16, seed=shift, dtype=dtype)
        x = flat[0, shift:shift + 6 * 5003].view(6, 5003)
        check(st, x, s.expand(2, 3).contiguous() - torch.arange(6, device="cuda").view(2, 3), 7)


def test_masked_dead_and_ended(st):
    x, s = logits(12, 3001, seed=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.3] = -INF
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.01] = NAN
    x[3] = -INF                      # a row without continuations
    x[4, :] = torch.finfo(torch.float32).min
    x[5, 7:] = -INF                  # a row with seven
    s = s.view(3, 4)
    s[0, 1], s[2, 2] = -INF, NAN
    ended = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    ended[0, 0] = ended[2, 3] = True
    x[0] = NAN                       # not read
    check(st, x, s, 9, ended, pad=17)
    check(st, x, s, 64, ended, pad=3000)


def test_fewer_than_K(st):
    x = torch.full((6, 50), -INF, device="cuda")
    x[0, 3], x[0, 9], x[2, 49] = 1.0, 2.0, 0.0
    s = torch.tensor([[0.0, -1.0, -2.0], [-INF, -INF, NAN]], device="cuda")
    check(st, x, s, 8)
    ended = torch.ones(2, 3, dtype=torch.bool, device="cuda")
    got = check(st, x, s, 8, ended, pad=5)
    assert got[1][0].tolist() == [0, 1, 2, -1, -1, -1, -1, -1] and got[2][0, 0] == 5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [40, 9001])
def test_equal_values(st, dtype, cols):
    """Ties within a row go to the lower column, between beams of one value to the lower beam."""
    x = torch.zeros(8, cols, device="cuda", dtype=dtype)
    check(st, x, torch.zeros(2, 4, device="cuda"), 64)
    x = torch.randint(-2, 3, (8, cols), device="cuda").to(dtype)
    x[1:4] = x[0]
    x[5:8] = x[4]
    check(st, x, torch.full((2, 4), -3.25, device="cuda"), 33)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [1003, 50257])
def test_identical_rows_at_other_alignments(st, dtype, cols):
    """Rows of the same values start at different places of their 16 bytes, so their fp32 sums
    differ in the last bits: the exact sums find them equal."""
    x, _ = logits(1, cols, seed=5, dtype=dtype)
    check(st, x.expand(12, cols).contiguous(), torch.full((2, 6), -7.5, device="cuda"), 20)


def test_near_values(st):
    """Beams whose values differ by less than the fp32 sums' error, in either order: the scores
    differ by one unit in the last place, the rows are permutations (equal sums)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    for trial in range(20):
        row = torch.randn(7777, generator=g, device="cuda") * 3
        x = torch.stack([row[torch.rand(7777, generator=g, device="cuda").argsort()]
                         for _ in range(6)])
        s = torch.full((1, 6), -2.0, device="cuda")
        up = torch.rand(6, generator=g, device="cuda") < 0.5
        s[0, up] = torch.nextafter(s[0, up], torch.zeros((), device="cuda"))
        got = st.beam_select(x, s, 12)
        # the row's best six values, each in the better beams first; equal sums: by index
        best = row.sort(descending=True).values
        order = sorted(range(6), key=lambda i: (not bool(up[i]), i))
        assert got[1][0].tolist() == (order * 2)[:12]
        cols = [int(torch.nonzero(x[b] == best[j // 6])[0]) for j, b in enumerate(order * 2)]
        assert got[2][0].tolist() == cols


def test_infinite_and_large_logits(st):
    x, s = logits(8, 700, seed=7)
    x[0, 5] = x[0, 600] = INF
    x[1, 699] = INF
    x[2] *= 1e4
    x[3] = -3.4e38
    x[3, 11] = 3.4e38
    x[4] = 2.0 ** 127
    x[5] -= 1e30
    check(st, x, s.view(2, 4), 12)


def test_rising_rows(st):
    """Every tile passes the ones before it; and falling ones, which none passes."""
    up = torch.arange(50000, device="cuda").float()
    x = torch.stack([up * 1e-3, -up * 1e-3, up * 10, (up % 4096) * 0.01])
    check(st, x, torch.tensor([[-1.0, -1.5, -40.0, -2.0]], device="cuda"), 24)


def test_first_step(st):
    """One beam alone has a score."""
    x, _ = logits(1, 32000, seed=9)
    s = torch.full((1, 8), -INF, device="cuda")
    s[0, 0] = 0.0
    got = check(st, x.expand(8, 32000).contiguous(), s, 16)
    assert (got[1] == 0).all()


def test_buffers_and_refusals(st):
    x, s = logits(6, 500, seed=3)
    s = s.view(2, 3)
    out = torch.zeros(2, 5, device="cuda")
    parents, tokens = (torch.zeros(2, 5, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(st.os_beam_select_workspace(2, 3, 500, 5, 0), dtype=torch.uint8, device="cuda")
    got = check(st, x, s, 5, out=out, parents=parents, tokens=tokens, workspace=ws)
    assert got[0] is out and got[1] is parents and got[2] is tokens
    assert st.beam_select(x, s)[0].shape == (2, 3)
    none = st.beam_select(x[:0], s[:0], 4)
    assert none[0].shape == (0, 4)
    for error, args, kw in (
            (ValueError, (x[:5], s), {}), (ValueError, (x, s.view(-1)), {}),
            (ValueError, (x, s.double()), {}), (ValueError, (x.t(), s), {}),
            (ValueError, (x, s, 4), dict(ended=torch.zeros(2, 3, device="cuda"))),
            (ValueError, (x, s, 4), dict(out=out)), (ValueError, (x, s, 5), dict(workspace=ws[1:])),
            (TypeError, (x.half(), s), {}), (st.OsError, (x, s, 0), {}),
            (st.OsError, (x, s, 65), {}), (st.OsError, (x, s, 4), dict(pad=500)),
            (st.OsError, (x, s, 4), dict(pad=-1)), (st.OsError, (x, s, 4), dict(pad=2 ** 32)),
            (st.OsError, (x, s, 2 ** 32 + 4), {})):
        with pytest.raises(error):
            st.beam_select(*args, **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [511, 513, 600, 1105, 1793, 2000, 4095, 9297])
@pytest.mark.parametrize("K", [1, 8, 17, 64])
def test_rows_that_fill_a_tile_in_part(st, dtype, cols, K):
    """A bound that K values reach, where only some threads have columns."""
    x, s = logits(6, cols, seed=cols, dtype=dtype)
    check(st, x, s.view(2, 3), K)


def test_long_rows(st):
    """More than 2^22 columns: runs of many tiles, sums of many segments; equal rows tie."""
    cols = 5_000_011
    x, _ = logits(1, cols, seed=21, dtype=torch.bfloat16)
    x = torch.cat([x, x.flip(1), x])
    s = torch.tensor([[-3.0, -3.25, -3.0]], device="cuda")
    got = st.beam_select(x, s, 9)
    want = ref.beam_select(x[:2], s[:, :2], 9)[0]
    # beams 0 and 2 are equal: each of beam 0's columns comes in both, the lower beam first
    assert got[1][0, :2].tolist() == [0, 2] and got[2][0, 0] == got[2][0, 1]
    assert abs(float(got[0][0, 0]) - want[0, 0]) <= 200 * 2.0 ** -23 + 2.0 ** -24 * abs(want[0, 0])
    both = got[0][0][got[1][0] != 1]
    assert torch.equal(both[0:2 * (len(both) // 2):2], both[1:2 * (len(both) // 2):2])
