"""The bound of the fp32 sums of beam search's selection (csrc/beam_error.h), which decides which
beams are summed again exactly: against its terms worked out another way, and against the kernel's
arithmetic replayed in fp32 with every ex2.approx off by as much as it may be."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "softmax_topk_gb300", "csrc")
U = 2.0 ** -23
f32 = np.float32


@pytest.fixture(scope="module")
def bound(tmp_path_factory):
    """beam_lse_error(cols, share) in units of 2^-23."""
    d = tmp_path_factory.mktemp("beam_error")
    src, lib = d / "bound.cpp", d / "bound.so"
    src.write_text('#include "beam_error.h"\n'
                   'extern "C" double bound(long long cols, long long share) {\n'
                   '    return os::beam_lse_error(cols, share);\n}\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)],
                   check=True)
    fn = ctypes.CDLL(str(lib)).bound
    fn.restype, fn.argtypes = ctypes.c_double, [ctypes.c_longlong] * 2
    return lambda cols, share: fn(cols, share) / U


# columns of a row, columns that one thread sums of a run
SIZES = [(1, 16), (7, 16), (1000, 16), (50257, 32), (128256, 512), (5_000_011, 640),
         (5_000_011, 20000), (2 ** 31 - 1, 2 ** 18), (2 ** 31 - 1, 2 ** 23)]


@pytest.mark.parametrize("cols,share", SIZES)
def test_changes_of_the_reference(bound, cols, share):
    """`share` weights near the first reference, then values that each pass the reference by just
    over 1: what k changes of 1.25 units leave on the whole sum, for the worst k, beside the terms
    that do not depend on the share.  (No constant of 40 units is a bound for 20000 columns a
    thread.)"""
    worst, later = 0.0, 0.0
    for k in range(1, 60):
        later += math.exp(1 - k)  # the values that came, beside the last
        mass = share * math.exp(-k)
        worst = max(worst, 1.25 * k * mass / (mass + later))
    rest = 0.612 * (3 + math.log(cols)) + 2.5 + 2 + 5 + 10.75
    assert bound(cols, share) >= rest + worst
    if share >= 20000:
        assert rest + worst + share ** 2 * 2.0 ** -26 > 40


def test_mean_distance_and_mean_number_of_changes():
    """Of n weights e^-y, one of them 1, y is at most 1 + ln n in the mean; of `share` weights of
    which those behind j changes are below e^-j, the changes at most ln share + 0.6."""
    rng = np.random.default_rng(0)
    for n in (1, 2, 10, 512, 10 ** 5, 10 ** 9, 2 ** 31):
        for y in np.concatenate([np.linspace(0, 40, 2001), rng.random(200) * 40]):
            # all other columns at one distance: the worst place for them
            rest = (n - 1) * math.exp(-y)
            assert rest * y / (rest + 1) <= 1 + math.log(n)
        mean = sum(min(1.0, n * math.exp(-j)) for j in range(1, 100))
        assert mean <= math.log(n) + 0.6


def fma(a, b, c):
    return (np.float64(a) * np.float64(b) + np.float64(c)).astype(f32)


def exp1(z):
    """The library's accurate exponential, operation by operation."""
    z = np.maximum(np.asarray(z, f32), f32(-88))
    t = fma(z, f32(1.442695022), f32(12582912))
    n = t - f32(12582912)
    r = fma(n, f32(-0.693145751953125), z)
    r = fma(n, f32(-1.428606765e-06), r)
    p = fma(f32(0.0013843592), r, f32(0.008374209))
    for c in (0.041668005, 0.1666643, 0.49999994, 1.0, 1.0):
        p = fma(p, r, f32(c))
    return p * np.exp2(n.astype(np.float64)).astype(f32)


def test_exp1_is_within_three_quarters_of_a_unit():
    worst = 0.0
    for e in range(-24, 7):
        z = -np.ldexp(1 + np.arange(0, 2 ** 23, 37) * U, e).astype(f32)
        z = z[z >= -86.5]
        worst = max(worst, np.abs(exp1(z) / np.exp(z.astype(np.float64)) - 1).max())
    assert worst <= 0.75 * U


def replay(row, per, off):
    """ln d below the row's maximum as the kernels form it: 256 threads, tiles of `per` columns a
    thread, one run; ex2.approx off by `off` units everywhere."""
    def ex2(t):
        return (np.exp2(t.astype(np.float64)) * (1 + off * U)).astype(f32)

    L, T = f32(1.442695022), 256
    tiles = -(-len(row) // (T * per))
    x = np.full(tiles * T * per, -np.inf, f32)
    x[:len(row)] = row
    x = x.reshape(tiles, per // 4, T, 4)
    m, d, lost, largest = (np.full(T, v, f32) for v in (-np.inf, 0, 0, -np.inf))
    for tile in x:
        tile = tile.transpose(1, 0, 2).reshape(T, per)
        top = tile.max(1)
        up = top > m + f32(1)
        f = np.where(up, np.where(top == m, f32(1), exp1(np.where(up, m - top, 0))), f32(1))
        d, lost, m = (d * f).astype(f32), (lost * f).astype(f32), np.where(up, top, m)
        largest = np.maximum(largest, top)
        live = m > -np.inf
        ref = np.where(live, m, 0).astype(f32)
        c = (ref * L).astype(f32)
        w = ex2(fma(tile, L, -c[:, None]))
        part = np.zeros((T, 4), f32)
        for i in range(0, per, 4):
            part = (part + w[:, i:i + 4]).astype(f32)
        s = (part[:, 0] + part[:, 1]) + (part[:, 2] + part[:, 3])
        s = np.where(live, s * ex2(fma(ref, -L, c)), 0).astype(f32)
        new = (d + s).astype(f32)
        lost = (lost + np.where(d >= s, (d - new) + s, (s - new) + d)).astype(f32)
        d = new

    def tree(v):
        while v.shape[1] > 1:
            h = v.shape[1] // 2
            v = (v[:, :h] + v[:, h:]).astype(f32)
        return v[:, 0]

    warps = largest.reshape(8, 32).max(1)
    gap = np.repeat(warps, 32)
    gone = ~(m > -np.inf)
    mine = np.where(gone, 0, (d + lost) * exp1(np.where(gone, 0, m - gap))).astype(f32)
    dw = tree(mine.reshape(8, 32))
    top = warps.max()
    dead = ~(warps > -np.inf)
    total = tree(np.where(dead, 0, dw * exp1(np.where(dead, 0, warps - top))).astype(f32)[None])[0]
    return math.log(float(total))


def rows():
    rng = np.random.default_rng(1)
    yield "normal", (rng.standard_normal(128256) * 2.5).astype(f32)
    yield "wide", (rng.standard_normal(128256) * 12).astype(f32)
    yield "far from 0", (rng.standard_normal(50257) * 3 + 9e4).astype(f32)
    yield "far beyond 2^24", np.float64(2 ** 27) - 16 * rng.integers(0, 9, 50257)
    yield "all but equal", (rng.random(300000) * 1e-3).astype(f32)
    # nearly all the mass 17 below the maximum
    low = np.full(2 ** 20, -17.0, f32) + (rng.random(2 ** 20) * 0.1).astype(f32)
    low[12345] = 0
    yield "low mass", low
    for r in (1.32122802734375, 1.72967529296875, 1.000123):
        for k in (3, 5, 6, 8):
            x = np.zeros((200, 4, 256, 4), f32)
            x -= (rng.random(x.shape) * 0.3).astype(f32)
            for j in range(k):
                x[-k + j] = -60
                x[-k + j, 0, :, 0] = f32((j + 1) * r)
            yield f"{k} tiles that rise by {r}", x.reshape(-1)


def test_replayed_sums_stay_within_the_bound(bound):
    for name, row in rows():
        row = row.astype(f32)
        far = 5.5 if np.abs(row).max() >= 2 ** 24 else 0
        top = float(row.max())
        want = math.log(math.fsum(np.exp(row.astype(np.float64) - top)))
        share = -(-len(row) // 4096) * 16
        for off in (-2, 0, 2):
            err = abs(replay(row, 16, off) - want) / U
            # (the last logarithm is not replayed)
            assert err <= bound(len(row), share) + far - 0.5, (name, off, err)
