"""The attention gradient on the GPU against the float64 oracle, element by element.

Tolerance, from the kernel's arithmetic (u = 2^-24 the fp32 and h = 2^-8 the bf16 half step):
a score is an fp32 sum of d exact products, |ds| <= d 2u max_ij sum |q_ic k_jc|, and P carries
e_p = scale |ds| + (|s| + |L| + 8) 2u relative.  dP and delta are fp32 sums of d products.  P and
dS are rounded to bf16 (h relative) as operands, their products are summed in fp32 (n terms) and
the result is rounded to bf16 (h relative).  So
  |d dV_j|  <= (e_p + h + n u) sum_i P_ij |dO_i| + h |dV_j|,
  |d dS_ij| <= P_ij (|dP - delta| (e_p + h + 2u) + d 2u (sum |dO v| + sum |dO o|) + 2u |dL|),
  |d dQ_i|  <= scale sum_j (|d dS_ij| + n u |dS_ij|) |k_j| + h |dQ_i|, and dK likewise.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import operators as ref

pytestmark = pytest.mark.gpu
U, H = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def _f64(t):
    return t.double().cpu().numpy()


def bounds(q, k, v, o, lse, do, scale, causal, dlse=None):
    """The oracle's gradients and the bound of each element's error."""
    want = ref.attention_backward(q, k, v, o, lse, do, scale, causal, dlse)
    p = ref.attention_probs(q, k, lse, scale, causal)
    q, k, v, o, do, lse = (_f64(t) for t in (q, k, v, o, do, lse))
    n, d = q.shape[1:]
    most = np.einsum("bid,bjd->bij", np.abs(q), np.abs(k)).max()
    large = scale * most + np.abs(lse[np.isfinite(lse)]).max(initial=0) + 8
    e_p = scale * d * 2 * U * most + large * 2 * U
    delta = (o * do).sum(-1)
    dl = 0.0 if dlse is None else _f64(dlse)
    dp = np.einsum("bid,bjd->bij", do, v)
    diff = np.abs(dp - (delta - dl)[:, :, None])
    rough = d * 2 * U * (np.einsum("bid,bjd->bij", np.abs(do), np.abs(v)) +
                         (np.abs(o) * np.abs(do)).sum(-1)[:, :, None]) + \
        2 * U * np.broadcast_to(np.abs(dl), delta.shape)[:, :, None]
    ds_err = p * (diff * (e_p + H + 2 * U) + rough) + n * U * p * diff
    dq_err = scale * np.einsum("bij,bjd->bid", ds_err, np.abs(k)) + H * np.abs(want[0])
    dk_err = scale * np.einsum("bij,bid->bjd", ds_err, np.abs(q)) + H * np.abs(want[1])
    dv_err = (e_p + H + n * U) * np.einsum("bij,bid->bjd", p, np.abs(do)) + H * np.abs(want[2])
    return want, [e + 1e-30 for e in (dq_err, dk_err, dv_err)]


def check(got, want, err, label=""):
    for name, g, w, e in zip(("dq", "dk", "dv"), got, want, err):
        g = _f64(g)
        assert np.isfinite(g).all(), f"{label} {name}: not finite"
        bad = np.abs(g - w) > e
        assert not bad.any(), f"{label} {name}: {bad.sum()} of {bad.size} off, worst " \
                              f"{(np.abs(g - w) / e).max():.2f} of the bound at {np.argwhere(bad)[0]}"


def make(bh, n, d, seed, qk=1.0, dv=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    q, k, v, do = (torch.randn(bh, n, d, generator=g, device="cuda") for _ in range(4))
    return (q * qk).bfloat16(), (k * qk).bfloat16(), v.bfloat16(), (do * dv).bfloat16()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 7, 64, 127, 128, 129, 300, 513])
def test_matches_oracle(st, n, d, causal):
    q, k, v, do = make(3, n, d, seed=n * 10 + d)
    o, lse = st.attention(q, k, v, causal=causal)
    got = st.attention_backward(q, k, v, o, lse, do, causal=causal)
    torch.cuda.synchronize()
    st.os_device_status(None)
    want, err = bounds(q, k, v, o, lse, do, 1 / math.sqrt(d), causal)
    check(got, want, err, f"n={n} d={d} causal={causal}")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_more_items_than_sms(st, d, causal):
    """Persistent CTAs walk several items each: 200 slices of two tiles."""
    q, k, v, do = make(200, 190, d, seed=5)
    o, lse = st.attention(q, k, v, causal=causal)
    got = st.attention_backward(q, k, v, o, lse, do, causal=causal)
    want, err = bounds(q, k, v, o, lse, do, 1 / math.sqrt(d), causal)
    check(got, want, err)


@pytest.mark.parametrize("causal", [False, True])
def test_gradient_of_the_logsumexp(st, causal):
    q, k, v, do = make(2, 200, 64, seed=11)
    o, lse = st.attention(q, k, v, causal=causal, scale=0.3)
    dlse = torch.randn_like(lse) * 3
    got = st.attention_backward(q, k, v, o, lse, do, causal=causal, scale=0.3, dlse=dlse)
    want, err = bounds(q, k, v, o, lse, do, 0.3, causal, dlse)
    check(got, want, err)


@pytest.mark.parametrize("d", [64, 128])
def test_peaked_rows(st, d):
    """Scores tens apart: nearly one-hot rows, P down to 0."""
    q, k, v, do = make(2, 260, d, seed=12, qk=3.0)
    o, lse = st.attention(q, k, v, causal=True)
    got = st.attention_backward(q, k, v, o, lse, do, causal=True)
    want, err = bounds(q, k, v, o, lse, do, 1 / math.sqrt(d), True)
    check(got, want, err)


def test_rows_without_keys(st):
    """L = -inf: the query takes no part and its dQ is 0."""
    q, k, v, do = make(2, 150, 64, seed=13)
    o, lse = st.attention(q, k, v)
    lse[0, 3] = lse[1, 149] = float("-inf")
    got = st.attention_backward(q, k, v, o, lse, do)
    want, err = bounds(q, k, v, o, lse, do, 0.125, False)
    check(got, want, err)
    assert not got[0][0, 3].any() and not got[0][1, 149].any()


def test_against_differences(st):
    """The directional derivative of sum dO.O + dL.L by central differences of the float64
    forward, against the gradients' products with the direction."""
    q, k, v, do = make(2, 40, 64, seed=14)
    o, lse = st.attention(q, k, v, causal=True)
    dlse = torch.randn_like(lse)
    got = st.attention_backward(q, k, v, o, lse, do, causal=True, dlse=dlse)
    _, err = bounds(q, k, v, o, lse, do, 0.125, True, dlse)
    rng = np.random.default_rng(0)
    args = [_f64(t) for t in (q, k, v)]
    ddo, ddl = _f64(do), _f64(dlse)

    def loss(a):
        oo, ll = oracle.attention(*a, None, True)
        return (oo * ddo).sum() + (ll * ddl).sum()

    # the kernel's delta takes the forward's bf16 O: O off by up to 2 (2^-9 + 2^-8) of its row's
    # sum of P |v| moves delta_i, and with it dS_ij = P_ij (dP_ij - delta_i)
    p = ref.attention_probs(q, k, lse, 0.125, True)
    o_err = 4 * H * np.einsum("bij,bjd->bid", p, np.abs(args[2]))
    d_err = (np.abs(ddo) * o_err).sum(-1)
    ds_err = p * d_err[:, :, None]
    more = [0.125 * np.einsum("bij,bjd->bid", ds_err, np.abs(args[1])),
            0.125 * np.einsum("bij,bid->bjd", ds_err, np.abs(args[0])), 0.0]
    for i, name in enumerate(("dq", "dk", "dv")):
        way = rng.standard_normal(args[i].shape)
        h = 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * way, args[i] - h * way
        numeric = (loss(up) - loss(down)) / (2 * h)
        mine = (_f64(got[i]) * way).sum()
        tol = ((err[i] + more[i]) * np.abs(way)).sum() + 1e-6 * abs(numeric)
        assert abs(mine - numeric) <= tol, (name, mine, numeric, tol)


def test_same_bits_every_time_and_in_a_graph(st):
    q, k, v, do = make(5, 333, 128, seed=15)
    o, lse = st.attention(q, k, v, causal=True)
    first = [t.clone() for t in st.attention_backward(q, k, v, o, lse, do, causal=True)]
    outs = [torch.empty_like(q) for _ in range(3)]
    delta = torch.empty_like(lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.attention_backward(q, k, v, o, lse, do, causal=True, dq=outs[0], dk=outs[1],
                              dv=outs[2], delta=delta)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = st.attention_backward(q, k, v, o, lse, do, causal=True)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,causal", [(128, False), (64, True)])
def test_repeats_agree_at_size(st, d, causal):
    """Tiles that come late from memory, over and over: the same bits every time, no wait that
    gave up."""
    q, k, v, do = make(64, 4096, d, seed=18)
    o, lse = st.attention(q, k, v, causal=causal)
    first = [t.clone() for t in st.attention_backward(q, k, v, o, lse, do, causal=causal)]
    for _ in range(60):
        again = st.attention_backward(q, k, v, o, lse, do, causal=causal)
        for a, b in zip(first, again):
            assert torch.equal(a, b)
    st.os_device_status(None)


def test_writes_nothing_outside(st):
    """Outputs between guard rows that keep their pattern."""
    bh, n, d = 2, 131, 64
    q, k, v, do = make(bh, n, d, seed=16)
    o, lse = st.attention(q, k, v)
    size, guard = bh * n * d, 128 * d
    raw = [torch.full((size + 2 * guard,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    outs = [r[guard:guard + size].view(bh, n, d) for r in raw]
    wide = torch.full((bh * n + 256,), 7.0, device="cuda")
    delta = wide[128:128 + bh * n].view(bh, n)
    st.attention_backward(q, k, v, o, lse, do, dq=outs[0], dk=outs[1], dv=outs[2], delta=delta)
    torch.cuda.synchronize()
    for r in raw:
        assert (r[:guard] == 7).all() and (r[guard + size:] == 7).all()
    assert (wide[:128] == 7).all() and (wide[128 + bh * n:] == 7).all()
    want, err = bounds(q, k, v, o, lse, do, 0.125, False)
    check(outs, want, err)


@pytest.mark.parametrize("shape", [(0, 128, 64), (2, 0, 64)])
def test_empty(st, shape):
    q = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(shape[:-1], device="cuda")
    for t in st.attention_backward(q, q, q, q, lse, q):
        assert t.shape == shape


@pytest.mark.slow
@pytest.mark.parametrize("d,causal", [(128, False), (64, True)])
def test_full_size_rows(st, d, causal):
    """64 x 4096: two slices, whole, on the GPU in 64 bits (the oracle's formula)."""
    q, k, v, do = make(64, 4096, d, seed=17)
    o, lse = st.attention(q, k, v, causal=causal)
    got = st.attention_backward(q, k, v, o, lse, do, causal=causal)
    scale = 1 / math.sqrt(d)
    for s in (0, 63):
        a, b, c, e, f = (t[s].double() for t in (q, k, v, o, do))
        p = (a @ b.T * scale - lse[s].double()[:, None]).exp()
        if causal:
            p = p.tril()
        ds = p * (f @ c.T - (e * f).sum(-1, keepdim=True))
        want = (ds @ b * scale, ds.T @ a * scale, p.T @ f)
        size = (ds.abs() @ b.abs() * scale, ds.T.abs() @ a.abs() * scale, p.T @ f.abs())
        most = (a.abs() @ b.abs().T).max()
        rel = float(scale * d * 2 * U * most + (scale * most + 30) * 2 * U + H + 4096 * U)
        rough = d * 2 * U * p * (f.abs() @ c.abs().T + (e * f).abs().sum(-1, keepdim=True))
        extra = (rough @ b.abs() * scale, rough.T @ a.abs() * scale, 0.0)
        for name, g, w, z, x in zip(("dq", "dk", "dv"), got, want, size, extra):
            off = (g[s].double() - w).abs() - (rel * z + x + H * w.abs() + 1e-30)
            assert float(off.max()) <= 0, (name, s, float(off.max()))
