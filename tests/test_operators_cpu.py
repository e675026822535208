"""The attention gradient, the router and the sampler on a machine without a GPU: refusals of
their C entry points and tensor functions, and the float64 oracle against what does not depend
on it (differences, brute force, closed forms).  No kernel is launched here."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import operators as ref

F32, BF16 = 0, 1
OK, NULL, SHAPE, DTYPE, KERR, ALIAS, CUDA, TIMEOUT, PATH, ALIGN, VALUE = range(11)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def st():
    import __graft_entry__
    __graft_entry__._builder().build()
    import softmax_topk_gb300
    return softmax_topk_gb300


# ------------------------------------------------------------------ refusals
def at(i):  # disjoint fake device addresses, 16-byte aligned
    return 0x10000000 * (i + 1)


def test_attention_bwd_refusals(st):
    names = ["q", "k", "v", "o", "lse", "dout", "dlse", "dq", "dk", "dv", "delta"]
    base = {name: at(i) for i, name in enumerate(names)}

    def call(bh=2, n=128, d=64, scale=0.125, causal=0, **kw):
        p = {**base, **kw}
        return st._lib.os_attention_bwd(*[p[a] for a in names], bh, n, d, scale, causal, None)

    assert call(bh=-1) == SHAPE and call(n=-1) == SHAPE and call(d=96) == SHAPE
    assert call(n=2 ** 31) == SHAPE and call(bh=2 ** 31, n=4096) == SHAPE
    for scale in (0.0, -1.0, INF, NAN):
        assert call(scale=scale) == VALUE
    assert call(causal=2) == VALUE
    for name in names:
        if name != "dlse":
            assert call(**{name: None}) == NULL, name
        step = 2 if name in ("lse", "dlse", "delta") else 8
        assert call(**{name: base[name] + step}) == ALIGN, name
    for out in ("dq", "dk", "dv", "delta"):
        for name in names:
            if name != out:
                assert call(**{out: base[name]}) == ALIAS, (out, name)
    assert call(bh=0, q=None, dq=None) == OK and call(n=0, q=None) == OK


def test_route_refusals(st):
    base = dict(x=at(0), bias=at(1), weights=at(2), idx=at(3), rows=4, experts=64, K=4, groups=4,
                topk_groups=2, group_top=2, score=1, renorm=1, scale=1.0, dtype=F32)

    def call(**kw):
        p = {**base, **kw}
        return st._lib.os_route_topk(*[p[a] for a in base], None)

    assert call(rows=-1) == SHAPE and call(experts=0) == SHAPE and call(experts=1028) == SHAPE
    assert call(rows=2 ** 60) == SHAPE
    assert call(groups=0) == SHAPE and call(groups=5) == SHAPE and call(groups=64) == SHAPE
    assert call(topk_groups=0) == SHAPE and call(topk_groups=5) == SHAPE
    assert call(group_top=0) == SHAPE and call(group_top=3) == SHAPE
    assert call(experts=4, groups=4, K=1) == SHAPE  # a second-best of one expert
    assert call(K=0) == KERR and call(K=33) == KERR and call(K=17, topk_groups=1) == KERR
    assert call(score=2) == VALUE and call(renorm=2) == VALUE
    for scale in (NAN, INF, -INF):
        assert call(scale=scale) == VALUE
    assert call(dtype=2) == DTYPE
    for name in ("x", "weights", "idx"):
        assert call(**{name: None}) == NULL
    for name in ("x", "bias", "weights", "idx"):
        assert call(**{name: base[name] + 2}) == ALIGN, name
    for out, name in (("weights", "x"), ("weights", "bias"), ("weights", "idx"), ("idx", "x"),
                      ("idx", "bias")):
        assert call(**{out: base[name]}) == ALIAS, (out, name)
    assert call(rows=0, x=None, weights=None) == OK


def test_route_bwd_refusals(st):
    base = dict(x=at(0), idx=at(1), dweights=at(2), dx=at(3), rows=4, experts=60, K=4, score=0,
                renorm=0, scale=1.0, dtype=BF16)

    def call(**kw):
        p = {**base, **kw}
        return st._lib.os_route_bwd(*[p[a] for a in base], None)

    assert call(rows=-1) == SHAPE and call(experts=0) == SHAPE and call(experts=1025) == SHAPE
    assert call(K=0) == KERR and call(K=33) == KERR and call(K=5, experts=4) == KERR
    assert call(score=-1) == VALUE and call(renorm=3) == VALUE and call(scale=NAN) == VALUE
    assert call(dtype=3) == DTYPE
    for name in ("x", "idx", "dweights", "dx"):
        assert call(**{name: None}) == NULL
        assert call(**{name: base[name] + 1}) == ALIGN
    for name in ("x", "idx", "dweights"):
        assert call(dx=base[name]) == ALIAS
    assert call(rows=0, x=None) == OK


def test_sample_refusals(st):
    def call(x=at(0), u=at(1), out=at(2), prob=at(3), rows=4, cols=100, dtype=F32, null=False, **kw):
        s = st.Sampling(temperature_all=1.0, top_p_all=1.0)
        for name, v in kw.items():
            setattr(s, name, v)
        return st._lib.os_sample(x, u, None if null else ctypes.byref(s), out, prob, rows, cols,
                                 dtype, None)

    assert call(dtype=2) == DTYPE
    assert call(rows=-1) == SHAPE and call(cols=0) == SHAPE and call(cols=2 ** 31) == SHAPE
    assert call(null=True) == NULL
    for kw in ({"temperature_all": -1.0}, {"temperature_all": NAN}, {"temperature_all": INF},
               {"top_k_all": -1}, {"top_p_all": -0.1}, {"top_p_all": 1.5}, {"top_p_all": NAN},
               {"min_p_all": -0.1}, {"min_p_all": 2.0}, {"min_p_all": NAN}):
        assert call(**kw) == VALUE, kw
    assert call(x=None) == NULL and call(u=None) == NULL and call(out=None) == NULL
    assert call(x=at(0) + 2) == ALIGN and call(u=at(1) + 1) == ALIGN
    assert call(out=at(2) + 2) == ALIGN and call(prob=at(3) + 2) == ALIGN
    for name in ("temperature", "top_k", "top_p", "min_p"):
        assert call(**{name: at(5) + 2}) == ALIGN
        assert call(**{name: at(2)}) == ALIAS and call(**{name: at(3)}) == ALIAS
    assert call(out=at(0) + 16) == ALIAS and call(prob=at(0)) == ALIAS
    assert call(out=at(1)) == ALIAS and call(prob=at(2)) == ALIAS
    assert call(rows=0, x=None, u=None, out=None) == OK


def test_tensor_functions_refuse_host_tensors(st):
    import torch
    x = torch.zeros(2, 8)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        st.attention_backward(q, q, q, q, torch.zeros(1, 4), q)
    with pytest.raises(ValueError):
        st.route(x, 2)
    with pytest.raises(ValueError):
        st.route_backward(x, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))
    with pytest.raises(ValueError):
        st.sample(x, torch.zeros(2))


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("causal", [False, True])
def test_oracle_attention_gradient_by_differences(causal):
    rng = np.random.default_rng(1)
    q, k, v, do = (rng.standard_normal((2, 9, 5)) for _ in range(4))
    dl = rng.standard_normal((2, 9))
    o, lse = oracle.attention(q, k, v, 0.4, causal)
    grads = ref.attention_backward(q, k, v, o, lse, do, 0.4, causal, dl)
    args = [q, k, v]

    def loss(a):
        oo, ll = oracle.attention(*a, 0.4, causal)
        return (oo * do).sum() + (ll * dl).sum()

    for i in range(3):
        way = rng.standard_normal(q.shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-5 * way, args[i] - 1e-5 * way
        numeric = (loss(up) - loss(down)) / 2e-5
        assert abs((grads[i] * way).sum() - numeric) <= 1e-7 * (1 + abs(numeric))


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_oracle_route_gradient_by_differences(score, renorm):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, 12))
    w, idx = ref.route(x, 3, score=score, renorm=renorm, scale=1.7)
    dw = rng.standard_normal(w.shape)
    dx = ref.route_backward(x, idx, dw, score=score, renorm=renorm, scale=1.7)
    way = rng.standard_normal(x.shape)

    def loss(a):
        s = ref.route_scores(a, score)
        t = np.take_along_axis(s, idx.astype(np.int64), 1)
        if renorm:
            t = t / t.sum(1, keepdims=True)
        return (1.7 * t * dw).sum()

    numeric = (loss(x + 1e-6 * way) - loss(x - 1e-6 * way)) / 2e-6
    assert abs((dx * way).sum() - numeric) <= 1e-7 * (1 + abs(numeric))


def test_oracle_route_closed_forms():
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    w, idx = ref.route(x, 2, renorm=False)
    assert idx.tolist() == [[2, 1]] and np.allclose(w, [[0.5, 0.25]])
    w, idx = ref.route(x, 2, bias=[1, 0, 0, 1])
    assert idx.tolist() == [[0, 3]] and np.allclose(w, [[0.5, 0.5]])
    w, idx = ref.route(x, 2, groups=2, topk_groups=1, group_top=2)  # {1, 2} against {4, 1}
    assert idx.tolist() == [[2, 3]] and np.allclose(w, [[0.8, 0.2]])
    w, idx = ref.route(np.full((1, 4), -np.inf), 2)
    assert idx.tolist() == [[0, 1]] and not w.any()


def test_oracle_sample_frequencies_and_filters():
    x = np.log(np.array([0.5, 0.25, 0.125, 0.125]))
    n = 1 << 12
    u = (np.arange(n) + 0.5) / n
    counts = np.bincount([ref.sample_row(x, t)[0] for t in u], minlength=4) / n
    assert np.abs(counts - [0.5, 0.25, 0.125, 0.125]).max() < 2 / n
    assert ref.sample_row(x, 0.9, top_k=3)[2].tolist() == [0, 1, 2]      # the tie goes to the lower
    assert ref.sample_row(x, 0.9, top_p=0.6)[2].tolist() == [0, 1]
    assert ref.sample_row(x, 0.9, min_p=0.3)[2].tolist() == [0, 1]
    assert ref.sample_row(x, 0.9, top_k=3, top_p=0.8)[2].tolist() == [0, 1]  # of 0.875
    assert ref.sample_row(x, 0.9, temperature=0)[0] == 0
    assert ref.sample_row(np.full(4, -np.inf), 0.5)[0] == -1
