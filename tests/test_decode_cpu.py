"""The paged cache's operators and beam search's selection on a machine without a GPU: refusals of
their C entry points and tensor functions, and the float64 oracle against what does not depend on
it.  No kernel is launched here."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import decode as ref

F32, BF16 = 0, 1
OK, NULL, SHAPE, DTYPE, KERR, ALIAS, CUDA, TIMEOUT, PATH, ALIGN, VALUE = range(11)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def st():
    import __graft_entry__
    __graft_entry__._builder().build()
    import softmax_topk_gb300
    return softmax_topk_gb300


def at(i):  # disjoint fake device addresses, 16-byte aligned
    return 0x10000000 * (i + 1)


CACHE = dict(k=at(0), v=at(1), table=at(2), lengths=at(3), pages=9, seqs=6, width=4, kv_heads=2,
             page_size=16, head_dim=64)
POINTERS = ("k", "v", "table", "lengths")


def cache(st, **kw):
    return ctypes.byref(st.PagedCache(**{n: kw.get(n, CACHE[n]) for n in CACHE}))


def refuses_bad_caches(st, call):
    """What every entry point of the cache checks; call(cache) gives its status."""
    assert call(None) == NULL
    for bad in (dict(pages=0), dict(seqs=-1), dict(width=0), dict(kv_heads=0), dict(page_size=0),
                dict(head_dim=96), dict(pages=2 ** 27), dict(width=2 ** 28), dict(pages=2 ** 40),
                dict(width=2 ** 40), dict(kv_heads=2 ** 31 - 1)):
        assert call(cache(st, **bad)) == SHAPE, bad
    for name in POINTERS:
        assert call(cache(st, **{name: None})) == NULL, name
        step = 8 if name in "kv" else 2
        assert call(cache(st, **{name: CACHE[name] + step})) == ALIGN, name


def test_heads_and_pages_that_32_bits_cannot_count(st):
    """A token's heads and a page's rows are counted in 16-byte pieces of 32 bits."""
    def append(rows, **kw):
        return st._lib.os_paged_append(cache(st, pages=1, seqs=1, **kw), at(10), rows, at(11),
                                       rows, None, 0, None, None, None, 1, 0, 0, 0, None)

    def reorder(**kw):
        return st._lib.os_paged_reorder(cache(st, pages=1, seqs=0, **kw), None, None, None, 1, 1,
                                        None)

    many = dict(page_size=1, head_dim=128)
    assert append(2 ** 28, kv_heads=2 ** 20 + 1, **many) == SHAPE
    assert reorder(kv_heads=2 ** 20 + 1, **many) == SHAPE and reorder(kv_heads=2 ** 20, **many) == OK
    long = dict(kv_heads=1, width=1)
    assert append(64, page_size=2 ** 24 + 1, **long) == SHAPE
    assert reorder(page_size=2 ** 24 + 1, **long) == SHAPE
    assert reorder(page_size=2 ** 24, **long) == OK


def test_append_refusals(st):
    base = dict(k=at(10), k_stride=128, v=at(11), v_stride=128, q=at(12), q_stride=256,
                q_out=at(13), starts=at(14), inv_freq=at(15), tokens=20, q_heads=4, rot=64,
                interleaved=0)

    def call(c=None, **kw):
        p = {**base, **kw}
        return st._lib.os_paged_append(cache(st) if c is None else c, *[p[n] for n in base], None)

    def call_cache(c):
        return st._lib.os_paged_append(c, *base.values(), None)

    refuses_bad_caches(st, call_cache)
    assert call(tokens=-1) == SHAPE and call(tokens=2 ** 31) == SHAPE
    assert call(starts=None) == SHAPE  # 20 tokens, 6 sequences
    for name in ("k_stride", "v_stride"):
        for bad in (127, 120, 132, -128, 2 ** 62):
            assert call(**{name: bad}) == SHAPE, (name, bad)
    assert call(q_stride=248) == SHAPE and call(q_stride=260) == SHAPE
    for rot in (0, 8, 24, 80, -16):
        assert call(rot=rot) == SHAPE, rot
    assert call(interleaved=2) == VALUE
    assert call(q_heads=1) == SHAPE  # fewer than the cache has
    for name in ("k", "v", "q_out"):
        assert call(**{name: None}) == NULL, name
    assert call(q=None) == NULL  # q_out without q
    for name in ("k", "v", "q", "q_out"):
        assert call(**{name: base[name] + 8}) == ALIGN, name
    for name in ("starts", "inv_freq"):
        assert call(**{name: base[name] + 2}) == ALIGN, name
    for other in (at(0), at(1), at(2), at(3), at(10), at(11), at(12), at(14), at(15)):
        assert call(q_out=other) == ALIAS, other
    for name in ("k", "v", "q", "starts", "inv_freq"):
        assert call(**{name: CACHE["k"]}) == ALIAS and call(**{name: CACHE["v"]}) == ALIAS, name
    assert call_cache(cache(st, v=CACHE["k"])) == ALIAS
    assert call_cache(cache(st, table=CACHE["k"])) == ALIAS
    assert call(tokens=0, k=None) == OK
    assert call(cache(st, seqs=0, k=None)) == OK
    assert call(cache(st, seqs=0), starts=None, tokens=0) == OK


def test_attention_refusals(st):
    base = dict(q=at(10), q_stride=256, out=at(11), lse=at(12), workspace=at(13), q_heads=4,
                scale=0.125)

    def call(c=None, **kw):
        p = {**base, **kw}
        return st._lib.os_paged_attention(cache(st) if c is None else c, *p.values(), None)

    refuses_bad_caches(st, lambda c: st._lib.os_paged_attention(c, *base.values(), None))
    for bad in (0, 1, 3, 5, -4, 2 ** 31 - 2):
        assert call(q_heads=bad) == SHAPE, bad
    for bad in (248, 260, -256):
        assert call(q_stride=bad) == SHAPE, bad
    for scale in (0.0, -1.0, INF, NAN):
        assert call(scale=scale) == VALUE
    for name in ("q", "out", "workspace"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: base[name] + 8}) == ALIGN, name
    assert call(lse=base["lse"] + 2) == ALIGN
    for name in ("out", "lse"):
        for other in (at(0), at(1), at(2), at(3), at(10)):
            assert call(**{name: other}) == ALIAS, (name, other)
    assert call(lse=base["out"]) == ALIAS
    assert call(cache(st, seqs=0, k=None), q=None) == OK
    assert st._lib.os_paged_attention_workspace(None) == NULL


def test_reorder_refusals(st):
    base = dict(parents=at(10), out_table=at(11), out_lengths=at(12), beams=3, layers=2)

    def call(c=None, **kw):
        p = {**base, **kw}
        return st._lib.os_paged_reorder(cache(st) if c is None else c, *p.values(), None)

    refuses_bad_caches(st, lambda c: st._lib.os_paged_reorder(c, *base.values(), None))
    for bad in (0, -3, 4, 7):
        assert call(beams=bad) == SHAPE, bad
    assert call(layers=0) == SHAPE and call(layers=2 ** 31 - 1) == SHAPE
    for name in ("parents", "out_table"):
        assert call(**{name: None}) == NULL, name
    for name in ("parents", "out_table", "out_lengths"):
        assert call(**{name: base[name] + 2}) == ALIGN, name
    for name in ("out_table", "out_lengths"):
        for other in (at(0), at(1), at(2), at(3), at(10)):
            assert call(**{name: other}) == ALIAS, (name, other)
    assert call(out_lengths=base["out_table"]) == ALIAS
    # a second layer that reaches into v
    layer = 9 * 2 * 16 * 64 * 2
    assert call(cache(st, v=CACHE["k"] + layer), layers=1, parents=None) == NULL
    assert call(cache(st, v=CACHE["k"] + layer)) == ALIAS
    assert call(cache(st, seqs=0, k=None), parents=None) == OK


def test_select_refusals(st):
    base = dict(x=at(0), scores=at(1), ended=at(2), out=at(3), parents=at(4), tokens=at(5),
                workspace=at(6), groups=2, beams=3, cols=100, K=4, pad=7, dtype=F32)

    def call(**kw):
        return st._lib.os_beam_select(*{**base, **kw}.values(), None)

    assert call(dtype=2) == DTYPE
    assert call(groups=-1) == SHAPE and call(groups=2 ** 26) == SHAPE
    assert call(beams=0) == SHAPE and call(beams=65) == SHAPE
    assert call(cols=0) == SHAPE and call(cols=2 ** 31) == SHAPE
    assert call(K=0) == KERR and call(K=65) == KERR
    assert call(pad=-1) == VALUE and call(pad=100) == VALUE
    for name in ("x", "scores", "out", "parents", "tokens", "workspace"):
        assert call(**{name: None}) == NULL, name
    for name in ("x", "scores", "out", "parents", "tokens"):
        assert call(**{name: base[name] + 2}) == ALIGN, name
    assert call(workspace=base["workspace"] + 8) == ALIGN
    for name in ("out", "parents", "tokens"):
        for other in ("x", "scores", "ended"):
            assert call(**{name: base[other]}) == ALIAS, (name, other)
    assert call(out=base["parents"]) == ALIAS and call(tokens=base["parents"]) == ALIAS
    assert call(groups=0, x=None) == OK
    n = ctypes.c_int64()
    f = st._lib.os_beam_select_workspace
    assert f(2, 0, 100, 4, F32, ctypes.byref(n)) == SHAPE and f(2, 3, 100, 4, F32, None) == NULL
    assert f(2, 3, 100, 65, F32, ctypes.byref(n)) == KERR


def test_tensor_functions_refuse(st):
    pool, table = torch.zeros(3, 2, 16, 64).bfloat16(), torch.zeros(2, 4).int()
    k, lengths = torch.zeros(2, 2, 64).bfloat16(), torch.ones(2).int()
    for call in (lambda: st.paged_append(pool, pool, table, lengths, k, k),
                 lambda: st.paged_attention(k, pool, pool, table, lengths),
                 lambda: st.paged_reorder(pool, pool, table, lengths, table[:1, :2], table),
                 lambda: st.beam_select(torch.zeros(6, 10), torch.zeros(2, 3))):
        with pytest.raises(ValueError):  # no CUDA tensors
            call()


# ------------------------------------------------------------------ the oracle
def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 3, 64))
    f = 10000.0 ** (-np.arange(16) / 16)
    for way in (False, True):
        a, b = ref.rotate(q, 7, f, way), ref.rotate(k, 4, f, way)
        assert np.allclose((a ** 2).sum(1), (q ** 2).sum(1))
        assert np.array_equal(a[:, 32:], q[:, 32:])
        later = (ref.rotate(q, 1007, f, way) * ref.rotate(k, 1004, f, way)).sum(1)
        assert np.allclose((a * b).sum(1), later)
    assert np.array_equal(ref.rotate(q, 0, f, False), q)


def test_attention_of_a_cache_is_attention():
    """Over a cache filled token by token: the last row of causal attention."""
    import oracle
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 1, 21, 2, 64))
    pools = np.full((2, 8, 2, 4, 64), np.nan)
    table = np.array([[3, 0, 7, 1, 5, 2, -1]])
    for t in range(21):
        pools[0], pools[1], _ = ref.append(*pools, table, [t + 1], k[:, t], v[:, t])
    out, lse, _ = ref.attention(q[:, 20], *pools, table, [21], 0.125)
    want, want_lse = oracle.attention(*(a[0].transpose(1, 0, 2) for a in (q, k, v)), 0.125, True)
    assert np.allclose(out[0], want[:, 20]) and np.allclose(lse[0], want_lse[:, 20])
    # a page that is not there hides its keys; no keys, no output
    table[0, 2] = 8
    out, lse, _ = ref.attention(q[:, 20], *pools, table, [21], 0.125)
    keep = [p for p in range(21) if p // 4 != 2]
    s = 0.125 * np.einsum("hd,nhd->hn", q[0, 20], k[0, keep])
    assert np.allclose(lse[0], np.log(np.exp(s).sum(1)))
    out, lse, _ = ref.attention(q[:, 20], *pools, table, [0], 0.125)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_append_all_at_once_is_append_one_by_one():
    rng = np.random.default_rng(2)
    f = 10000.0 ** (-np.arange(8) / 8)
    k, v, q = rng.standard_normal((3, 11, 2, 64))
    table = rng.permutation(12).reshape(3, 4)
    pool = rng.standard_normal((12, 2, 3, 64))
    starts, lengths = [0, 4, 4, 9], [6, 5, 5]
    a = ref.append(pool, pool, table, lengths, k, v, q, starts, f)
    b = [pool, pool]
    for seq in (0, 2):
        for i, t in enumerate(range(starts[seq], starts[seq + 1])):
            one = [lengths[s] - (starts[s + 1] - starts[s]) + i + 1 if s == seq else 0
                   for s in range(3)]
            rows = np.zeros((3, 2, 64)) + k[t], np.zeros((3, 2, 64)) + v[t]
            b = ref.append(*b[:2], table, one, *rows, None, None, f)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    assert (a[2][9:] == 0).all()  # behind the last sequence


def test_selection_by_brute_force():
    rng = np.random.default_rng(3)
    x = rng.integers(-3, 4, (6, 9)).astype(float)
    x[rng.random(x.shape) < 0.2] = -np.inf
    scores = np.array([[-1.0, -2.0, -np.inf], [-0.5, -0.5, np.nan]])
    ended = [[False, True, False], [False, False, False]]
    values, parents, tokens = ref.beam_select(x, scores, 12, ended, pad=4)
    for g in range(2):
        every = []
        for i in range(3):
            if not scores[g, i] > -np.inf:
                continue
            if ended[g][i]:
                every.append((scores[g, i], i, 4))
                continue
            row = x[3 * g + i]
            lse = np.log(np.exp(row[row > -np.inf]).sum())
            every += [(scores[g, i] + row[c] - lse, i, c) for c in range(9) if row[c] > -np.inf]
        every.sort(key=lambda e: (-round(e[0], 12), e[1], e[2]))
        n = min(12, len(every))
        assert np.allclose(values[g, :n], [e[0] for e in every[:n]])
        assert [*zip(parents[g, :n], tokens[g, :n])] == [e[1:] for e in every[:n]]
        assert (parents[g, n:] == -1).all() and (values[g, n:] == -np.inf).all()


def test_reorder_keeps_histories():
    """Whatever the parents, a sequence's tokens behind the reordering are its parent's."""
    rng = np.random.default_rng(4)
    pool = rng.standard_normal((2, 40, 1, 4, 64))
    table, new = rng.permutation(40)[:36].reshape(2, 6, 3)
    lengths, parents = [9, 9, 9, 4, 4, 4], [[2, 2, 0], [1, -1, 1]]
    k, _, out, out_lengths = ref.reorder(pool, pool, table, lengths, parents, new, 4)
    for j, p in enumerate((2, 2, 0, 4, None, 4)):
        if p is None:
            assert out_lengths[j] == 0 and np.array_equal(out[j], new[j])
            continue
        assert out_lengths[j] == lengths[p]
        for pos in range(lengths[p]):
            was, now = (tab[pos // 4] for tab in (table[p], out[j]))
            assert np.array_equal(k[:, now, :, pos % 4], pool[:, was, :, pos % 4])
