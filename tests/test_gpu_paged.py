"""The paged key-value cache on the GPU: append with rotation, attention of one new token, and the
reordering of states, against the float64 oracle.

Tolerances.  A result of a product or a rotation is rounded once to bf16, half a step: 2^-8 of the
value.  Attention's weights are fp32 exponentials of scores with an error of at most
(d + 8) 2^-24 sum |q_i k_i| scale (fp32 sums of exact products), as two bf16 numbers (2^-17): with
the scores here that stays below 2^-11 of the weighted sum of |v|.  A rotation's sine and cosine
are good to 2^-22 of a turn's 2 pi (angles) and 2^-23 (their own rounding), its two products and
their sum to 2^-23: 2^-19 of |x| + |y|."""
import numpy as np
import pytest
import torch

from oracle import decode as ref

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def np64(t):
    return t.detach().cpu().double().numpy()


class Pool:
    """A cache whose unused places hold what would show if it were used."""

    def __init__(self, lengths, kv_heads, page, d, seed=0, extra_width=0, junk=NAN, capacity=None):
        g = self.g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        lengths = torch.tensor(lengths, device="cuda")
        room = lengths.clamp(min=0) if capacity is None else torch.full_like(lengths, capacity)
        need = (room + page - 1) // page
        seqs, width = len(lengths), max(1, int(need.max())) + extra_width
        pages = int(need.sum()) + 2
        shape = (pages, kv_heads, page, d)
        self.k, self.v = (self.randn(*shape).bfloat16() for _ in range(2))
        ids = torch.rand(pages, generator=g, device="cuda").argsort().int()
        # what lies behind the lengths in the table: no page, or far outside the pool
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
        self.table[:, 1::2] = 2 ** 31 - 1
        first = 0
        used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
        for b, (n, length) in enumerate(zip(need.tolist(), lengths.tolist())):
            self.table[b, :n] = ids[first:first + n]
            slots = (torch.arange(n * page, device="cuda") < length).view(n, page)
            used[ids[first:first + n].long()] = slots
            first += n
        for pool in (self.k, self.v):
            pool.masked_fill_(~used[:, None, :, None], junk)
        self.lengths = lengths.int()

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")


# ------------------------------------------------------------------ attention
def check_attention(st, pool, q, scale=None, **kw):
    out, lse = st.paged_attention(q, pool.k, pool.v, pool.table, pool.lengths, scale=scale, **kw)
    s = q.shape[-1] ** -0.5 if scale is None else scale
    want, want_lse, weighted = ref.attention(q, pool.k.cpu(), pool.v.cpu(), pool.table,
                                             pool.lengths, s)
    err = np.abs(np64(out) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * weighted), float(err.max())
    got = np64(lse)
    gone = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got), gone)
    assert (np64(out)[gone] == 0).all()
    if (~gone).any():
        assert np.abs(got[~gone] - want_lse[~gone]).max() <= 2.0 ** -11
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [1, 3, 16, 20, 128])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (2, 4), (1, 8), (2, 11), (3, 16), (1, 40)])
def test_attention(st, d, page, kv_heads, group):
    lengths = [1, 0, 15, 16, 17, 33, 300, -5, 129]
    pool = Pool(lengths, kv_heads, page, d, seed=page + group, extra_width=1)
    check_attention(st, pool, 2 * pool.randn(len(lengths), kv_heads * group, d).bfloat16())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[1], [16], [48], [193], [5000], [40000], [1] * 500,
                                     [0] * 40, [0, 0, 7, 0, 20000, 0], [3000, 1, 1, 1, 1, 1, 1]])
def test_attention_split_over_the_gpu(st, d, lengths):
    """Units inside one warp's run, over warps, over many CTAs, and CTAs without any."""
    pool = Pool(lengths, 2, 16, d, seed=len(lengths))
    check_attention(st, pool, 2 * pool.randn(len(lengths), 6, d).bfloat16())


@pytest.mark.parametrize("seqs,kv_heads,group", [(75, 2, 2), (76, 2, 2), (151, 1, 16), (152, 1, 3),
                                                 (40, 1, 24), (3, 1, 40)])
def test_attention_about_as_many_units_as_ctas(st, seqs, kv_heads, group):
    """The join goes by units below one per SM (152 of them), and by CTAs from there on."""
    lengths = [(97 * i + 50) % 700 if i % 7 else 0 for i in range(seqs)]
    lengths[-1] = 4000
    pool = Pool(lengths, kv_heads, 16, 64, seed=seqs)
    check_attention(st, pool, 2 * pool.randn(seqs, kv_heads * group, 64).bfloat16())


def test_attention_more_sequences_than_threads(st):
    lengths = [(7 * i) % 40 for i in range(1500)]
    pool = Pool(lengths, 1, 8, 64)
    check_attention(st, pool, 2 * pool.randn(1500, 2, 64).bfloat16())


@pytest.mark.parametrize("junk", [INF, -INF, 3.3e38])
def test_attention_ignores_what_is_behind(st, junk):
    pool = Pool([5, 17, 64], 2, 16, 128, junk=junk)
    check_attention(st, pool, pool.randn(3, 4, 128).bfloat16())


def test_attention_pages_that_are_not_there(st):
    pool = Pool([100, 100, 40, 30], 2, 16, 64)
    pool.table[0, 2] = -1
    pool.table[1, 0] = pool.k.shape[0]
    pool.table[2, :] = -7
    pool.table[3, 1] = -2 ** 31
    check_attention(st, pool, pool.randn(4, 6, 64).bfloat16())


def test_attention_lengths_past_the_table(st):
    pool = Pool([48, 32], 1, 16, 64, capacity=48)
    pool.v[pool.table[1, 2].long()] = 0.5
    pool.k[pool.table[1, 2].long()] = 0.25
    pool.lengths[:] = torch.tensor([2 ** 31 - 1, 49])
    check_attention(st, pool, pool.randn(2, 3, 64).bfloat16())


def test_attention_longest(st):
    """A length of 2^31 - 2, all pages but the first and the last not there: those two are the
    same page, so that its keys count twice."""
    page, width = 662, 3243933  # their product is 2^31 - 2
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    k, v = (torch.randn(1, 1, page, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = table[0, -1] = 0
    q = torch.randn(1, 2, 64, generator=g, device="cuda").bfloat16()
    out, lse = st.paged_attention(q, k, v, table, torch.tensor([2 ** 31 - 1]).int().cuda())
    s = k[0, 0].double() @ q[0].double().T / 8
    w = s.softmax(0)
    want, weighted = w.T @ v[0, 0].double(), w.T @ v[0, 0].double().abs()
    err = (out[0].double() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + 2.0 ** -11 * weighted).all()), float(err.max())
    assert float((lse[0].double() - s.logsumexp(0) - np.log(2)).abs().max()) <= 2.0 ** -11


def test_attention_of_large_scores(st):
    """Scores that rise and fall by hundreds: the running maximum is raised again and again."""
    pool = Pool([700, 700], 1, 16, 64)
    flat = pool.table[0, :44].long()
    pool.k[flat] = 0
    for pos in range(700):
        pool.k[flat[pos // 16], 0, pos % 16, 0] = float(pos % 97) * (1 if pos < 400 else -1)
    q = torch.zeros(2, 3, 64, device="cuda").bfloat16()
    q[0, 0, 0], q[0, 1, 0], q[0, 2, 0] = 8.0, -8.0, 0.125
    q[1] = pool.randn(3, 64).bfloat16()
    check_attention(st, pool, q, scale=1.0)


@pytest.mark.parametrize("length", [40, 20000])
def test_attention_not_a_number(st, length):
    """A head whose scores are NaN or +inf has NaN in O and in L, the others what they had;
    a dimension with an infinite value is not finite (a weight's two parts times it are infinities
    of either sign, or NaN for a part of 0)."""
    pool = Pool([length, length], 2, 16, 64)
    q = pool.randn(2, 8, 64).bfloat16()
    args = (pool.k, pool.v, pool.table, pool.lengths)
    want, want_lse = st.paged_attention(q, *args)
    q[0, 1, 5] = NAN
    q[1, 4] = 3e38
    at = pool.table[1, (length - 1) // 16].long(), 1, (length - 1) % 16
    pool.k[at] = 3e38  # a score of +inf for head 4 of sequence 1, whose key head is 1
    out, lse = st.paged_attention(q, *args)
    assert out[0, 1].isnan().all() and lse[0, 1].isnan()
    assert out[1, 4].isnan().all() and lse[1, 4].isnan()
    for b, h in [(0, 0), (0, 2), (0, 3), (0, 4), (0, 7), (1, 0), (1, 3)]:
        assert torch.equal(out[b, h], want[b, h]) and lse[b, h] == want_lse[b, h], (b, h)
    pool.v[pool.table[0, 0].long(), 1, 3, 17] = INF
    out, lse = st.paged_attention(q, *args)
    assert not out[0, 4:, 17].isfinite().any() and torch.equal(out[0, 4:, :17], want[0, 4:, :17])
    assert torch.equal(out[0, 4:, 18:], want[0, 4:, 18:]) and torch.equal(lse[0, 4:], want_lse[0, 4:])


def test_attention_shared_pages(st):
    """Sequences that share pages, as beams do."""
    pool = Pool([90] * 4, 2, 16, 128)
    pool.table[1:, :5] = pool.table[0, :5]
    check_attention(st, pool, pool.randn(4, 8, 128).bfloat16())


def test_attention_strides_buffers_and_scale(st):
    pool = Pool([70, 0, 9], 2, 16, 64)
    whole = pool.randn(3, 9, 64).bfloat16()
    q = whole[:, 1:7]
    out = torch.full((3, 6, 64), 7.0, device="cuda").bfloat16()
    lse = torch.zeros(3, 6, device="cuda")
    ws = torch.empty(st.os_paged_attention_workspace() + 16, dtype=torch.uint8, device="cuda")
    got = check_attention(st, pool, q, scale=0.3, out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse
    alone, none = st.paged_attention(q.contiguous(), pool.k, pool.v, pool.table, pool.lengths,
                                     scale=0.3, want_lse=False)
    assert none is None and torch.equal(alone, out)
    one = check_attention(st, Pool([70], 2, 16, 64), whole[:1, 2:6])
    assert one[0].shape == (1, 4, 64)


def test_attention_same_bits(st):
    pool = Pool([9000, 40, 1200], 2, 16, 128)
    q = pool.randn(3, 8, 128).bfloat16()
    first = st.paged_attention(q, pool.k, pool.v, pool.table, pool.lengths)
    for _ in range(5):
        again = st.paged_attention(q, pool.k, pool.v, pool.table, pool.lengths)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ------------------------------------------------------------------ append
def check_append(st, pool, lengths, starts, q_heads, rot, interleaved, tokens, seed=0):
    kv_heads, d = pool.k.shape[1], pool.k.shape[3]
    # one projection's result, padded, of which q, k and v are slices
    qkv = pool.randn(tokens, q_heads + 2 * kv_heads + 1, d).bfloat16()
    q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:-1]
    inv = None if rot == 0 else \
        (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))).float().cuda()
    lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    starts = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    q_out = torch.full((tokens, q_heads, d), 9.0, device="cuda").bfloat16() if q_heads else None
    want = ref.append(pool.k, pool.v, pool.table, lengths, k, v, q if q_heads else None, starts,
                      inv, interleaved, q_out)
    before = pool.k.clone(), pool.v.clone()
    got = st.paged_append(pool.k, pool.v, pool.table, lengths, k, v, q=q if q_heads else None,
                          starts=starts, inv_freq=inv, interleaved=interleaved, q_out=q_out)
    assert got is q_out
    size = 2 * max(float(qkv.abs().max()), 1.0)
    for name, mine, ideal in (("k", pool.k, want[0]), ("q", q_out, want[2])):
        if mine is not None:
            err = np.abs(np64(mine) - ideal)
            assert np.all(err <= 2.0 ** -8 * np.abs(ideal) + 2.0 ** -19 * size), name
    assert np.array_equal(np64(pool.v), want[1])
    if rot == 0:
        assert np.array_equal(np64(pool.k), want[0])
    # what no token went to is as it was
    touched = torch.from_numpy(np.any(want[1] != np64(before[1]), axis=(1, 3))).cuda()
    for now, then in ((pool.k, before[0]), (pool.v, before[1])):
        same = (now == then).all(dim=3).all(dim=1)
        assert bool((same | touched).all())


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 0), (128, 128), (128, 32), (128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("page", [1, 16, 20])
def test_append_one_each(st, d, rot, interleaved, page):
    lengths = [1, 5, 0, 40, 16, 17, -3]
    pool = Pool([0] * 7, 2, page, d, capacity=48, junk=0.0)
    check_append(st, pool, lengths, None, 6, rot, interleaved, 7)


@pytest.mark.parametrize("starts,lengths", [
    ([0, 3, 3, 20, 21], [3, 9, 40, 30]),         # whole prompts, behind prefixes, none, one
    ([2, 2, 5, 5, 9], [0, 3, 0, 48]),            # rows before the first and behind the last
    ([0, 0, 0, 0, 0], [1, 1, 1, 1]),             # no token at all
    ([0, 10, 20, 30, 30], [4, 60, 30, 0]),       # begins before position 0; ends past the table
])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_ragged(st, starts, lengths, interleaved):
    pool = Pool([0] * 4, 3, 16, 64, capacity=48, junk=0.0)
    check_append(st, pool, lengths, starts, 3, 64, interleaved, 33)


@pytest.mark.parametrize("seqs", [1, 33, 700])
def test_append_large(st, seqs):
    """As many tokens as fill the GPU: several per CTA, sequences found over several rounds."""
    counts = [1 + (i * 13) % 17 for i in range(seqs)] if seqs > 1 else [4999]
    starts = [0, *np.cumsum(counts).tolist()]
    pool = Pool([0] * seqs, 1, 64, 64, capacity=max(counts) + 11, junk=0.0)
    check_append(st, pool, [c + i % 11 for i, c in enumerate(counts)], starts, 2, 32, False,
                 starts[-1] + 5)


def test_append_pages_that_are_not_there(st):
    pool = Pool([0] * 3, 2, 16, 64, capacity=32, junk=0.0)
    pool.table[0, 0], pool.table[1, 1], pool.table[2, 0] = -1, pool.k.shape[0], 2 ** 31 - 1
    check_append(st, pool, [4, 20, 16], None, 2, 64, False, 3)


@pytest.mark.parametrize("pos", [2 ** 20 + 1, 2 ** 24 - 3, 2 ** 30 + 7, 2 ** 31 - 2])
def test_append_far_positions(st, pos):
    """Angles of many turns: q is rotated though the position is beyond the table."""
    pool = Pool([0], 1, 16, 64, capacity=16, junk=0.0)
    check_append(st, pool, [pos + 1], None, 2, 64, False, 1)


def test_append_then_attention(st):
    """A cache filled a token at a time is the cache filled at once."""
    one, all_ = (Pool([0] * 3, 2, 8, 64, capacity=40, junk=NAN) for _ in range(2))
    k, v = one.randn(3, 40, 2, 64).bfloat16(), one.randn(3, 40, 2, 64).bfloat16()
    inv = (100.0 ** (-torch.arange(32) / 32)).float().cuda()
    ends = [40, 1, 23]
    for t in range(40):
        lengths = torch.tensor([t + 1 if t < e else 0 for e in ends], dtype=torch.int32).cuda()
        st.paged_append(one.k, one.v, one.table, lengths, k[:, t], v[:, t], inv_freq=inv)
    lengths = torch.tensor(ends, dtype=torch.int32).cuda()
    starts = torch.tensor([0, 40, 41, 64], dtype=torch.int32).cuda()
    st.paged_append(all_.k, all_.v, all_.table, lengths, torch.cat([a[:e] for a, e in zip(k, ends)]),
                    torch.cat([a[:e] for a, e in zip(v, ends)]), starts=starts, inv_freq=inv)
    assert torch.equal(one.k.isnan(), all_.k.isnan())
    assert torch.equal(one.k.nan_to_num(), all_.k.nan_to_num())
    assert torch.equal(one.v.nan_to_num(), all_.v.nan_to_num())
    all_.lengths = lengths
    check_attention(st, all_, one.randn(3, 4, 64).bfloat16())


# ------------------------------------------------------------------ reorder
@pytest.mark.parametrize("layers", [None, 1, 3])
@pytest.mark.parametrize("page,d", [(1, 64), (4, 128), (20, 64), (64, 128)])
def test_reorder(st, layers, page, d):
    g = torch.Generator(device="cuda")
    g.manual_seed(page)
    groups, beams, width, kv_heads = 3, 4, 5, 3
    seqs = groups * beams
    pages = seqs * width * 2 + 1
    shape = (layers or 1, pages, kv_heads, page, d)
    k, v = (torch.randn(*shape, generator=g, device="cuda").bfloat16() for _ in range(2))
    if layers is None:
        k, v = k[0], v[0]
    ids = torch.rand(pages, generator=g, device="cuda").argsort().int()
    table, new = (ids[i * seqs * width:(i + 1) * seqs * width].view(seqs, width).clone()
                  for i in range(2))
    lengths = torch.tensor([0, 1, page, page + 1, 2 * page - 1, 2 * page, 3 * page + page // 2,
                            5 * page, 4 * page + page - 1, 7, -2, 9 * page], device="cuda").int()
    parents = torch.tensor([[3, 3, 0, 2], [1, 0, 3, 2], [0, -1, 1, 4]], device="cuda").int()
    new[0, 1] = -1                 # a page of its own that is not there: nothing is copied
    table[11, 4] = pages
    want = ref.reorder(*(np64(c).reshape(shape) for c in (k, v)), table, lengths, parents, new, page)
    out, out_lengths = st.paged_reorder(k, v, table, lengths, parents, new)
    assert out is new
    assert np.array_equal(np64(k).reshape(shape), want[0])
    assert np.array_equal(np64(v).reshape(shape), want[1])
    assert np.array_equal(out.cpu().numpy(), want[2])
    assert np.array_equal(out_lengths.cpu().numpy(), want[3])
    # again: the same
    st.paged_reorder(k, v, table, lengths, parents, new, out_lengths=out_lengths)
    assert np.array_equal(np64(k).reshape(shape), want[0])


def test_reorder_own_page_stays(st):
    """A table that names the parent's own page is no copy."""
    k = torch.randn(4, 1, 8, 64, device="cuda").bfloat16()
    v, table = k.clone(), torch.tensor([[0], [1]], device="cuda").int()
    new = torch.tensor([[0], [2]], device="cuda").int()
    st.paged_reorder(k, v, table, torch.tensor([5, 5]).int().cuda(),
                     torch.tensor([[0, 0]]).int().cuda(), new)
    assert torch.equal(k[2, :, :5], k[0, :, :5]) and torch.equal(v[2, :, 5:], v[2, :, 5:])
    assert new.tolist() == [[0], [2]]


# ------------------------------------------------------------------ far offsets, refusals
@pytest.mark.parametrize("page", [16, 24])
def test_offsets_past_32_bits(st, page):
    """A pool of more than 2^32 bytes, of which the last pages are used."""
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GB")
    kv_heads, d = 8, 128
    pages = 2 ** 32 // (kv_heads * page * d) + 40
    k, v = (torch.zeros(pages, kv_heads, page, d, dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    table = (pages - 1 - torch.arange(6, device="cuda")).int().view(2, 3).contiguous()
    new_k, new_v = torch.randn(2, 2, 60, kv_heads, d, device="cuda").bfloat16()
    lengths = torch.tensor([40, 33], device="cuda").int()
    starts = torch.tensor([0, 40, 73], device="cuda").int()
    st.paged_append(k, v, table, lengths, torch.cat([new_k[0, :40], new_k[1, :33]]),
                    torch.cat([new_v[0, :40], new_v[1, :33]]), starts=starts)
    q = torch.randn(2, 8, d, device="cuda").bfloat16()
    out, lse = st.paged_attention(q, k, v, table, lengths)
    small = [c[-6:].clone() for c in (k, v)]
    at = table - (pages - 6)
    want = st.paged_attention(q, *small, at, lengths)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(small[0][at[0, 0], :, 5], new_k[0, 5])
    new = table.flip(0).contiguous() - 100
    new_small = torch.full_like(new, -1)
    st.paged_reorder(k, v, table, lengths, torch.tensor([[1, 0]]).int().cuda(), new)
    full = 33 // page
    assert torch.equal(new[0, :full], table[1, :full])
    if 33 % page:
        assert torch.equal(k[new[0, full].long(), :, :33 % page],
                           k[table[1, full].long(), :, :33 % page])
    del new_small


def test_tensor_refusals(st):
    pool = Pool([20, 20], 2, 16, 64)
    q = pool.randn(2, 4, 64).bfloat16()
    good = (pool.k, pool.v, pool.table, pool.lengths)

    def refused(error, f, *args, **kw):
        with pytest.raises(error):
            f(*args, **kw)

    k = q[:, :2]
    for i, bad in enumerate((pool.k.float(), pool.v[:1], pool.table.long(), pool.lengths[:1])):
        c = [*good]
        c[i] = bad
        refused(ValueError, st.paged_attention, q, *c)
        refused(ValueError, st.paged_append, *c, k, k)
        refused(ValueError, st.paged_reorder, *c, pool.table[:1], pool.table.clone())
    refused(ValueError, st.paged_attention, q.float(), *good)
    refused(ValueError, st.paged_attention, q[:1], *good)
    refused(ValueError, st.paged_attention, q.transpose(1, 2), *good)
    refused(ValueError, st.paged_attention, q[:, :, ::2].repeat(1, 1, 2)[:, :, ::2], *good)
    refused(st.OsError, st.paged_attention, q[:, :3], *good)
    refused(ValueError, st.paged_attention, q, *good, out=q[:, :2])
    refused(st.OsError, st.paged_attention, q, *good, out=q)
    refused(ValueError, st.paged_attention, q, *good,
            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    refused(st.OsError, st.paged_attention, q, *good, scale=-1.0)
    refused(ValueError, st.paged_append, *good, k, k, q_out=q)
    refused(ValueError, st.paged_append, *good, k, k[:1])
    refused(ValueError, st.paged_append, *good, k[0, 0, 0], k[0, 0, 0])
    refused(st.OsError, st.paged_append, *good, k[:1], k[:1])
    refused(ValueError, st.paged_append, *good, k, k, starts=torch.zeros(2).int().cuda())
    refused(st.OsError, st.paged_append, *good, k, k, inv_freq=torch.ones(12).cuda())
    refused(st.OsError, st.paged_append, *good, k, k, inv_freq=torch.ones(64).cuda())
    refused(ValueError, st.paged_append, *good, k, k, inv_freq=torch.ones(32).double().cuda())
    parents = torch.zeros(1, 2).int().cuda()
    refused(ValueError, st.paged_reorder, *good, parents[0], pool.table.clone())
    refused(ValueError, st.paged_reorder, *good, parents.repeat(2, 1), pool.table.clone())
    refused(st.OsError, st.paged_reorder, *good, parents, pool.table)
    # no sequences, no tokens
    none = torch.zeros(0, 3).int().cuda()
    out, lse = st.paged_attention(q[:0], pool.k, pool.v, none, pool.lengths[:0])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert st.paged_append(pool.k, pool.v, none, pool.lengths[:0], k[:0], k[:0]) is None
    st.paged_append(*good, k[:0], k[:0], starts=torch.zeros(3).int().cuda())
