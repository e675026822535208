"""The paged cache's states, checked to the last row: what a reordering copies and what it leaves, in
both pools, far offsets among them; keys and values of beams' histories; beams that die; tables much
wider than their sequences; append's angles and lengths at their limits; captures in which other
things than kernels come before a call."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import decode as ref
from tests.test_gpu_decode_step import Model, prompts
from tests.test_gpu_paged import Pool, check_attention, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ reorder
def test_reorder_touches_the_filled_rows_alone(st):
    """A copy, and a table that names the parent's own page, which is none."""
    g = generator(0)
    k, v = randn(g, 4, 2, 8, 64).bfloat16(), randn(g, 4, 2, 8, 64).bfloat16()
    was = k.clone(), v.clone()
    new = torch.tensor([[0], [2]], device="cuda").int()
    st.paged_reorder(k, v, torch.tensor([[0], [1]]).int().cuda(), torch.tensor([5, 5]).int().cuda(),
                     torch.tensor([[0, 0]]).int().cuda(), new)
    for now, then in zip((k, v), was):
        then[2, :, :5] = then[0, :, :5]
        assert torch.equal(now, then)
    assert new.tolist() == [[0], [2]]


@pytest.mark.parametrize("page", [16, 24])
def test_reorder_past_32_bits(st, page):
    """Pages more than 2^32 bytes apart, from the pool's end to its start and back: keys and values
    of both sequences, and nothing else."""
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GB")
    g, kv_heads, d = generator(page), 8, 128
    pages = 2 ** 32 // (kv_heads * page * d) + 40
    k, v = (torch.zeros(pages, kv_heads, page, d, dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    last = pages - 1
    table = torch.tensor([[last, last - 1, last - 2], [0, 1, 2]], device="cuda").int()
    new = torch.tensor([[10, 11, 12], [last - 10, last - 11, last - 12]], device="cuda").int()
    lengths = torch.tensor([2 * page + 7, page + 3], device="cuda").int()
    rows = torch.tensor([0, 1, 2, *range(10, 13), *range(last - 12, last + 1)], device="cuda")
    for pool in (k, v):
        pool[rows] = randn(g, len(rows), kv_heads, page, d).bfloat16()
    was = [pool[rows].clone() for pool in (k, v)]
    where = {int(r): i for i, r in enumerate(rows)}
    out, out_lengths = st.paged_reorder(k, v, table, lengths, torch.tensor([[1, 0]]).int().cuda(),
                                        new)
    assert out_lengths.tolist() == [page + 3, 2 * page + 7]
    assert out.tolist() == [[0, 11, 12], [last, last - 1, last - 12]]
    for pool, then in zip((k, v), was):
        then[where[11], :, :3] = then[where[1], :, :3]
        then[where[last - 12], :, :7] = then[where[last - 2], :, :7]
        assert torch.equal(pool[rows], then)
        for low, high in ((3, 10), (13, last - 12)):
            assert all(int(torch.count_nonzero(part)) == 0 for part in pool[low:high].split(4096))


# ------------------------------------------------------------------ histories
def test_beam_search_keeps_keys_and_values(st):
    """Every beam's cache behind every reordering: its own tokens' keys, rotated by their positions
    (rounded once, half a step), and values."""
    m = Model(st, 2, 3, seed=5)
    given = prompts(4)
    m.prompt(given)
    seqs = m.groups * m.beams
    history = [given[j // m.beams].tolist() for j in range(seqs)]
    for step in range(10):
        now = 1 - step % 2
        history = [h + [t] for h, t in zip(history, m.tokens.tolist())]
        m.step(now)
        parents = m.parents.flatten().tolist()
        history = [history[j // m.beams * m.beams + parents[j]] for j in range(seqs)]
        table = m.tables[1 - now].cpu().numpy()
        for j, h in enumerate(history):
            at = [(int(table[j, p // m.page]), p % m.page) for p in range(len(h))]
            for layer in range(m.layers):
                rows = m.embed[layer][h]
                v = torch.stack([m.v[layer, page, :, slot] for page, slot in at])
                assert torch.equal(v, rows[:, -m.kv_heads:])
                k = np64(torch.stack([m.k[layer, page, :, slot] for page, slot in at]))
                plain = np64(rows[:, m.q_heads:-m.kv_heads])
                want = np.stack([ref.rotate(x, p, m.inv_freq, False) for p, x in enumerate(plain)])
                # 2^-19 of |x| + |y|, as for the append itself
                slack = 2.0 ** -19 * 2 * np.abs(plain).max()
                assert np.all(np.abs(k - want) <= 2.0 ** -8 * np.abs(want) + slack)


def test_beams_that_die(st):
    """Steps that leave fewer continuations than beams: the places without one stay idle (length 0)
    until a later choice fills them, and the others' pages, which their tables still name, keep what
    they hold."""
    g = generator(8)
    beams, page, width, vocab = 4, 4, 8, 50
    embed = randn(g, vocab, 1, 64).bfloat16()
    pages = 2 * beams * width
    k, v = (torch.full((pages, 1, page, 64), float("nan"), device="cuda").bfloat16()
            for _ in range(2))
    tables = [t.clone() for t in torch.randperm(pages, generator=g, device="cuda").int()
              .view(2, beams, width)]
    lengths = [torch.tensor([0, 0, 0, 0], dtype=torch.int32, device="cuda") for _ in range(2)]
    lengths[0].fill_(1)
    history = [[3], [4], [5], [6]]
    st.paged_append(k, v, tables[0], lengths[0], *(embed[[3, 4, 5, 6]] for _ in range(2)))
    scores = -torch.arange(4.0, device="cuda").view(1, 4)
    now = 0
    for step in range(20):
        x = randn(g, beams, vocab)
        if step % 4 == 2:  # two of one beam, one of another
            keep = torch.full_like(x, float("-inf"))
            live = torch.nonzero(lengths[now] > 0).flatten().tolist()
            keep[live[0], 7], keep[live[0], 9], keep[live[-1], 11] = 0.5, 0.25, 0.0
            x = keep
        elif step % 4 == 3:
            x[:, 2:] = float("-inf")  # two of each
        scores, parents, tokens = st.beam_select(x, scores, beams)
        st.paged_reorder(k, v, tables[now], lengths[now], parents, tables[1 - now],
                         out_lengths=lengths[1 - now])
        now = 1 - now
        p, t = parents.flatten().tolist(), tokens.flatten().tolist()
        history = [history[p[j]] + [t[j]] if p[j] >= 0 else None for j in range(beams)]
        if step % 4 == 2:
            assert sum(h is not None for h in history) == 3
        lengths[now].add_((lengths[now] > 0).int())
        new = embed[tokens.flatten().clamp(min=0).long()]
        st.paged_append(k, v, tables[now], lengths[now], new, new)
        table = tables[now].cpu().numpy()
        assert lengths[now].tolist() == [0 if h is None else len(h) for h in history]
        for j, h in enumerate(history):
            if h is None:
                continue
            held = torch.stack([v[int(table[j, i // page]), :, i % page] for i in range(len(h))])
            assert torch.equal(held, embed[h]), (step, j)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("seqs,length,kv_heads,group,d", [
    (1, 1000, 2, 8, 128), (1, 16, 2, 8, 64), (4, 200, 1, 16, 128), (30, 60, 4, 1, 64),
    (100, 33, 1, 8, 64), (3, 700, 1, 40, 128)])
def test_attention_under_a_wide_table(st, seqs, length, kv_heads, group, d):
    """A table for 131072 keys, as a captured step has, and short sequences."""
    pool = Pool([max(1, length - 7 * i) for i in range(seqs)], kv_heads, 16, d, seed=seqs,
                extra_width=8192 - -(-length // 16))
    check_attention(st, pool, 2 * pool.randn(seqs, kv_heads * group, d).bfloat16())


def test_captures_behind_copies_and_other_streams(st):
    """A call behind memory copies, and one that waits for another stream, in one graph."""
    g = generator(1)
    k, v = (randn(g, 300, 2, 16, 64).bfloat16() for _ in range(2))
    given = [(torch.randint(0, 300, (8, 20), generator=g, device="cuda").int(),
              torch.randint(0, 321, (8,), generator=g, device="cuda").int(),
              randn(g, 8, 4, 64).bfloat16()) for _ in range(3)]
    held, source = ([t.clone() for t in given[0]] for _ in range(2))
    table, lengths, q = held
    st.paged_attention(q, k, v, table, lengths)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        for to, of in zip(held, source):
            to.copy_(of)
        first = st.paged_attention(q, k, v, table, lengths)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            twice = q * 2
        second = st.paged_attention(q, k, v, table, lengths)
        torch.cuda.current_stream().wait_stream(side)
        third = st.paged_attention(twice, k, v, table, lengths)
    for table_now, lengths_now, q_now in given:
        for to, of in zip(source, (table_now, lengths_now, q_now)):
            to.copy_(of)
        graph.replay()
        want = st.paged_attention(q_now, k, v, table_now, lengths_now)
        want2 = st.paged_attention(q_now * 2, k, v, table_now, lengths_now)
        for got, w in ((first, want), (second, want), (third, want2)):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])


# ------------------------------------------------------------------ append
def test_append_lengths_past_the_table(st):
    """Lengths are not clamped here: positions beyond the table are not stored."""
    pool = Pool([0, 0], 1, 16, 64, capacity=48, junk=0.0)
    new = pool.randn(8, 1, 64).bfloat16()
    was = pool.v.clone()
    st.paged_append(pool.k, pool.v, pool.table, torch.tensor([50, 2 ** 31 - 1]).int().cuda(), new,
                    new, starts=torch.tensor([0, 5, 8]).int().cuda())
    for i, pos in enumerate(range(45, 48)):
        was[int(pool.table[0, pos // 16]), :, pos % 16] = new[i]
    assert torch.equal(pool.v, was)


@pytest.mark.parametrize("pos", [0, 1000, 2 ** 20 + 1, 2 ** 31 - 2])
@pytest.mark.parametrize("top", [1.0, 1000.0, 3.0e5])
def test_append_angles_of_large_frequencies(st, pos, top):
    """A turn's fraction is good to 2^-51 of the turns' number; sine, cosine and the two products to
    2^-20 of |x| + |y| with it."""
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    g = generator(pos % 1000)
    inv = (top * torch.rand(32, generator=g, device="cuda")).float()
    q = randn(g, 1, 2, 64).bfloat16()
    k, v = (torch.zeros(1, 1, 16, 64, device="cuda").bfloat16() for _ in range(2))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    out = np64(st.paged_append(k, v, table, torch.tensor([pos + 1]).int().cuda(), q[:, :1], q[:, :1],
                               q=q, inv_freq=inv))
    x, y = np64(q)[..., :32], np64(q)[..., 32:]
    turns = [Fraction(pos) * Fraction(f) / (2 * pi) for f in inv.tolist()]
    angle = np.array([float((t - round(t)) * 2 * pi) for t in turns])
    off = 2 * math.pi * np.array([float(t) for t in turns]) * 2.0 ** -51 + 2.0 ** -20
    for got, want in ((out[..., :32], x * np.cos(angle) - y * np.sin(angle)),
                      (out[..., 32:], y * np.cos(angle) + x * np.sin(angle))):
        slack = off * (np.abs(x) + np.abs(y))
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * (np.abs(want) + slack) + slack)
