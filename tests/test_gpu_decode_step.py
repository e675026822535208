"""The decode loop's operators together, as a serving or beam-search program uses them: append with
rotation, attention over the cache, logits, the search's selection, and the reordering of the
states; in eager steps against the float64 oracle over every beam's own history, in captured
graphs that take turns, and from several threads."""
import threading

import numpy as np
import pytest
import torch

from oracle import decode as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


class Model:
    """Layers of attention and an output projection, with everything that a step needs."""
    layers, q_heads, kv_heads, d, vocab, page, width = 2, 4, 2, 64, 211, 4, 8

    def __init__(self, st, groups, beams, seed=0):
        self.st, self.groups, self.beams = st, groups, beams
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        seqs = groups * beams

        def randn(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        heads = self.q_heads + 2 * self.kv_heads
        self.embed = randn(self.layers, self.vocab, heads, self.d).bfloat16()
        self.out = (randn(self.layers * self.q_heads * self.d, self.vocab) * 0.3).bfloat16()
        self.inv_freq = (100.0 ** (-torch.arange(self.d // 2) / (self.d // 2))).float().cuda()
        pages = 2 * seqs * self.width
        shape = (self.layers, pages, self.kv_heads, self.page, self.d)
        self.k, self.v = (torch.full(shape, float("nan"), device="cuda").bfloat16()
                          for _ in range(2))
        ids = torch.rand(pages, generator=g, device="cuda").argsort().int()
        # two tables that take turns, each with pages of its own for every place
        self.tables = [t.clone() for t in ids.view(2, seqs, self.width)]
        self.lengths = [torch.zeros(seqs, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.scores = torch.zeros(groups, beams, device="cuda")
        self.tokens = torch.zeros(seqs, dtype=torch.int64, device="cuda")
        self.parents = torch.zeros(groups, beams, dtype=torch.int32, device="cuda")

    def qkv(self, layer, tokens):
        x = self.embed[layer][tokens]
        return x[:, :self.q_heads], x[:, self.q_heads:-self.kv_heads], x[:, -self.kv_heads:]

    def prompt(self, prompts):
        """Each group's prompt into its first beam's pages; then all beams go on from it."""
        table, lengths = self.tables[0], self.lengths[0]
        starts, at = [0], 0
        for p in prompts:
            starts += [at + len(p)] * self.beams
            at += len(p)
            lengths[(len(starts) - 2) // self.beams * self.beams] = len(p)
        tokens = torch.cat(prompts)
        starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        for layer in range(self.layers):
            _, k, v = self.qkv(layer, tokens)
            self.st.paged_append(self.k[layer], self.v[layer], table, lengths, k, v, starts=starts,
                                 inv_freq=self.inv_freq)
        self.st.paged_reorder(self.k, self.v, table, lengths, self.parents, self.tables[1],
                              out_lengths=self.lengths[1])
        self.tokens.copy_(torch.stack([p[-1] for p in prompts]).repeat_interleave(self.beams))
        self.scores.fill_(float("-inf"))
        self.scores[:, 0] = 0.0

    def step(self, now):
        """A token for every beam, from table `now` to the other one."""
        st, table, lengths = self.st, self.tables[now], self.lengths[now]
        lengths.add_(1)
        outs = []
        for layer in range(self.layers):
            q, k, v = self.qkv(layer, self.tokens)
            q = st.paged_append(self.k[layer], self.v[layer], table, lengths, k, v, q=q,
                                inv_freq=self.inv_freq)
            outs.append(st.paged_attention(q, self.k[layer], self.v[layer], table, lengths)[0])
        logits = (torch.cat(outs, 1).flatten(1) @ self.out).float()
        scores, parents, tokens = st.beam_select(logits, self.scores, self.beams)
        st.paged_reorder(self.k, self.v, table, lengths, parents, self.tables[1 - now],
                         out_lengths=self.lengths[1 - now])
        self.scores.copy_(scores)
        self.parents.copy_(parents)
        self.tokens.copy_(tokens.flatten())
        return outs, logits


def prompts(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [torch.randint(0, Model.vocab, (n,), generator=g, device="cuda") for n in (5, 8)]


def test_beam_search_keeps_every_history(st):
    m = Model(st, 2, 3)
    given = prompts(1)
    m.prompt(given)
    seqs = m.groups * m.beams
    # the positions' tokens that each sequence's cache holds, and the token to come
    history = [given[j // m.beams].tolist() for j in range(seqs)]
    scores = m.scores.clone()
    for step in range(14):
        now = 1 - step % 2
        history = [h + [t] for h, t in zip(history, m.tokens.tolist())]
        before = m.scores.clone()
        outs, logits = m.step(now)
        assert m.lengths[now].tolist() == [len(h) for h in history]
        for layer, out in enumerate(outs):
            embed = m.embed[layer].double().cpu().numpy()
            for j, h in enumerate(history):
                rows = embed[h]
                k = np.stack([ref.rotate(x, p, m.inv_freq, False) for p, x in
                              enumerate(rows[:, m.q_heads:-m.kv_heads])])
                q = ref.rotate(rows[-1][:m.q_heads], len(h) - 1, m.inv_freq, False)
                for head in range(m.q_heads):
                    kv = head // (m.q_heads // m.kv_heads)
                    s = k[:, kv] @ q[head] * m.d ** -0.5
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    v = rows[:, m.q_heads + m.kv_heads + kv]
                    # q and k are each rounded once to bf16: 2^-8 of sum |q k| scale and more in
                    # a score, and as much of the weights; O half a step
                    slack = np.abs(k[:, kv]) @ np.abs(q[head]) * m.d ** -0.5 * 2.0 ** -6.9
                    bound = (w * (np.exp(2 * slack.max()) - 1)) @ np.abs(v) + 2.0 ** -8 * np.abs(w @ v)
                    assert np.all(np.abs(out[j, head].double().cpu().numpy() - w @ v) <= bound)
        want = ref.beam_select(logits, before, m.beams)
        assert np.array_equal(m.parents.cpu().numpy(), want[1])
        assert np.array_equal(m.tokens.view(m.groups, m.beams).cpu().numpy(), want[2])
        parents = m.parents.flatten().tolist()
        history = [history[j // m.beams * m.beams + parents[j]] for j in range(seqs)]
        # the cache holds each history, key for key, behind the reordering too
        table = m.tables[1 - now].cpu().numpy()
        assert m.lengths[1 - now].tolist() == [len(h) for h in history]
        for j, h in enumerate(history):
            for layer in range(m.layers):
                v = m.embed[layer][h][:, -m.kv_heads:]
                at = [(int(table[j, p // m.page]), p % m.page) for p in range(len(h))]
                held = torch.stack([m.v[layer, page, :, slot] for page, slot in at])
                assert torch.equal(held, v)
    assert not torch.equal(scores, m.scores)


def test_graphs_that_take_turns(st):
    """The two steps of the tables' turns, captured and replayed: the eager loop's bits."""
    a, b = Model(st, 2, 4, seed=3), Model(st, 2, 4, seed=3)
    for m in (a, b):
        m.prompt(prompts(2))
    graphs = []
    saved = [t.clone() for t in (b.k, b.v, *b.tables, *b.lengths, b.scores, b.tokens, b.parents)]
    for now in (1, 0):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.step(now)
        graphs.append(graph)
    for t, s in zip((b.k, b.v, *b.tables, *b.lengths, b.scores, b.tokens, b.parents), saved):
        t.copy_(s)
    for step in range(12):
        a.step(1 - step % 2)
        graphs[step % 2].replay()
        for x, y in zip((*a.tables, *a.lengths, a.scores, a.tokens, a.parents),
                        (*b.tables, *b.lengths, b.scores, b.tokens, b.parents)):
            assert torch.equal(x, y)
    assert torch.equal(a.k.nan_to_num(), b.k.nan_to_num())
    assert torch.equal(a.v.nan_to_num(), b.v.nan_to_num())


def work(st, seed):
    """Inputs of every operator, large enough to split and join, and a function that runs them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    seqs, kv_heads, page, d, width = 6, 2, 16, 128, 200 + 30 * seed
    pages = seqs * width
    k, v = (randn(pages, kv_heads, page, d).bfloat16() for _ in range(2))
    table = torch.rand(pages, generator=g, device="cuda").argsort().int().view(seqs, width)
    table = table.contiguous()
    lengths = torch.tensor([width * page, 5, 0, 2000, 333, 1], device="cuda").int()
    q, kn, vn = randn(seqs, 8, d).bfloat16(), randn(seqs, 2, d).bfloat16(), randn(seqs, 2, d).bfloat16()
    inv = (10000.0 ** (-torch.arange(64) / 64)).float().cuda()
    x, s = randn(12, 30011) * 3, randn(3, 4)
    new = torch.full_like(table, -1)

    def run():
        q2 = st.paged_append(k, v, table, lengths, kn, vn, q=q, inv_freq=inv)
        out, lse = st.paged_attention(q2, k, v, table, lengths)
        some = st.beam_select(x, s, 9)
        new.fill_(-1)
        moved, _ = st.paged_reorder(k, v, table, lengths, some[1][:, :2].contiguous(), new)
        keep = (lengths > 0)[:, None, None]
        return [q2.masked_fill(~keep, 0), out, lse, *some, moved.clone()]

    return run


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


def test_threads_on_streams_of_their_own(st):
    runs = [work(st, s) for s in range(4)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    wrong = []

    def repeat(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got = [runs[i]() for _ in range(8)]
                torch.cuda.current_stream().synchronize()
            wrong.extend(i for g in got if not same(g, want[i]))
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=repeat, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


def test_two_threads_on_one_stream(st):
    """Calls of two launches that interleave on a stream do not share a workspace."""
    runs = [work(st, s) for s in range(2)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    wrong = []

    def repeat(i):
        try:
            got = [runs[i]() for _ in range(20)]
            torch.cuda.synchronize()
            wrong.extend(i for g in got if not same(g, want[i]))
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=repeat, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == []


def test_graphs_replayed_at_once(st):
    runs = [work(st, s) for s in range(2)]
    want = [[t.clone() for t in r()] for r in runs]
    graphs, outs = [], []
    for r in runs:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(r())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all(same(o, w) for o, w in zip(outs, want))


def test_graph_with_other_lengths(st):
    """Lengths are read on the device: a captured step serves a batch that grows and shrinks."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    k, v = (torch.randn(400, 2, 16, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.rand(400, generator=g, device="cuda").argsort().int().view(4, 100).contiguous()
    lengths = torch.zeros(4, dtype=torch.int32, device="cuda")
    q = torch.randn(4, 4, 64, generator=g, device="cuda").bfloat16()
    st.paged_attention(q, k, v, table, lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = st.paged_attention(q, k, v, table, lengths)
    for now in ([0, 0, 0, 0], [1, 0, 1600, 3], [1600] * 4, [17, 900, 0, 16], [0, 0, 0, 1]):
        lengths.copy_(torch.tensor(now))
        graph.replay()
        want = st.paged_attention(q, k, v, table, lengths)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_what_the_kernel_before_wrote(st):
    """Calls that may be put in place early still read what the kernels just before them write."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    k, v = (randn(300, 2, 16, 64).bfloat16() for _ in range(2))
    tables = [torch.randint(0, 200, (8, 20), generator=g, device="cuda").int() for _ in range(4)]
    lengths = [torch.randint(0, 321, (8,), generator=g, device="cuda").int() for _ in range(4)]
    own = torch.arange(200, 296, device="cuda").int().view(8, 12)
    queries = [randn(8, 4, 64).bfloat16() for _ in range(4)]
    parents = [torch.randint(0, 4, (2, 4), generator=g, device="cuda").int() for _ in range(4)]
    table, length, q = (torch.zeros_like(x[0]) for x in (tables, lengths, queries))
    parent, out_table = torch.zeros_like(parents[0]), torch.zeros_like(tables[0])

    def run(wait):
        got = []
        for i in range(40):
            q.copy_(queries[i % 4])
            table.copy_(tables[i % 3])
            length.copy_(lengths[i % 4])
            wait()
            got += [t.clone() for t in st.paged_attention(q, k, v, table, length)]
            out_table.fill_(-1)
            out_table[:, 8:] = own
            parent.copy_(parents[i % 4])
            wait()
            got += [t.clone() for t in st.paged_reorder(k, v, table, length, parent, out_table)]
            wait()
        return got

    want = run(torch.cuda.synchronize)
    assert same(run(lambda: None), want)


COLD = """
import torch
import softmax_topk_gb300 as st
g = torch.Generator(device="cuda")
g.manual_seed(1)
def randn(*shape):
    return torch.randn(*shape, generator=g, device="cuda")
k, v = (randn(120, 2, 16, 64).bfloat16() for _ in range(2))
table = torch.arange(60, device="cuda").int().view(2, 30).contiguous()
lengths = torch.tensor([480, 33], device="cuda").int()
q, kn = randn(2, 4, 64).bfloat16(), randn(2, 2, 64).bfloat16()
inv = torch.ones(32, device="cuda")
x, s = randn(2, 9000), torch.zeros(1, 2, device="cuda")
new = table + 60  # pages of the sequences' own
def step():
    q2 = st.paged_append(k, v, table, lengths, kn, kn, q=q, inv_freq=inv)
    out, lse = st.paged_attention(q2, k, v, table, lengths)
    some = st.beam_select(x, s, 2)
    return [q2, out, lse, *some, *st.paged_reorder(k, v, table, lengths, some[1], new)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("same")
"""


def test_first_calls_inside_a_capture():
    """A process whose first call of every operator is recorded into a graph."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", COLD], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
