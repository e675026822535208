"""The attention gradient, the router and its gradient and the sampler called from several threads
on streams of their own, replayed from two graphs at once, and on tensors whose offsets pass
32 bits: the same bits as one call at a time on a small tensor."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


def work(st, seed):
    """One set of inputs and a function that runs every operator on them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    q, k, v, do = (randn(3, 200 + 50 * seed, 64).bfloat16() for _ in range(4))
    o, lse = st.attention(q, k, v, causal=seed % 2 == 0)
    x, bias = randn(3000, 256), randn(256) * 0.1
    rows = randn(5 + 40 * seed, 30011) * 3
    u = torch.rand(len(rows), generator=g, device="cuda")

    def run():
        grads = st.attention_backward(q, k, v, o, lse, do, causal=seed % 2 == 0)
        w, idx = st.route(x, 8, score="sigmoid", bias=bias, groups=8, topk_groups=4, group_top=2)
        dx = st.route_backward(x, idx, w, score="softmax")
        return [*grads, w, idx, dx, *st.sample(rows, u, temperature=0.9, top_p=0.8),
                *st.sample(rows, u, top_k=30, min_p=0.01), *st.sample(rows, u, top_k=1500)]

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
                got = [runs[i]() for _ in range(6)]
                torch.cuda.current_stream().synchronize()
            wrong.extend(i for g in got if not same(g, want[i]))
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=repeat, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_two_graphs_replayed_at_once(st):
    runs = [work(st, s) for s in (1, 2)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(r())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert same(outs[0], want[0]) and same(outs[1], want[1])


def test_sample_without_probabilities(st):
    x = torch.randn(3, 1000, device="cuda")
    u = torch.rand(3, device="cuda")
    want, _ = st.sample(x, u, top_p=0.7)
    out = torch.empty_like(want)
    settings = st.Sampling(temperature_all=1.0, top_k_all=0, top_p_all=0.7, min_p_all=0.0)
    st.os_sample(x.data_ptr(), u.data_ptr(), settings, out.data_ptr(), None, 3, 1000, st.OS_F32,
                 torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_attention_gradient_past_32_bits(st):
    bh, n, d = 2 ** 17 + 9, 130, 128  # 2.2e9 elements a tensor
    small = [torch.randn(11, n, d, device="cuda").bfloat16() for _ in range(4)]
    o, lse = st.attention(*small[:3], causal=True)
    want = st.attention_backward(*small[:3], o, lse, small[3], causal=True)
    rep = (bh + 10) // 11

    def tile(t):
        return t.repeat(rep, *([1] * (t.dim() - 1)))[:bh].contiguous()

    big = [tile(t) for t in (*small[:3], o, lse, small[3])]
    got = st.attention_backward(*big, causal=True)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for at in (0, bh // 2, bh - 1):
            assert torch.equal(g[at], w[at % 11])


def test_router_past_32_bits(st):
    rows, experts = 2 ** 23 + 1003, 260  # 2.2e9 logits; 260: one warp per row
    small = torch.randn(1009, experts, device="cuda").bfloat16()
    x = small.repeat((rows + 1008) // 1009, 1)[:rows]
    w, idx = st.route(x, 5, score="sigmoid")
    ws, ids = st.route(small, 5, score="sigmoid")
    dx = st.route_backward(x, idx, w, score="softmax", renorm=False)
    ds = st.route_backward(small, ids, ws, score="softmax", renorm=False)
    last = torch.arange(rows - 500, rows, device="cuda")
    assert torch.equal(idx[last], ids[last % 1009]) and torch.equal(w[last], ws[last % 1009])
    assert torch.equal(dx[last], ds[last % 1009])
    del dx
    x = x.view(-1)[:(2 ** 31 // 256 + 1003) * 256].view(-1, 256)  # 256: four threads per row
    w, idx = st.route(x, 5, score="sigmoid")
    ws, ids = st.route(x[-500:].clone(), 5, score="sigmoid")
    assert torch.equal(idx[-500:], ids) and torch.equal(w[-500:], ws)


def test_sampler_past_32_bits(st):
    rows, cols = 17000, 128256  # 2.18e9 logits
    small = (torch.randn(13, cols, device="cuda") * 3).bfloat16()
    x = small.repeat((rows + 12) // 13, 1)[:rows]
    u = torch.rand(rows, device="cuda")
    for kw in ({"temperature": 0.7}, {"top_p": 0.9}, {"top_k": 50}):
        out, prob = st.sample(x, u, **kw)
        some = torch.arange(rows - 13, rows, device="cuda")
        want, want_p = st.sample(small[some % 13].contiguous(), u[some].contiguous(), **kw)
        assert torch.equal(out[some], want) and torch.equal(prob[some], want_p)
