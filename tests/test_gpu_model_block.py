"""The operators together, as a model's step runs them: attention, a router over experts, their
mix, logits and a sampler; and the gradients back through router and attention, against
float64 autograd of the same block with the same experts chosen.

Tolerance: q, k, v, the attention's output and the gradient that reaches it are rounded to bf16
(2^-8 each), P, dS and the three gradients inside its backward pass too, so a gradient of the
block carries at most eight such roundings, 8 * 2^-8 = 2^-5 of its norm; the rest is fp32."""
import numpy as np
import pytest
import torch

from oracle import operators as ref

pytestmark = pytest.mark.gpu
HEADS, N, D, E, K, VOCAB = 2, 150, 64, 16, 4, 1003
ROUTE = dict(score="sigmoid", groups=4, topk_groups=2, group_top=2, renorm=True, scale=2.0)


@pytest.fixture(scope="module")
def st():
    import softmax_topk_gb300
    return softmax_topk_gb300


@pytest.fixture(scope="module")
def net():
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def randn(*shape, scale):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    width = HEADS * D
    return dict(x=randn(N, width, scale=1.0), wqkv=randn(3, width, width, scale=width ** -0.5),
                wr=randn(width, E, scale=width ** -0.5 * 3), bias=randn(E, scale=0.1),
                we=randn(E, width, width, scale=width ** -0.5),
                wv=randn(width, VOCAB, scale=0.3), u=torch.rand(N, generator=g, device="cuda"),
                g=randn(N, width, scale=1.0))


def heads(t):  # [N, HEADS * D] -> [HEADS, N, D]
    return t.view(N, HEADS, D).transpose(0, 1).contiguous()


def forward(st, p, out=None):
    q, k, v = (heads(p["x"] @ w).bfloat16() for w in p["wqkv"])
    o, lse = st.attention(q, k, v, causal=True)
    h = o.float().transpose(0, 1).reshape(N, -1)
    z = h @ p["wr"]
    w, idx = st.route(z, K, bias=p["bias"], **ROUTE)
    each = torch.stack([torch.bmm(h[:, None], p["we"][idx[:, j].long()])[:, 0] for j in range(K)], 1)
    y = (w[:, :, None] * each).sum(1)
    token, prob = st.sample(y @ p["wv"], p["u"], temperature=0.8, top_k=40, top_p=0.9, min_p=0.01)
    return dict(q=q, k=k, v=v, o=o, lse=lse, h=h, z=z, w=w, idx=idx, each=each, y=y, token=token,
                prob=prob)


def test_block_forward_and_backward(st, net):
    f = forward(st, net)
    w, idx = ref.route(f["z"], K, bias=net["bias"].cpu().numpy().astype(np.float64), **ROUTE)
    assert (f["idx"].cpu().numpy() == idx).all()
    logits = f["y"] @ net["wv"]
    token, _ = ref.sample(logits, net["u"], 0.8, 40, 0.9, 0.01)
    assert (f["token"].cpu().numpy() == token).all()

    # back from the gradient of y
    g = net["g"]
    dw = (f["each"] * g[:, None]).sum(-1)
    dz = st.route_backward(f["z"], f["idx"], dw, score="sigmoid", renorm=True, scale=2.0)
    dh = dz @ net["wr"].T
    for j in range(K):
        dh += f["w"][:, j:j + 1] * torch.bmm(g[:, None], net["we"][f["idx"][:, j].long()].mT)[:, 0]
    do = heads(dh).bfloat16()
    grads = st.attention_backward(f["q"], f["k"], f["v"], f["o"], f["lse"], do, causal=True)
    dx = sum(t.float().transpose(0, 1).reshape(N, -1) @ wm.T for t, wm in zip(grads, net["wqkv"]))

    # the same in float64, the chosen experts held
    x = net["x"].double().requires_grad_(True)
    q, k, v = (heads(x @ wm.double()) for wm in net["wqkv"])
    s = (q @ k.mT) * D ** -0.5
    s = s.masked_fill(torch.ones(N, N, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
    h = (s.softmax(-1) @ v).transpose(0, 1).reshape(N, -1)
    z = h @ net["wr"].double()
    chosen = z.sigmoid().gather(1, f["idx"].long())
    weight = 2.0 * chosen / chosen.sum(1, keepdim=True)
    y = sum(weight[:, j:j + 1] * torch.bmm(h[:, None], net["we"].double()[f["idx"][:, j].long()])[:, 0]
            for j in range(K))
    want = torch.autograd.grad((y * g.double()).sum(), x)[0]
    off = (dx.double() - want).norm() / want.norm()
    assert off <= 2.0 ** -5, float(off)


def test_block_in_a_graph(st, net):
    p = dict(net)
    forward(st, p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = forward(st, p)
    for seed in (1, 2):
        p["x"].copy_(torch.randn(p["x"].shape, generator=torch.Generator("cuda").manual_seed(seed),
                                 device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        direct = forward(st, p)
        for name in ("o", "lse", "w", "idx", "token", "prob"):
            assert torch.equal(f[name], direct[name]), (name, seed)
