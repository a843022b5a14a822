"""A block as the models around the layer have it, of the library's parts: layer norm, projections (torch), a norm of every
head's q and k, windowed attention, the gated residual tail; its gradients, its training step (orthogonalised for
the matrices, AdamW for the rest), replayed from a graph; and the same block token by token over a rolling cache.

Tolerances: fp32 throughout.  The parts' own tests hold each to 2^-16 at most; the projections (torch, fp32 sums of 128
terms) and five parts after one another, whose errors add: 8 * 2^-16 for outputs and gradients.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

H, HK, D, C, N = 4, 2, 64, 128, 200
LENS = [90, 0, 1, 109]
MASK = dict(block=4, before=6, after=0, sinks=8)
TOL = 8 * 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from test_weight_layers_amd import ttt
    ttt.load()


def parameters(seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    return dict(g1=1 + 0.1 * rn(C), b1=0.1 * rn(C), wqkv=rn(C, (H + 2 * HK) * D) / C ** 0.5, gq=1 + 0.1 * rn(D), gk=1 + 0.1 * rn(D),
                wo=rn(H * D, C) / (H * D) ** 0.5, gr=1 + 0.1 * rn(C), ga=0.5 + 0.1 * rn(C))


def forward(p, x, cu):
    """Everything that the gradient needs."""
    from test_weight_layers_amd import ttt
    s = {"x": x}
    s["h"] = ttt.layer_norm(x, p["g1"], p["b1"])
    s["qkv"] = s["h"] @ p["wqkv"]
    s["q"] = ttt.layer_norm(s["qkv"][:, :H * D], p["gq"], norm_width=D)
    s["k"] = ttt.layer_norm(s["qkv"][:, H * D:(H + HK) * D], p["gk"], norm_width=D)
    s["v"] = s["qkv"][:, (H + HK) * D:]
    s["o"], s["lse"] = ttt.window_attention(s["q"], s["k"], s["v"], heads=H, key_heads=HK, cu_seqlens=cu, **MASK)
    s["u"] = s["o"] @ p["wo"]
    s["y"], _ = ttt.gated_residual(x, s["u"], None, p["gr"], p["ga"])
    return s


def backward(p, s, gy, cu):
    from test_weight_layers_amd import ttt
    g = {}
    gx, gu, _, g["gr"], g["ga"], _ = ttt.gated_residual_backward(gy, None, s["y"], s["u"], None, p["gr"], p["ga"])
    g["wo"] = s["o"].t() @ gu
    go = gu @ p["wo"].t()
    gqkv = torch.empty_like(s["qkv"])
    parts = (gqkv[:, :H * D], gqkv[:, H * D:(H + HK) * D], gqkv[:, (H + HK) * D:])
    ttt.window_attention_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], go, heads=H, key_heads=HK, cu_seqlens=cu, out=parts, **MASK)
    _, g["gq"], _ = ttt.layer_norm_backward(parts[0], s["qkv"][:, :H * D], p["gq"], norm_width=D, out=parts[0])
    _, g["gk"], _ = ttt.layer_norm_backward(parts[1], s["qkv"][:, H * D:(H + HK) * D], p["gk"], norm_width=D, out=parts[1])
    g["wqkv"] = s["h"].t() @ gqkv
    gh, g["g1"], g["b1"] = ttt.layer_norm_backward(gqkv @ p["wqkv"].t(), s["x"], p["g1"])
    return gx + gh, g


def reference(p, x):
    """The same in elementary operations."""
    def norm(t, gamma, beta, w):
        t = t.unflatten(1, (-1, w))
        c = t - t.mean(-1, keepdim=True)
        return (c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-6) * gamma + beta).flatten(1)

    qkv = norm(x, p["g1"], p["b1"], C) @ p["wqkv"]
    q, k, v = norm(qkv[:, :H * D], p["gq"], 0, D), norm(qkv[:, H * D:(H + HK) * D], p["gk"], 0, D), qkv[:, (H + HK) * D:]
    outs, a = [], 0
    for n in LENS:
        i, j = torch.arange(n, device=x.device)[:, None], torch.arange(n, device=x.device)[None, :]
        b = i // MASK["block"]
        ok = (j < (b + 1) * MASK["block"]) & ((j >= (b - MASK["before"]) * MASK["block"]) | (j < MASK["sinks"]))
        qs = q[a:a + n].view(n, H, D).transpose(0, 1)
        ks, vs = (t[a:a + n].view(n, HK, D).transpose(0, 1).repeat_interleave(H // HK, 0) for t in (k, v))
        w = torch.softmax((qs @ ks.transpose(1, 2) / D ** 0.5).masked_fill(~ok, float("-inf")), -1)
        outs.append((w @ vs).transpose(0, 1).reshape(n, H * D))
        a += n
    u = torch.cat(outs) @ p["wo"]
    return x + p["ga"] * p["gr"] * u / torch.sqrt((u * u).mean(-1, keepdim=True) + 1e-6)


def rel(x, ref):
    assert torch.isfinite(x).all()
    return ((x.double() - ref.double()).norm() / ref.double().norm()).item()


def test_block_and_its_gradients():
    p = {k: v.cuda() for k, v in parameters().items()}
    g = torch.Generator().manual_seed(9)
    x, gy = torch.randn(N, C, generator=g).cuda(), torch.randn(N, C, generator=g).cuda()
    cu = torch.tensor([0] + LENS).cumsum(0).to(torch.int32).cuda()
    s = forward(p, x, cu)
    gx, grads = backward(p, s, gy, cu)
    leaves = {k: v.double().requires_grad_(True) for k, v in {**p, "x": x}.items()}
    y = reference(leaves, leaves["x"])
    ref = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), gy.double())))
    assert rel(s["y"], y.detach()) <= TOL
    for k, v in {**grads, "x": gx}.items():
        assert rel(v, ref[k]) <= TOL, k


@pytest.mark.parametrize("bits", [32, 8])
def test_training_step_from_a_graph(bits):
    """A captured step against the eager one, replayed with other inputs between eager work; graphs of two programs that
    were captured one after the other keep workspaces of their own."""
    from test_weight_layers_amd import ttt
    cu = torch.tensor([0] + LENS).cumsum(0).to(torch.int32).cuda()
    matrices, rest = ("wqkv", "wo"), ("g1", "b1", "gq", "gk", "gr", "ga")

    def program(seed):
        p = {k: v.cuda() for k, v in parameters(seed).items()}
        w = [p[k] for k in rest]
        if bits == 32:
            opt = ttt.adamw_tensors(w, [torch.zeros_like(x) for x in w], [torch.zeros_like(x) for x in w])
        else:
            scales = lambda: [torch.zeros(-(-x.numel() // 256), device="cuda") for x in w]
            opt = ttt.adamw_tensors(w, [torch.zeros_like(x, dtype=torch.int8) for x in w],
                                    [torch.zeros_like(x, dtype=torch.uint8) for x in w], exp_avg_scales=scales(),
                                    exp_avg_sq_scales=scales())
        t = torch.zeros(1, dtype=torch.int64, device="cuda")

        def step(x, gy):
            s = forward(p, x, cu)
            gx, g = backward(p, s, gy, cu)
            t.add_(1)
            ttt.adamw_step(opt, [g[k] for k in rest], step=t, lr=1e-2, weight_decay=0.01)
            for k in matrices:
                p[k].sub_(0.02 * ttt.orthogonalise(g[k]))
            return s["y"], gx

        return p, step

    g = torch.Generator().manual_seed(11)
    x, gy = torch.randn(N, C, generator=g).cuda(), torch.randn(N, C, generator=g).cuda()
    p1, eager = program(1)
    captured = []
    eager(x, gy)                                         # (one eager step first, in every program)
    for _ in range(2):
        p2, step = program(1)
        step(x, gy)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(x, gy)
        captured.append((p2, step, graph, out))      # (the step holds the states)
    for _ in range(3):
        x.copy_(torch.randn(N, C, generator=g)), gy.copy_(torch.randn(N, C, generator=g))
        ref = eager(x, gy)
        for p2, _, graph, out in captured:
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
            off = {k: (p1[k] - p2[k]).abs().max().item() for k in p1 if not torch.equal(p1[k], p2[k])}
            assert not off, off


def test_block_token_by_token():
    """The last tokens of a stream, one at a time over a rolling cache that the prompt filled, against the whole prompt:
    sums in another order, TOL."""
    from test_weight_layers_amd import ttt
    p = {k: v.cuda() for k, v in parameters(2).items()}
    n, prompt, capacity = 120, 70, 40 + MASK["sinks"]
    x = torch.randn(n, C, generator=torch.Generator().manual_seed(5)).cuda()
    # blocks end with their last token: a prompt sees its whole block, a token what has come
    how = dict(heads=H, key_heads=HK, block=1, before=30, sinks=MASK["sinks"])

    def upto_qkv(x):
        qkv = ttt.layer_norm(x, p["g1"], p["b1"]) @ p["wqkv"]
        return (ttt.layer_norm(qkv[:, :H * D], p["gq"], norm_width=D),
                ttt.layer_norm(qkv[:, H * D:(H + HK) * D], p["gk"], norm_width=D), qkv[:, (H + HK) * D:])

    q, k, v = upto_qkv(x)
    whole, _ = ttt.gated_residual(x, ttt.window_attention(q, k, v, **how)[0] @ p["wo"], None, p["gr"], p["ga"])
    kc, vc = (torch.zeros(3, capacity, HK * D, device="cuda") for _ in range(2))
    at = torch.arange(prompt)
    keep = at[(at < MASK["sinks"]) | (at >= prompt - (capacity - MASK["sinks"]))]
    place = torch.where(keep < MASK["sinks"], keep, MASK["sinks"] + (keep - MASK["sinks"]) % (capacity - MASK["sinks"])).cuda()
    kc[1, place], vc[1, place] = k[keep.cuda()], v[keep.cuda()]
    slots = torch.tensor([1], dtype=torch.int32, device="cuda")
    for t in range(prompt, n):
        row = x[t:t + 1]
        q1, k1, v1 = upto_qkv(row)
        o = ttt.window_attention_step(kc, vc, q1, k1, v1, torch.tensor([t], dtype=torch.int32, device="cuda"), slots=slots, **how)
        y, _ = ttt.gated_residual(row, o @ p["wo"], None, p["gr"], p["ga"])
        assert rel(y, whole[t:t + 1]) <= TOL, t
