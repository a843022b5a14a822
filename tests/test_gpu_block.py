"""A fast-weight block as it is trained and served: the gated delta rule, the gated residual tail around
it, their gradients through a projection, and the projection's step by an orthogonalised gradient.

The reference is the same block in 64 bits, token by token, differentiated automatically.  fp32 tokens:
every operator is held to 5e-6 to 2e-5 by itself (see their tests) and the block runs each once, with
projections of 128 terms (fp32: 128 * 2^-24 = 8e-6) before and after: 1e-4 covers the sum.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from test_weight_layers_amd import ttt
    ttt.load()


def rel(x, ref):
    x, ref = x.double().cpu(), ref.double().cpu()
    assert torch.isfinite(x).all()
    return ((x - ref).norm() / ref.norm()).item()


H, DK, DV, C = 2, 64, 64, 128
CU = [0, 70, 71, 140]


def weights(dtype):
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    n = CU[-1]
    p = dict(x=rn(n, C), wq=rn(C, H * DK) / 11, wk=rn(C, H * DK) / 11, wv=rn(C, H * DV) / 11, wz=rn(C, C) / 11,
             gamma=1 + 0.1 * rn(C), alpha=0.5 + 0.1 * rn(C), gamma_next=1 + 0.1 * rn(C), beta=torch.sigmoid(rn(H, n)),
             decay=-0.1 * torch.exp(rn(H, n)), w0=rn(len(CU) - 1, H, DV, DK) / 8, gy=rn(n, C), gh=rn(n, C))
    return {k: v.to(dtype) for k, v in p.items()}


def reference(p):
    n = CU[-1]
    unit = lambda t: (t.view(n, H, DK) / t.view(n, H, DK).norm(dim=-1, keepdim=True)).reshape(n, -1)
    q, k, v, z = unit(p["x"] @ p["wq"]), unit(p["x"] @ p["wk"]), p["x"] @ p["wv"], p["x"] @ p["wz"]
    rows = []
    for s in range(len(CU) - 1):
        W = p["w0"][s]
        for t in range(CU[s], CU[s + 1]):
            W = W * torch.exp(p["decay"][:, t])[:, None, None]
            kt, vt, qt = k[t].view(H, DK), v[t].view(H, DV), q[t].view(H, DK)
            e = vt - (W * kt[:, None, :]).sum(-1)
            W = W + (p["beta"][:, t, None] * e)[:, :, None] * kt[:, None, :]
            rows.append((W * qt[:, None, :]).sum(-1).reshape(-1))
    o = torch.stack(rows)
    og = o.view(n, H, DV)
    u = (og / torch.sqrt((og * og).mean(-1, keepdim=True) + 1e-6)).reshape(n, C) * p["gamma"] * z * torch.sigmoid(z)
    y = p["x"] + p["alpha"] * u
    return y, y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * p["gamma_next"]


def test_block_trains():
    from test_weight_layers_amd import ttt
    ref = {k: v.requires_grad_(k not in ("gy", "gh")) for k, v in weights(torch.float64).items()}
    y_ref, h_ref = reference(ref)
    names = ("wq", "wk", "wv", "wz", "gamma", "alpha", "gamma_next", "beta", "decay", "w0", "x")
    grads = dict(zip(names, torch.autograd.grad((y_ref * ref["gy"]).sum() + (h_ref * ref["gh"]).sum(),
                                                [ref[x] for x in names])))
    p = {k: v.cuda() for k, v in weights(torch.float32).items()}
    n, cu = CU[-1], torch.tensor(CU, dtype=torch.int32, device="cuda")
    heads = lambda t: t.view(n, H, DK)
    q0, k0, v, z = p["x"] @ p["wq"], p["x"] @ p["wk"], p["x"] @ p["wv"], p["x"] @ p["wz"]
    qn, kn = heads(q0).norm(dim=-1, keepdim=True), heads(k0).norm(dim=-1, keepdim=True)
    q, k = (heads(q0) / qn).reshape(n, -1), (heads(k0) / kn).reshape(n, -1)
    o, w = ttt.delta(p["w0"], q, k, v, p["beta"], p["decay"], cu_seqlens=cu)
    y, h = ttt.gated_residual(p["x"], o, z, p["gamma"], p["alpha"], p["gamma_next"], 1e-6, norm_width=DV)
    assert rel(y, y_ref.detach()) <= 1e-4 and rel(h, h_ref.detach()) <= 1e-4
    gx, go, gz, gg, ga, gn = ttt.gated_residual_backward(p["gy"], p["gh"], y, o, z, p["gamma"], p["alpha"],
                                                         p["gamma_next"], 1e-6, norm_width=DV)
    gq, gk, gv, gb, gd, gw = ttt.delta_backward(p["w0"], q, k, v, p["beta"], p["decay"], go, None, cu_seqlens=cu)
    unnorm = lambda g, u, s: ((heads(g) - heads(u) * (heads(g) * heads(u)).sum(-1, keepdim=True)) / s).reshape(n, -1)
    gq, gk = unnorm(gq, q, qn), unnorm(gk, k, kn)
    got = dict(wq=p["x"].T @ gq, wk=p["x"].T @ gk, wv=p["x"].T @ gv, wz=p["x"].T @ gz, gamma=gg, alpha=ga, gamma_next=gn,
               beta=gb, decay=gd, w0=gw,
               x=gx + gq @ p["wq"].T + gk @ p["wk"].T + gv @ p["wv"].T + gz @ p["wz"].T)
    err = {x: rel(got[x], grads[x]) for x in names}
    print({k: f"{v:.1e}" for k, v in err.items()})
    assert max(err.values()) <= 1e-4, err
    # the optimiser's step on the four projections at once
    step = ttt.orthogonalise(torch.stack([got[x] for x in ("wq", "wk", "wv", "wz")]))
    for s, x in zip(step, ("wq", "wk", "wv", "wz")):
        m = grads[x] / (grads[x].norm() + 1e-7)
        for _ in range(5):
            a = m @ m.mT
            m = 3.4445 * m + (-4.7750 * a + 2.0315 * a @ a) @ m
        # the gradient's own 1e-4 is multiplied by up to 485 along directions that hold next to nothing of it
        assert rel(s, m) <= 2e-2


def test_block_serves():
    """A prompt in one call, then token by token from a pool of states, equals the prompt of both in one."""
    from test_weight_layers_amd import ttt
    g = torch.Generator().manual_seed(1)
    lens, extra = [90, 33, 1], 3
    B = len(lens)
    seqs = []
    for m in lens:
        unit = lambda t: t / t.norm(dim=-1, keepdim=True)
        seqs.append(dict(q=unit(torch.randn(m + extra, H, DK, generator=g)).reshape(-1, H * DK).bfloat16().cuda(),
                         k=unit(torch.randn(m + extra, H, DK, generator=g)).reshape(-1, H * DK).bfloat16().cuda(),
                         v=torch.randn(m + extra, H * DV, generator=g).bfloat16().cuda(),
                         beta=torch.sigmoid(torch.randn(H, m + extra, generator=g)).cuda(),
                         decay=(-0.1 * torch.rand(H, m + extra, generator=g)).cuda()))
    cat = lambda name, sl: torch.cat([s[name][sl(m)] if name in "qkv" else s[name][:, sl(m)] for s, m in zip(seqs, lens)],
                                     0 if name in "qkv" else 1).contiguous()
    args = lambda sl: [cat(x, sl) for x in ("q", "k", "v", "beta", "decay")]
    cu = lambda ls: torch.tensor([0] + ls, device="cuda").cumsum(0).to(torch.int32)
    w0 = torch.zeros(B, H, DV, DK, device="cuda")
    o_all, w_all = ttt.delta(w0, *args(lambda m: slice(0, m + extra)), cu_seqlens=cu([m + extra for m in lens]))
    pool = torch.zeros(8, H, DV, DK, device="cuda")
    slots = torch.tensor([5, 0, 3], dtype=torch.int32, device="cuda")
    o, w = ttt.delta(w0, *args(lambda m: slice(0, m)), cu_seqlens=cu(lens))
    pool[slots.long()] = w
    starts = cu([m + extra for m in lens]).tolist()
    for t in range(extra):
        row = ttt.delta_step(pool, *args(lambda m: slice(m + t, m + t + 1)), slots=slots)
        ref = torch.stack([o_all[starts[i] + lens[i] + t] for i in range(B)])
        # two bf16 roundings of nearly the same number differ by at most one step
        assert rel(row, ref) <= 2.0 ** -7
    assert rel(pool[slots.long()], w_all) <= 1e-6
    assert (pool[[1, 2, 4, 6, 7]] == 0).all()


def test_two_streams_at_once():
    from test_weight_layers_amd import ttt
    p = {k: v.cuda() for k, v in weights(torch.float32).items()}
    cu = torch.tensor(CU, dtype=torch.int32, device="cuda")
    n = CU[-1]
    q, k, v = (torch.randn(n, H * DK, device="cuda") / 8 for _ in range(3))
    big = torch.randn(3, 300, 200, device="cuda")

    def work():
        o, w = ttt.delta(p["w0"], q, k, v, p["beta"], p["decay"], cu_seqlens=cu)
        g = ttt.delta_backward(p["w0"], q, k, v, p["beta"], p["decay"], o, w, cu_seqlens=cu)
        y, h = ttt.gated_residual(p["x"], o, None, p["gamma"], p["alpha"], p["gamma_next"], norm_width=DV)
        r = ttt.gated_residual_backward(y, h, y, o, None, p["gamma"], p["alpha"], p["gamma_next"], norm_width=DV)
        return [o, w, *g, y, h, *[t for t in r if t is not None], ttt.orthogonalise(big)]

    ref = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(work())
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
