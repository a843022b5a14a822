"""Gated delta rule (ttt.delta, ttt.delta_backward, ttt.delta_step) against the recurrence token by
token in 64 bits, and the gradient against automatic differentiation of that recurrence and against
differences of the call itself.

Tolerances (relative 2-norm over a tensor).  A bf16 output is rounded once: at most eps/2 = 2^-8 of each
element.  Its inputs are exact, and operands of at least 17 bits (two bf16 parts) stand before it: a product
of two such operands is off by at most 3 * 2^-17 of the sum of its terms' sizes, and an output is reached
through at most five of them in a row (K W0^T, T, the states' update, A U and Q W0^T): 15 * 2^-17 = 1.2e-4
worst, were all errors alike.  They are independent over the 64 to 256 terms of a product, so the 2-norm
stays below a tenth of it, and fp32 results (states, rate gradients) are held to 2e-5 (their operands carry
24 bits, three parts: they come to 3e-7).  fp32 tokens run on 24 bits throughout, as fp32 products have:
five of up to 256 terms, 5 * 256 * 2^-24 = 7.6e-5 worst, by the same argument held to 5e-6.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: {torch.bfloat16: 2.0 ** -8, torch.float32: 2e-5},
       torch.float32: {torch.float32: 5e-6}}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from test_weight_layers_amd import ttt
    ttt.load()


def rel(x, ref):
    x, ref = x.double().cpu(), ref.double().cpu()
    assert torch.isfinite(x).all()
    d, n = (x - ref).norm().item(), ref.norm().item()
    return d / n if n else d


def inputs(lens, H, Hk, dk, dv, dtype, seed=0, tail=0, rate=0.2):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    n = sum(lens) + tail
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    d = dict(q=unit(rn(n, Hk, dk)).reshape(n, Hk * dk), k=unit(rn(n, Hk, dk)).reshape(n, Hk * dk), v=rn(n, H * dv),
             go=rn(n, H * dv))
    d = {x: t.to(dtype) for x, t in d.items()}
    d["beta"] = torch.sigmoid(rn(H, n)).float()
    d["decay"] = (-rate * torch.exp(rn(H, n))).float()
    d["w"] = (rn(len(lens), H, dv, dk) / math.sqrt(dk)).float()
    d["gw"] = (rn(len(lens), H, dv, dk) / math.sqrt(dk)).float()
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    d["cu"] = torch.tensor(cu, dtype=torch.int32)
    return d


def dev(d):
    return {k: v.cuda() for k, v in d.items()}


def recurrence(w, q, k, v, beta, decay, cu, Hk, scale=1.0):
    """Token by token in 64 bits on the CPU; differentiable."""
    S, H, dv, dk = w.shape
    n = q.shape[0]
    qh, kh, vh = q.view(n, Hk, dk), k.view(n, Hk, dk), v.view(n, H, dv)
    qh, kh = qh.repeat_interleave(H // Hk, 1), kh.repeat_interleave(H // Hk, 1)
    outs, states = [torch.zeros(H, dv, dtype=torch.float64)] * n, []
    for s in range(S):
        W = w[s]
        for t in range(cu[s], cu[s + 1]):
            W = W * torch.exp(decay[:, t])[:, None, None]
            e = vh[t] - (W * kh[t][:, None, :]).sum(-1)
            W = W + (beta[:, t, None] * e)[:, :, None] * kh[t][:, None, :]
            outs[t] = scale * (W * qh[t][:, None, :]).sum(-1)
        states.append(W)
    return torch.stack(outs).reshape(n, H * dv) if n else v, torch.stack(states)


def reference(d, Hk, scale=1.0, gradient=False):
    f = {x: d[x].double() for x in ("w", "q", "k", "v", "beta", "decay")}
    if gradient:
        for t in f.values():
            t.requires_grad_(True)
    o, w = recurrence(f["w"], f["q"], f["k"], f["v"], f["beta"], f["decay"], d["cu"].tolist(), Hk, scale)
    if not gradient:
        return o, w
    loss = (o * d["go"].double()).sum() + (w * d["gw"].double()).sum()
    names = ("q", "k", "v", "beta", "decay", "w")
    return torch.autograd.grad(loss, [f[x] for x in names])


CASES = [
    # lengths, H, Hk, dk, dv
    ([1], 1, 1, 64, 64),
    ([64], 2, 1, 64, 64),
    ([65], 1, 1, 128, 64),
    ([63, 0, 1, 130], 2, 2, 64, 128),
    ([0, 200], 3, 1, 128, 192),
    ([129, 64, 0], 2, 2, 256, 64),
    ([7, 1, 1, 300], 4, 2, 128, 128),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, dtype):
    from test_weight_layers_amd import ttt
    lens, H, Hk, dk, dv = case
    d = inputs(lens, H, Hk, dk, dv, dtype)
    o_ref, w_ref = reference(d, Hk, 0.7)
    g = dev(d)
    o, w = ttt.delta(g["w"], g["q"], g["k"], g["v"], g["beta"], g["decay"], key_heads=Hk, cu_seqlens=g["cu"], scale=0.7)
    assert rel(o, o_ref) <= TOL[dtype][dtype] and rel(w, w_ref) <= TOL[dtype][torch.float32]
    # in place on the states, and the same bits again
    w2 = g["w"].clone()
    o2, _ = ttt.delta(w2, g["q"], g["k"], g["v"], g["beta"], g["decay"], key_heads=Hk, cu_seqlens=g["cu"], scale=0.7,
                      w_out=w2)
    assert torch.equal(o, o2) and torch.equal(w, w2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case, dtype):
    from test_weight_layers_amd import ttt
    lens, H, Hk, dk, dv = case
    d = inputs(lens, H, Hk, dk, dv, dtype, seed=1)
    ref = reference(d, Hk, 0.7, gradient=True)
    g = dev(d)
    got = ttt.delta_backward(g["w"], g["q"], g["k"], g["v"], g["beta"], g["decay"], g["go"], g["gw"], key_heads=Hk,
                             cu_seqlens=g["cu"], scale=0.7)
    err = {}
    for name, x, r in zip(("q", "k", "v", "beta", "decay", "w"), got, ref):
        err[name] = (rel(x, r), TOL[dtype][x.dtype])
    print({k: f"{v[0]:.1e}" for k, v in err.items()})
    assert all(a <= b for a, b in err.values()), err


@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "decay", "w"])
def test_backward_against_differences(name):
    """Central differences of the fp32 call along one direction.  Both calls' outputs carry rounding of
    about 1e-6 of the loss' terms; at a step of 2^-6 the quotient is off by that over the step, and by
    the third derivative times step^2 / 6: 2e-3 of the gradient's norm covers both."""
    from test_weight_layers_amd import ttt
    d = inputs([70, 31], 2, 1, 64, 64, torch.float32, seed=2)
    g = dev(d)
    args = ("w", "q", "k", "v", "beta", "decay")
    grads = ttt.delta_backward(*[g[x] for x in args], g["go"], g["gw"], key_heads=1, cu_seqlens=g["cu"])
    grad = dict(zip(("q", "k", "v", "beta", "decay", "w"), grads))[name].double()
    u = torch.randn(grad.shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64).cuda()
    u = u / u.norm() + grad / grad.norm()
    u /= u.norm()

    def loss(h):
        a = dict(g)
        a[name] = (g[name].double() + h * u).float()
        o, w = ttt.delta(*[a[x] for x in args], key_heads=1, cu_seqlens=g["cu"])
        return (o.double() * g["go"].double()).sum().item() + (w.double() * g["gw"].double()).sum().item()

    h = 2.0 ** -6
    diff = (loss(h) - loss(-h)) / (2 * h)
    want = (grad * u).sum().item()
    assert abs(diff - want) <= 2e-3 * grad.norm().item(), (diff, want)


def test_repeated_keys_and_full_rates():
    """Equal keys at beta = 1 without decay: L is all ones below the diagonal, whose powers reach 1e17;
    the recurrence simply replaces the stored value."""
    from test_weight_layers_amd import ttt
    d = inputs([150], 1, 1, 64, 64, torch.float32, seed=4)
    d["k"] = d["k"][:1].expand(150, -1).contiguous()
    d["beta"].fill_(1.0)
    d["decay"].zero_()
    ref = reference(d, 1)
    gref = reference(d, 1, gradient=True)
    g = dev(d)
    for decay in (g["decay"], None):
        o, w = ttt.delta(g["w"], g["q"], g["k"], g["v"], g["beta"], decay)
        assert rel(o, ref[0]) <= 5e-6 and rel(w, ref[1]) <= 5e-6
        got = ttt.delta_backward(g["w"], g["q"], g["k"], g["v"], g["beta"], decay, g["go"], g["gw"])
        for i in (0, 1, 2, 5):
            # the values cancel down to their differences: 150 terms of the size of the largest
            assert rel(got[i], gref[i]) <= 5e-5
        if decay is None:
            assert got[4] is None


def test_decay_that_forgets_everything():
    from test_weight_layers_amd import ttt
    d = inputs([100], 2, 2, 64, 64, torch.float32, seed=5)
    d["decay"][:, 40] = -math.inf       # a reset
    d["decay"][:, 70:75] = -1e4
    d["w"][0, 0, 0, 0] = 3e30           # gone after the reset
    o_ref, w_ref = reference(d, 2)
    gref = reference(d, 2, gradient=True)
    g = dev(d)
    o, w = ttt.delta(g["w"], g["q"], g["k"], g["v"], g["beta"], g["decay"])
    assert rel(w, w_ref) <= 5e-6 and rel(o[40:], o_ref[40:]) <= 5e-6
    d["w"][0, 0, 0, 0] = 0.0
    gref = reference(d, 2, gradient=True)
    g = dev(d)
    got = ttt.delta_backward(g["w"], g["q"], g["k"], g["v"], g["beta"], g["decay"], g["go"], g["gw"])
    for i in range(6):
        # autograd gives 0 * -inf-free gradients: a decayed state has gradient 0
        assert rel(got[i], gref[i]) <= 2e-5, i


def test_rows_outside_the_sequences_and_strides():
    """Packed q, k, v as slices of one buffer, padded rows behind the last sequence, wider rate tensors."""
    from test_weight_layers_amd import ttt
    lens, H, Hk, dk, dv = [33, 70], 2, 1, 64, 64
    d = inputs(lens, H, Hk, dk, dv, torch.bfloat16, seed=6, tail=9)
    n = sum(lens) + 9
    buf = torch.full((n, 2 * Hk * dk + H * dv + 8), float("nan"), dtype=torch.bfloat16)
    q, k, v = buf[:, :64], buf[:, 64:128], buf[:, 128:128 + H * dv]
    q.copy_(d["q"]), k.copy_(d["k"]), v.copy_(d["v"])
    for t in (q, k, v):
        t[sum(lens):] = float("nan")    # padding is never read
    rates = torch.full((H, n + 5), float("nan"))
    rates[:, :sum(lens)] = d["beta"][:, :sum(lens)]
    d["decay"][:, sum(lens):] = float("nan")
    ref = reference({**d, "q": d["q"], "beta": d["beta"]}, Hk)
    buf, g = buf.cuda(), dev(d)
    q, k, v = buf[:, :64], buf[:, 64:128], buf[:, 128:128 + H * dv]
    out = torch.full((n, H * dv + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    o, w = ttt.delta(g["w"], q, k, v, rates.cuda(), g["decay"], key_heads=Hk, cu_seqlens=g["cu"], out=out[:, :H * dv])
    m = sum(lens)
    assert rel(out[:m, :H * dv], ref[0][:m]) <= 2.0 ** -8 and rel(w, ref[1]) <= 2e-5
    assert (out[m:] == 7.0).all() and (out[:, H * dv:] == 7.0).all()
    o2, _ = ttt.delta(g["w"], q, k, v, rates.cuda(), g["decay"], key_heads=Hk, cu_seqlens=g["cu"])
    assert torch.equal(o2[:m], out[:m, :H * dv]) and (o2[m:] == 0).all()
    gbuf = torch.full((n, 2 * 64 + H * dv), 5.0, dtype=torch.bfloat16, device="cuda")
    gq, gk, gv = gbuf[:, :64], gbuf[:, 64:128], gbuf[:, 128:]
    go = g["go"].clone()
    go[m:] = float("nan")
    got = ttt.delta_backward(g["w"], q, k, v, rates.cuda(), g["decay"], go, g["gw"], key_heads=Hk, cu_seqlens=g["cu"],
                             out=(gq, gk, gv))
    d2 = inputs(lens, H, Hk, dk, dv, torch.bfloat16, seed=6, tail=9)
    gref = reference({**d2, "go": torch.cat([d2["go"][:m], torch.zeros_like(d2["go"][m:])])}, Hk, gradient=True)
    for i in range(6):
        assert rel(got[i], gref[i]) <= TOL[torch.bfloat16][got[i].dtype], i
    assert (gbuf[m:] == 0).all() and (got[3][:, m:] == 0).all() and (got[4][:, m:] == 0).all()


def test_shared_rates_sum_their_gradient():
    from test_weight_layers_amd import ttt
    d = inputs([90], 3, 3, 64, 64, torch.float32, seed=7)
    d["beta"], d["decay"] = d["beta"][:1].expand(3, -1), d["decay"][:1].expand(3, -1)
    gref = reference({k: v.contiguous() for k, v in d.items()}, 3, gradient=True)
    g = dev({k: v.contiguous() for k, v in d.items()})
    beta, decay = g["beta"][0].contiguous(), g["decay"][0].contiguous()
    got = ttt.delta_backward(g["w"], g["q"], g["k"], g["v"], beta, decay, g["go"], g["gw"])
    assert got[3].shape == (90,) and got[4].shape == (90,)
    assert rel(got[3], gref[3].sum(0)) <= 2e-5 and rel(got[4], gref[4].sum(0)) <= 2e-5
    # the same rates as a [H, n] view of stride 0: a gradient for each head
    got = ttt.delta_backward(g["w"], g["q"], g["k"], g["v"], beta.expand(3, -1), decay.expand(3, -1), g["go"], g["gw"])
    assert rel(got[3], gref[3]) <= 2e-5 and rel(got[4], gref[4]) <= 2e-5


def test_offsets_out_of_order_stay_inside():
    """Offsets that run backwards or past the rows name empty or clipped sequences."""
    from test_weight_layers_amd import ttt
    d = inputs([20, 20, 20, 20], 1, 1, 64, 64, torch.float32, seed=8)
    g = dev(d)
    bad = torch.tensor([-5, 30, 10, 1000, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    same = torch.tensor([0, 30, 30, 80, 80], dtype=torch.int32, device="cuda")
    a = ttt.delta(g["w"], g["q"], g["k"], g["v"], g["beta"], g["decay"], cu_seqlens=bad)
    b = ttt.delta(g["w"], g["q"], g["k"], g["v"], g["beta"], g["decay"], cu_seqlens=same)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(b[1][1], g["w"][1]) and torch.equal(b[1][3], g["w"][3])


def test_many_short_sequences():
    from test_weight_layers_amd import ttt
    lens = [(7 * i) % 5 for i in range(700)]
    d = inputs(lens, 1, 1, 64, 64, torch.float32, seed=9)
    o_ref, w_ref = reference(d, 1)
    g = dev(d)
    o, w = ttt.delta(g["w"], g["q"], g["k"], g["v"], g["beta"], g["decay"], cu_seqlens=g["cu"])
    assert rel(o, o_ref) <= 5e-6 and rel(w, w_ref) <= 5e-6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64, 64), (5, 4, 2, 128, 192), (3, 2, 2, 256, 64)], ids=str)
def test_step(shape, dtype):
    from test_weight_layers_amd import ttt
    n, H, Hk, dk, dv = shape
    d = inputs([1] * n, H, Hk, dk, dv, dtype, seed=10)
    o_ref, w_ref = reference(d, Hk, 0.5)
    g = dev(d)
    pool = torch.randn(n + 4, H, dv, dk, device="cuda")
    slots = torch.randperm(n + 4, device="cuda")[:n].to(torch.int32)
    pool[slots.long()] = g["w"]
    before = pool.clone()
    o = ttt.delta_step(pool, g["q"], g["k"], g["v"], g["beta"], g["decay"], slots=slots, key_heads=Hk, scale=0.5)
    assert rel(o, o_ref) <= TOL[dtype][dtype]
    # one fp32 product of up to 256 terms and an update
    assert rel(pool[slots.long()], w_ref) <= 1e-6
    rest = torch.ones(n + 4, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert torch.equal(pool[rest], before[rest])
    w = g["w"].clone()
    o2 = ttt.delta_step(w, g["q"], g["k"], g["v"], g["beta"], g["decay"], key_heads=Hk, scale=0.5)
    assert torch.equal(o, o2) and torch.equal(w, pool[slots.long()])


def test_step_repeated_and_padded_slots():
    """Rows of one state apply in row order; slots outside the pool are padding."""
    from test_weight_layers_amd import ttt
    order = [2, -1, 0, 2, 5, 2, 0, 3]
    n = len(order)
    d = inputs([1] * n, 2, 1, 64, 64, torch.float32, seed=11)
    g = dev(d)
    pool = torch.randn(4, 2, 64, 64, generator=torch.Generator().manual_seed(1)).cuda()
    want, rows = pool.clone(), torch.zeros(n, 128, device="cuda")
    for i, s in enumerate(order):
        if 0 <= s < 4:
            one = want[s:s + 1].contiguous()
            sl = slice(i, i + 1)
            rows[sl] = ttt.delta_step(one, g["q"][sl], g["k"][sl], g["v"][sl], g["beta"][:, sl], g["decay"][:, sl],
                                      key_heads=1)
            want[s] = one[0]
    slots = torch.tensor(order, dtype=torch.int32, device="cuda")
    got = pool.clone()
    o = ttt.delta_step(got, g["q"], g["k"], g["v"], g["beta"], g["decay"], slots=slots, key_heads=1)
    assert torch.equal(got, want) and torch.equal(o, rows)
    out = torch.full((n, 128), 7.0, device="cuda")
    got = pool.clone()
    ttt.delta_step(got, g["q"], g["k"], g["v"], g["beta"], g["decay"], slots=slots, key_heads=1, out=out)
    assert (out[[1, 4]] == 7.0).all() and torch.equal(out[0], rows[0])


def test_prefill_then_steps_is_the_whole_sequence():
    from test_weight_layers_amd import ttt
    d = inputs([100], 2, 2, 128, 128, torch.bfloat16, seed=12)
    g = dev(d)
    o, w = ttt.delta(g["w"], g["q"], g["k"], g["v"], g["beta"], g["decay"])
    cut = lambda t, a, b: t[a:b] if t.shape[0] == 100 else t[:, a:b]
    part = lambda a, b: [cut(g[x], a, b) for x in ("q", "k", "v", "beta", "decay")]
    o1, w1 = ttt.delta(g["w"], *part(0, 77))
    rows = [o1]
    for t in range(77, 100):
        rows.append(ttt.delta_step(w1, *part(t, t + 1)))
    # two bf16 roundings of nearly the same number differ by at most one step
    assert rel(torch.cat(rows), o) <= 2.0 ** -7 and rel(w1, w) <= 2e-5


def test_captured_and_replayed():
    from test_weight_layers_amd import ttt
    d = inputs([70, 0, 65], 2, 1, 64, 64, torch.bfloat16, seed=13)
    g = dev(d)
    args = [g[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    kw = dict(key_heads=1, cu_seqlens=g["cu"])
    ttt.delta(*args, **kw), ttt.delta_backward(*args, g["go"], g["gw"], **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, w = ttt.delta(*args, **kw)
        grads = ttt.delta_backward(*args, g["go"], g["gw"], **kw)
        step = ttt.delta_step(w, *[a[:3] if a.shape[0] > 3 else a[:, :3] for a in args[1:]], key_heads=1)
    for seed in (14, 15, 16):
        new = dev(inputs([70, 0, 65], 2, 1, 64, 64, torch.bfloat16, seed=seed))
        for x in ("w", "q", "k", "v", "beta", "decay", "go", "gw"):
            g[x].copy_(new[x])
        graph.replay()
        e = [new[x] for x in ("w", "q", "k", "v", "beta", "decay")]
        o2, w2 = ttt.delta(*e, **kw)
        grads2 = ttt.delta_backward(*e, new["go"], new["gw"], **kw)
        step2 = ttt.delta_step(w2, *[a[:3] if a.shape[0] > 3 else a[:, :3] for a in e[1:]], key_heads=1)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(w, w2) and torch.equal(step, step2)
        assert all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_refusals():
    from test_weight_layers_amd import ttt
    d = dev(inputs([40, 40], 2, 2, 64, 64, torch.bfloat16, seed=17))
    w, q, k, v, be, de, cu = (d[x] for x in ("w", "q", "k", "v", "beta", "decay", "cu"))
    with pytest.raises(ValueError, match="cu_seqlens"):
        ttt.delta(w, q, k, v, be, de)
    with pytest.raises(ValueError, match="int32"):
        ttt.delta(w, q, k, v, be, de, cu_seqlens=cu.long())
    with pytest.raises(ValueError, match="float32"):
        ttt.delta(w.bfloat16(), q, k, v, be, de, cu_seqlens=cu)
    with pytest.raises(ValueError, match="dtype"):
        ttt.delta(w, q, k.float(), v, be, de, cu_seqlens=cu)
    with pytest.raises(ttt.TTTError, match="multiple of key_heads"):
        ttt.delta_workspace_bytes(2, 3, 64, 64, 80, 2, torch.bfloat16)
    with pytest.raises(ttt.TTTError, match="dk=96"):
        ttt.delta_workspace_bytes(2, 2, 96, 64, 80, 2, torch.bfloat16)
    with pytest.raises(ttt.TTTError, match="dv=96"):
        ttt.delta_workspace_bytes(2, 2, 64, 96, 80, 2, torch.bfloat16)
    with pytest.raises(ttt.TTTError, match="overlap"):
        ttt.delta(w, q, k, v, be, de, cu_seqlens=cu, out=v)
    with pytest.raises(ttt.TTTError, match="workspace"):
        ttt.delta(w, q, k, v, be, de, cu_seqlens=cu, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="must be on"):
        ttt.delta(w, q, k, v, be.cpu(), de, cu_seqlens=cu)
    with pytest.raises(ttt.TTTError, match="slots"):
        ttt.delta_step(w, q, k, v, be, de)
    with pytest.raises(ValueError, match="slots"):
        ttt.delta_step(w, q, k, v, be, de, slots=cu)


def test_no_rows_and_no_sequences_with_rows():
    from test_weight_layers_amd import ttt
    d = dev(inputs([0, 0, 0], 2, 1, 64, 64, torch.bfloat16, seed=18))
    args = [d[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    o, w = ttt.delta(*args, key_heads=1, cu_seqlens=d["cu"])
    assert o.shape == (0, 128) and torch.equal(w, d["w"])
    got = ttt.delta_backward(*args, d["go"], d["gw"], key_heads=1, cu_seqlens=d["cu"])
    assert got[0].shape == (0, 64) and torch.equal(got[5], d["gw"])
    got = ttt.delta_backward(*args, d["go"], None, key_heads=1, cu_seqlens=d["cu"])
    assert (got[5] == 0).all()
    assert ttt.delta_step(d["w"], *args[1:], key_heads=1).shape == (0, 128)
    # rows, but every sequence empty
    d = dev(inputs([20], 2, 1, 64, 64, torch.bfloat16, seed=19))
    cu = torch.tensor([7, 7], dtype=torch.int32, device="cuda")
    args = [d[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    o, w = ttt.delta(*args, key_heads=1, cu_seqlens=cu)
    assert (o == 0).all() and torch.equal(w, d["w"])
    got = ttt.delta_backward(*args, d["go"], d["gw"], key_heads=1, cu_seqlens=cu)
    assert all((got[i] == 0).all() for i in range(5)) and torch.equal(got[5], d["gw"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_wide_values(dtype):
    from test_weight_layers_amd import ttt
    d = inputs([100], 1, 1, 64, 1024, dtype, seed=20)
    o_ref, w_ref = reference(d, 1)
    gref = reference(d, 1, gradient=True)
    g = dev(d)
    args = [g[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    o, w = ttt.delta(*args)
    assert rel(o, o_ref) <= TOL[dtype][dtype] and rel(w, w_ref) <= TOL[dtype][torch.float32]
    got = ttt.delta_backward(*args, g["go"], g["gw"])
    for x, r in zip(got, gref):
        assert rel(x, r) <= TOL[dtype][x.dtype]


def test_sequences_do_not_reach_each_other():
    """A NaN in one sequence leaves the others' bits."""
    from test_weight_layers_amd import ttt
    d = dev(inputs([40, 30, 50], 1, 1, 64, 64, torch.bfloat16, seed=21))
    args = [d[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    ref = ttt.delta(*args, cu_seqlens=d["cu"])
    gref = ttt.delta_backward(*args, d["go"], d["gw"], cu_seqlens=d["cu"])
    for x in ("q", "k", "v", "go"):
        d[x][45] = float("nan")
    d["beta"][:, 46], d["decay"][:, 47] = float("nan"), float("nan")
    o, w = ttt.delta(*args, cu_seqlens=d["cu"])
    got = ttt.delta_backward(*args, d["go"], d["gw"], cu_seqlens=d["cu"])
    keep = torch.ones(120, dtype=torch.bool, device="cuda")
    keep[40:70] = False
    assert torch.equal(o[keep], ref[0][keep]) and torch.equal(w[[0, 2]], ref[1][[0, 2]])
    for i in range(3):
        assert torch.equal(got[i][keep], gref[i][keep])
    for i in (3, 4):
        assert torch.equal(got[i][:, keep], gref[i][:, keep])
    assert torch.equal(got[5][[0, 2]], gref[5][[0, 2]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,H,Hk,dk,dv", [([2000], 1, 1, 64, 64), ([1537], 2, 1, 128, 192), ([1700], 1, 1, 256, 64),
                                             ([2500, 0, 1, 70, 1900], 1, 1, 64, 64), ([0, 64, 1601], 1, 1, 64, 128)])
def test_long_sequences(lens, H, Hk, dk, dv, dtype):
    """Few long sequences, whose segments run at once and are joined; short and empty ones beside them."""
    from test_weight_layers_amd import ttt
    d = inputs(lens, H, Hk, dk, dv, dtype, seed=22, tail=3, rate=0.02)
    o_ref, w_ref = reference(d, Hk)
    g = dev(d)
    args = [g[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    o, w = ttt.delta(*args, key_heads=Hk, cu_seqlens=g["cu"])
    assert rel(o, o_ref) <= TOL[dtype][dtype]
    for s in range(len(lens)):
        assert rel(w[s], w_ref[s]) <= TOL[dtype][torch.float32], s
    assert torch.equal(ttt.delta(*args, key_heads=Hk, cu_seqlens=g["cu"])[1], w)
    ttt.delta(*args, key_heads=Hk, cu_seqlens=g["cu"], w_out=g["w"])
    assert torch.equal(g["w"], w)


def test_long_sequence_keeps_nan_to_its_rows():
    """Not a number in a value or a starting state stays in that row of the state, through the joins too."""
    from test_weight_layers_amd import ttt
    d = dev(inputs([3000], 1, 1, 64, 64, torch.float32, seed=23, rate=0.02))
    args = [d[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    ref = ttt.delta(*args)
    d["v"][700, 5], d["w"][0, 0, 40, 3] = float("nan"), float("inf")
    o, w = ttt.delta(*args)
    keep = torch.ones(64, dtype=torch.bool, device="cuda")
    keep[5] = keep[40] = False
    assert torch.equal(w[0, 0][keep], ref[1][0, 0][keep]) and not torch.isfinite(w[0, 0, [5, 40]]).any()
    assert torch.equal(o[:, keep], ref[0][:, keep]) and torch.equal(o[:640, 5], ref[0][:640, 5])    # 640: its chunk
    assert not torch.isfinite(o[700:, 5]).any() and not torch.isfinite(o[:, 40]).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,H,Hk,dk,dv", [([1537], 2, 1, 64, 64), ([1300], 1, 1, 128, 192), ([1900], 1, 1, 256, 64),
                                             ([2200, 0, 1, 70, 1500], 1, 1, 64, 64), ([0, 64, 1601], 1, 1, 64, 128)])
def test_long_sequences_backward(lens, H, Hk, dk, dv, dtype):
    from test_weight_layers_amd import ttt
    d = inputs(lens, H, Hk, dk, dv, dtype, seed=24, tail=3, rate=0.02)
    ref = reference(d, Hk, gradient=True)
    g = dev(d)
    args = [g[x] for x in ("w", "q", "k", "v", "beta", "decay", "go", "gw")]
    got = ttt.delta_backward(*args, key_heads=Hk, cu_seqlens=g["cu"])
    for name, x, r in zip(("q", "k", "v", "beta", "decay", "w"), got, ref):
        assert rel(x, r) <= TOL[dtype][x.dtype], name
        assert name == "w" or (x[-3:] if name in "qkv" else x[:, -3:]).abs().max() == 0
    for s in range(len(lens)):
        assert rel(got[5][s], ref[5][s]) <= TOL[dtype][torch.float32], s
    again = ttt.delta_backward(*args, key_heads=Hk, cu_seqlens=g["cu"])
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_long_sequences_captured_and_replayed():
    """Segments are laid out on the device: other lengths at a replay are other segments."""
    from test_weight_layers_amd import ttt
    d = dev(inputs([1500, 700], 1, 1, 64, 64, torch.bfloat16, seed=25, rate=0.02))
    args = [d[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    run = lambda: (*ttt.delta(*args, cu_seqlens=d["cu"]),
                   *ttt.delta_backward(*args, d["go"], d["gw"], cu_seqlens=d["cu"]))
    for _ in range(2):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for i, cut in enumerate([1500, 0, 2200, 64, 1301, 1500]):
        d["cu"][1] = cut
        d["v"].mul_(1.0 if i % 2 else -0.5)
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), cut


def test_long_sequences_with_offsets_out_of_order():
    """Any offsets name disjoint rows, in segments too: clamped to the rows and to a running maximum."""
    from test_weight_layers_amd import ttt
    d = dev(inputs([1400, 600, 100], 1, 1, 64, 64, torch.bfloat16, seed=26, rate=0.02))
    args = [d[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    for cu, same in (([0, 1800, 900, 1 << 30], [0, 1800, 1800, 2100]), ([-5, 1400, -7, 2000], [0, 1400, 1400, 2000]),
                     ([500, 300, 2100, 2100], [500, 500, 2100, 2100])):
        a, b = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, same))
        got = (*ttt.delta(*args, cu_seqlens=a), *ttt.delta_backward(*args, d["go"], d["gw"], cu_seqlens=a))
        want = (*ttt.delta(*args, cu_seqlens=b), *ttt.delta_backward(*args, d["go"], d["gw"], cu_seqlens=b))
        assert all(torch.equal(x, y) for x, y in zip(got, want)), cu


def test_many_sequences_backward():
    """More sequences than a wave lays out for itself, empty ones among them."""
    from test_weight_layers_amd import ttt
    lens = [3, 0, 70, 1] * 17 + [64]
    d = inputs(lens, 2, 1, 64, 64, torch.float32, seed=27, tail=2)
    ref = reference(d, 1, gradient=True)
    g = dev(d)
    got = ttt.delta_backward(*[g[x] for x in ("w", "q", "k", "v", "beta", "decay", "go", "gw")], key_heads=1,
                             cu_seqlens=g["cu"])
    for x, r in zip(got, ref):
        assert rel(x, r) <= TOL[torch.float32][torch.float32]
