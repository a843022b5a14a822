"""Windowed attention (ttt.window_attention, its gradient, the one-token form) against the formulas in 64 bits.

Tolerances (relative 2-norm; inputs are independent normal values).
bf16, eps/2 = 2^-8 a rounding: an output is rounded once (2^-8), and every probability once as an operand: errors
e_j p_j v_j with |e_j| <= 2^-8, independent of v, add to 2^-8 of the 2-norm of the sum.  Together 2^-7.  A gradient's
dS = P (dP - delta) is rounded once, the output once, and delta comes from an o rounded to 2^-8: 3 * 2^-8.
fp32: a score is a sum of up to 256 products in 64 steps of four, each with a rounding of 2^-24 of a partial sum that is at
most about 6 (scores are sums over d of normal values, over sqrt(d)): below 64 * 6 * 2^-24 < 2^-15 at the worst and, as the
roundings are independent, about 8 * 6 * 2^-24 < 2^-18.  This absolute error is the relative one of P = e^s.  Sums over keys
are sums of such terms: 2^-17 for outputs, and 2^-16 for gradients, where dP - delta is a difference of two sums of the
same size.  lse: the absolute error of the scores, 2^-17.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 2.0 ** -7, F32: 2.0 ** -17}
GTOL = {BF: 3 * 2.0 ** -8, F32: 2.0 ** -16}


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


def mask(lq, lk, block, before, after, sinks):
    """[lq, lk] visibility."""
    p = torch.arange(lq).double()[:, None] + (lk - lq)
    j = torch.arange(lk).double()[None, :]
    b = torch.floor(p / block)
    ok = torch.ones(lq, lk, dtype=torch.bool)
    if after is not None:
        ok &= j < (b + after + 1) * block
    if before is not None:
        ok &= (j >= (b - before) * block) | (j < sinks)
    return ok


def reference(q, k, v, H, Hk, lens, lens_k, how, scale=None, grad_o=None):
    """o, lse and gradients in fp64, sequence by sequence."""
    d = q.shape[1] // H
    scale = d ** -0.5 if scale is None else scale
    q, k, v = (t.double().cuda().requires_grad_(grad_o is not None) for t in (q, k, v))
    outs, lses, a, b = [], [], 0, 0
    for lq, lk in zip(lens, lens_k):
        ok = mask(lq, lk, *how).cuda()
        qs = q[a:a + lq].view(lq, H, d).transpose(0, 1)
        ks, vs = (t[b:b + lk].view(lk, Hk, d).transpose(0, 1).repeat_interleave(H // Hk, 0) for t in (k, v))
        s = (qs @ ks.transpose(1, 2) * scale).masked_fill(~ok, -math.inf)
        any_key = ok.any(1)
        safe = s.masked_fill(~any_key[:, None], 0.0) if lk else s
        w = torch.softmax(safe, -1) * any_key[:, None] if lk else s
        outs.append((w @ vs).transpose(0, 1).reshape(lq, H * d))
        lses.append(torch.logsumexp(s, -1) if lk else s.new_full((H, lq), -math.inf))
        a, b = a + lq, b + lk
    o, lse = torch.cat(outs), torch.cat(lses, 1)
    grads = torch.autograd.grad(o, (q, k, v), grad_o.double().cuda(), allow_unused=True) if grad_o is not None else None
    return o.detach(), lse.detach(), grads


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def inputs(nq, nk, H, Hk, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, h * d, generator=g).to(dtype) for n, h in ((nq, H), (nk, Hk), (nk, Hk), (nq, H))]


def lse_off(lse, ref):
    """Absolute error; infinities have to stand at the same places."""
    lse, ref = lse.double(), ref.double()
    f = torch.isfinite(ref)
    assert torch.equal(lse[~f], ref[~f])
    return (lse - ref)[f].abs().max().item() if f.any() else 0.0


# heads, key heads, d, query lengths, key lengths, (block, before, after, sinks), dtype
CASES = [
    (1, 1, 64, [1], [1], (1, None, 0, 0), F32),
    (2, 1, 64, [1], [1], (1, 0, 0, 3), BF),
    (3, 3, 64, [37], [37], (1, None, 0, 0), BF),
    (4, 2, 128, [65], [65], (1, 16, 0, 0), F32),
    (2, 2, 256, [130], [130], (1, 40, 0, 4), BF),
    (2, 1, 256, [70], [70], (1, 20, 0, 3), F32),
    (4, 4, 64, [300], [300], (64, 0, 0, 0), BF),                 # blocks of their own
    (2, 2, 128, [200], [200], (37, 1, 1, 0), F32),               # both sides
    (2, 2, 64, [257], [257], (1, None, None, 0), BF),            # all keys
    (2, 2, 64, [129], [129], (1, 10, None, 7), F32),             # no end
    (6, 2, 64, [50, 0, 1, 333, 64], [50, 0, 1, 333, 64], (1, 99, 0, 5), BF),
    (4, 4, 128, [100, 31], [228, 31], (16, 2, 0, 20), BF),       # queries at the end of more keys
    (4, 1, 64, [1, 5, 3], [700, 0, 2000], (1, None, 0, 0), F32),      # a sequence without keys, few rows of many keys
    (2, 2, 64, [90, 10], [20, 10], (1, None, 0, 0), BF),         # queries before the first key see nothing
    (2, 1, 128, [90], [20], (8, 1, 2, 3), F32),
    (8, 8, 64, [1374], [1374], (1374, 0, 0, 0), BF),
    (1, 1, 64, [3000], [3000], (1, 63, 0, 4), BF),               # sinks that far more queries see than their window
    (4, 2, 64, [2500, 900], [2500, 900], (10, 3, 0, 300), F32),
    (2, 2, 128, [3], [9000], (1, None, 0, 0), BF),
    (2, 2, 256, [40], [3000], (100, 4, 0, 130), BF),
    # many heads: the tiles of large calls
    (128, 128, 64, [1100], [1100], (1, 200, 0, 5), BF),
    (64, 64, 64, [1100], [1100], (1, None, None, 0), BF),
    (128, 64, 64, [1100], [1100], (1, None, None, 0), F32),
    (128, 128, 64, [700, 0, 400], [700, 3, 400], (10, 3, 0, 30), F32),
    (64, 64, 128, [1100], [1100], (1, None, 0, 0), BF),
    (64, 32, 128, [600, 501], [600, 501], (1, 300, 0, 8), F32),
    (64, 32, 256, [1100], [1100], (1, None, 0, 0), BF),
    (64, 64, 256, [37, 1000], [37, 1000], (8, 20, 2, 9), BF),
    (64, 64, 256, [520], [520], (1, 100, 0, 3), F32),
    # more tiles than run at once: the last ones' keys in ranges
    (40, 20, 128, [2200], [2200], (1, None, None, 0), BF),
    (40, 40, 64, [2200], [2200], (1, 1500, 0, 10), F32),
    (60, 60, 64, [1200, 1000], [2400, 1300], (1, None, None, 0), BF),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradient(case):
    from test_weight_layers_amd import ttt
    H, Hk, d, lens, lens_k, how, dtype = case
    q, k, v, go = inputs(sum(lens), sum(lens_k), H, Hk, d, dtype)
    o_ref, lse_ref, grads_ref = reference(q, k, v, H, Hk, lens, lens_k, how, grad_o=go)
    kw = dict(heads=H, key_heads=Hk, block=how[0], before=how[1], after=how[2], sinks=how[3], cu_seqlens=offsets(lens),
              cu_seqlens_k=offsets(lens_k))
    q, k, v, go = (t.cuda() for t in (q, k, v, go))
    o, lse = ttt.window_attention(q, k, v, **kw)
    assert rel(o, o_ref) <= TOL[dtype] and lse_off(lse, lse_ref) <= 2.0 ** -17 * max(1.0, lse_ref[lse_ref > -math.inf].abs().max().item())
    grads = ttt.window_attention_backward(q, k, v, o, lse, go, **kw)
    again = ttt.window_attention_backward(q, k, v, o, lse, go, **kw)
    o2, lse2 = ttt.window_attention(q, k, v, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # where a query sees one key alone its dS is a difference of equal numbers: errors are relative to the terms
    err = {}
    for name, a, b, r, other in zip("qkv", grads, again, grads_ref, (k, q, go)):
        assert torch.equal(a, b) and torch.isfinite(a).all()
        r = torch.zeros_like(a).double() if r is None else r
        scale = max(r.norm().item(), 0.05 * go.double().norm().item())
        err[name] = (a.double() - r).norm().item() / scale
    print({x: f"{e:.1e}" for x, e in err.items()})
    assert all(e <= GTOL[dtype] for e in err.values()), err
    if len(lens) == 1:                                   # without offsets: one sequence of all rows
        del kw["cu_seqlens"], kw["cu_seqlens_k"]
        o3, lse3 = ttt.window_attention(q, k, v, **kw)
        assert rel(o3, o_ref) <= TOL[dtype] and lse_off(lse3, lse_ref) <= 2.0 ** -13
        for a, b in zip(grads, ttt.window_attention_backward(q, k, v, o, lse, go, **kw)):
            assert rel(b, a) <= 2 * GTOL[dtype] or a.norm() < 0.05 * go.norm()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_many_sequences(dtype):
    """More than a wave has lanes, and than the table's groups: empty ones among them."""
    from test_weight_layers_amd import ttt
    g = torch.Generator().manual_seed(3)
    for n in (64, 1500):
        lens = torch.randint(0, 9, (n,), generator=g).tolist()
        lens[5] = 300
        q, k, v, go = inputs(sum(lens), sum(lens), 2, 1, 64, dtype)
        how = (1, 7, 0, 2)
        o_ref, lse_ref, gr = reference(q, k, v, 2, 1, lens, lens, how, grad_o=go)
        kw = dict(heads=2, key_heads=1, before=7, sinks=2, cu_seqlens=offsets(lens))
        q, k, v, go = (t.cuda() for t in (q, k, v, go))
        o, lse = ttt.window_attention(q, k, v, **kw)
        assert rel(o, o_ref) <= TOL[dtype] and lse_off(lse, lse_ref) <= 2.0 ** -14
        for a, r in zip(ttt.window_attention_backward(q, k, v, o, lse, go, **kw), gr):
            assert rel(a, r) <= GTOL[dtype]


def test_gradient_against_differences():
    """Central differences of the fp32 call over a step of 2^-6: its outputs are off by 2^-17 of the loss' terms, whose
    sum's 2-norm is that of the gradient's size; the third derivative adds step^2 / 6: together below 1% of the norm."""
    from test_weight_layers_amd import ttt
    H, Hk, d, lens = 2, 1, 64, [40, 23]
    t = [x.cuda() for x in inputs(63, 63, H, Hk, d, F32, seed=5)]
    kw = dict(heads=H, key_heads=Hk, block=5, before=2, after=1, sinks=3, cu_seqlens=offsets(lens), scale=0.2)
    o, lse = ttt.window_attention(*t[:3], **kw)
    grads = ttt.window_attention_backward(*t[:3], o, lse, t[3], **kw)
    for i in range(3):
        u = torch.randn(grads[i].shape, generator=torch.Generator().manual_seed(i)).cuda().double()
        u = u / u.norm() + grads[i].double() / grads[i].double().norm()
        u /= u.norm()

        def loss(h):
            x = list(t[:3])
            x[i] = (x[i].double() + h * u).float()
            return (ttt.window_attention(*x, **kw)[0].double() * t[3]).sum().item()

        h = 2.0 ** -6
        diff = (loss(h) - loss(-h)) / (2 * h)
        assert abs(diff - (grads[i].double() * u).sum().item()) <= 1e-2 * grads[i].norm().item(), i


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")], ids=str)
def test_what_is_not_finite_reaches_only_rows_that_see_it(dtype, value):
    not_finite(2, 64, dtype, value)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H, d", [(400, 64), (2, 128), (180, 128), (2, 256), (180, 256)])
def test_what_is_not_finite_in_every_kind_of_tile(H, d, dtype):
    not_finite(H, d, dtype, float("nan"))


def not_finite(H, d, dtype, value):
    from test_weight_layers_amd import ttt
    n = 300
    q, k, v, go = (t.cuda() for t in inputs(n, n, H, H, d, dtype, seed=7))
    kw = dict(heads=H, before=40, sinks=3)
    ok = mask(n, n, 1, 40, 0, 3).cuda()
    o, lse = ttt.window_attention(q, k, v, **kw)
    grads = ttt.window_attention_backward(q, k, v, o, lse, go, **kw)
    for j in (1, 150, 299):
        sees = ok[:, j]
        v2 = v.clone()
        v2[j, 5] = value
        o2, lse2 = ttt.window_attention(q, k, v2, **kw)
        assert torch.equal(o2[~sees], o[~sees]) and torch.equal(lse2, lse)
        assert torch.equal(o2[:, torch.arange(H * d, device="cuda") != 5], o[:, torch.arange(H * d, device="cuda") != 5])
        assert not torch.isfinite(o2[sees, 5]).any()
        k2 = k.clone()
        k2[j, 7] = value
        o3, _ = ttt.window_attention(q, k2, v, **kw)
        assert torch.equal(o3[~sees], o[~sees]) and torch.equal(o3[:, d:], o[:, d:])
        # the gradients of rows that it has nothing to do with
        g2 = ttt.window_attention_backward(q, k, v2, o, lse, go, **kw)
        assert torch.equal(g2[0][~sees], grads[0][~sees]) and torch.equal(g2[2], grads[2])
        apart = ~ok[sees].any(0)                     # keys that no query that sees j sees
        assert torch.equal(g2[1][apart], grads[1][apart])
        g3 = ttt.window_attention_backward(q, k2, v, o, lse, go, **kw)
        assert torch.equal(g3[0][~sees], grads[0][~sees])
    i = 200
    for name in ("q", "go"):
        q2, go2 = q.clone(), go.clone()
        (q2 if name == "q" else go2)[i, 3] = value
        g4 = ttt.window_attention_backward(q2, k, v, o, lse, go2, **kw)
        other = torch.arange(n, device="cuda") != i
        assert torch.equal(g4[0][other], grads[0][other])
        for a, b in zip(g4[1:], grads[1:]):
            assert torch.equal(a[~ok[i]], b[~ok[i]])


def test_values_of_any_size():
    """Scores of hundreds, and rows whose every visible score is the type's lowest."""
    from test_weight_layers_amd import ttt
    q, k, v, go = (t.cuda() for t in inputs(130, 130, 1, 1, 64, F32, seed=8))
    q *= 30.0
    o, lse = ttt.window_attention(q, k, v, heads=1)
    o_ref, lse_ref, _ = reference(q.cpu(), k.cpu(), v.cpu(), 1, 1, [130], [130], (1, None, 0, 0))
    # scores 30 times as large: 30 times the absolute error
    assert rel(o, o_ref) <= 30 * TOL[F32] and lse_off(lse, lse_ref) <= 30 * 2.0 ** -16
    # sums of |q| of 64 elements are between 8 and 4000 here: times 1e18 * 1e18 the products are beyond fp32's 3.4e38 (at
    # least 8e36 * 30), -inf in every row but for chance, and the softmax of nothing else is NaN, as the formula has it
    low = torch.full_like(k, -1e18)
    assert ((q.abs() * 1e18).double() @ low[0].double()).max() < -3.4e38
    o, lse = ttt.window_attention(q.abs() * 1e18, low, v, heads=1)
    assert o.isnan().all()
    # a hundredth of it is not: every visible score the same, as low as it may be
    low = torch.full_like(k, -1e16)
    o, lse = ttt.window_attention(q.abs() * 1e18, low, v, heads=1)
    mean = v.double().cumsum(0) / torch.arange(1, 131, device="cuda")[:, None]
    assert rel(o, mean) <= TOL[F32] and torch.isfinite(lse).all() and (lse < -1e34).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_rows_of_no_sequence_and_strides(dtype):
    from test_weight_layers_amd import ttt
    H, Hk, d, n = 4, 2, 64, 150
    q, k, v, go = (t.cuda() for t in inputs(n, n, H, Hk, d, dtype, seed=9))
    cu = torch.tensor([10, 60, 60, 140], dtype=torch.int32, device="cuda")
    kw = dict(heads=H, key_heads=Hk, before=20, sinks=2, cu_seqlens=cu)
    o, lse = ttt.window_attention(q, k, v, **kw)
    unused = torch.ones(n, dtype=torch.bool, device="cuda")
    unused[10:140] = False
    assert (o[unused] == 0).all() and (lse[:, unused] == -math.inf).all()
    ref = ttt.window_attention(q[10:140].contiguous(), k[10:140].contiguous(), v[10:140].contiguous(),
                               **{**kw, "cu_seqlens": cu - 10})
    assert torch.equal(o[10:140], ref[0])
    # column slices of one buffer, a given output; what stands in unused rows is not read
    w = (H + 2 * Hk) * d
    buf = torch.full((n, w + 8), float("nan"), dtype=dtype, device="cuda")
    qs, ks, vs = buf[:, :H * d], buf[:, H * d:(H + Hk) * d], buf[:, (H + Hk) * d:w]
    for to, x in ((qs, q), (ks, k), (vs, v)):
        to[10:140] = x[10:140]
    out = torch.full((n, H * d), 5.0, dtype=dtype, device="cuda")
    o2, lse2 = ttt.window_attention(qs, ks, vs, out=out, **kw)
    assert o2 is out and torch.equal(out[10:140], o[10:140]) and (out[unused] == 5.0).all() and torch.equal(lse, lse2)
    gbuf = torch.full_like(buf, 3.0)
    gs = (gbuf[:, :H * d], gbuf[:, H * d:(H + Hk) * d], gbuf[:, (H + Hk) * d:w])
    got = ttt.window_attention_backward(qs, ks, vs, out, lse, go, out=gs, **kw)
    ref = ttt.window_attention_backward(q, k, v, o, lse, go, **kw)
    for a, b in zip(got, ref):
        assert torch.equal(a, b) and (a[unused] == 0).all()
    assert (gbuf[:, w:] == 3.0).all()


def test_offsets_of_any_values():
    """Offsets outside the rows or out of order name disjoint rows inside them."""
    from test_weight_layers_amd import ttt
    q, k, v, go = (t.cuda() for t in inputs(100, 100, 1, 1, 64, F32, seed=10))
    bad = torch.tensor([-5, 70, 30, 1000], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 70, 70, 100], dtype=torch.int32, device="cuda")
    a, b = (ttt.window_attention(q, k, v, heads=1, cu_seqlens=c) for c in (bad, good))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = (ttt.window_attention_backward(q, k, v, *b, go, heads=1, cu_seqlens=c) for c in (bad, good))
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))


def test_no_rows():
    from test_weight_layers_amd import ttt
    e = torch.empty(0, 64, device="cuda")
    o, lse = ttt.window_attention(e, e.clone(), e.clone(), heads=1)
    assert o.shape == (0, 64) and lse.shape == (1, 0)
    x = torch.randn(5, 64, device="cuda")
    o, lse = ttt.window_attention(x, e, e.clone(), heads=1)
    assert (o == 0).all() and (lse == -math.inf).all()
    gq, gk, gv = ttt.window_attention_backward(x, e, e.clone(), o, lse, x.clone(), heads=1)
    assert (gq == 0).all() and gk.shape == (0, 64)
    gq, gk, gv = ttt.window_attention_backward(e, x, x.clone(), e.clone(), lse[:, :0].contiguous(), e.clone(), heads=1)
    assert gq.shape == (0, 64) and (gk == 0).all() and (gv == 0).all()
    cache = torch.zeros(2, 8, 64, device="cuda")
    assert ttt.window_attention_step(cache, cache.clone(), e, e, e, torch.empty(0, dtype=torch.int32, device="cuda"),
                                     heads=1).shape == (0, 64)


def test_sinks_without_keys_and_of_many_sequences():
    from test_weight_layers_amd import ttt
    x, e = torch.randn(300, 128, device="cuda"), torch.empty(0, 64, device="cuda")
    kw = dict(heads=2, key_heads=1, before=10, sinks=4)
    o, lse = ttt.window_attention(x, e, e.clone(), **kw)
    gq, gk, gv = ttt.window_attention_backward(x, e, e.clone(), o, lse, x.clone(), **kw)
    assert (o == 0).all() and (gq == 0).all() and gk.shape == gv.shape == (0, 64)
    # more of them than their sums are kept apart for (64 MB)
    lens, how = [300, 7] * 300, (1, 20, 0, 4)
    q, k, v, go = inputs(sum(lens), sum(lens), 4, 4, 64, BF)
    _, _, ref = reference(q, k, v, 4, 4, lens, lens, how, grad_o=go)
    q, k, v, go = (t.cuda() for t in (q, k, v, go))
    kw = dict(heads=4, before=20, sinks=4, cu_seqlens=offsets(lens))
    o, lse = ttt.window_attention(q, k, v, **kw)
    for a, r in zip(ttt.window_attention_backward(q, k, v, o, lse, go, **kw), ref):
        assert rel(a, r) <= GTOL[BF]


# ------------------------------------------------------------------ one token
def ring_place(p, capacity, sinks):
    return p if p < sinks else sinks + (p - sinks) % (capacity - sinks)


def step_reference(history, q, H, Hk, p, capacity, block, before, sinks, scale):
    """history: k and v rows [p + 1] in fp64."""
    d = q.shape[-1] // H
    lo = 0 if before is None else max(0, (p // block - before) * block)
    if p >= capacity:
        lo = max(lo, p + 1 - (capacity - sinks))
    js = [j for j in range(p + 1) if j >= lo or j < sinks]
    ks, vs = (x[js].view(len(js), Hk, d).transpose(0, 1).repeat_interleave(H // Hk, 0) for x in history)
    s = (ks @ q.double().view(H, d, 1))[..., 0] * scale
    return (torch.softmax(s, -1)[:, None] @ vs).reshape(-1)


# heads, key heads, d, capacity, block, before, sinks, dtype
STEPS = [
    (1, 1, 64, 1, 1, None, 0, F32),
    (2, 2, 64, 33, 1, None, 4, BF),
    (4, 2, 128, 50, 1, 20, 3, F32),
    (40, 2, 64, 40, 1, 33, 0, BF),               # 20 heads of a key head
    (3, 1, 256, 37, 10, 1, 5, BF),
    (2, 1, 256, 70, 16, 2, 0, F32),
    (2, 2, 128, 64, 7, None, 1, BF),
]


@pytest.mark.parametrize("case", STEPS, ids=str)
def test_stream_of_single_tokens(case):
    """Streams of uneven ages in shuffled caches, a padded row between them, until they went round their caches."""
    from test_weight_layers_amd import ttt
    H, Hk, d, capacity, block, before, sinks, dtype = case
    g = torch.Generator().manual_seed(1)
    pool, n, T = 5, 3, 2 * capacity + 7
    k, v = (torch.randn(n, T, Hk * d, generator=g).to(dtype).cuda() for _ in range(2))
    q = torch.randn(n, T, H * d, generator=g).to(dtype).cuda()
    kc, vc = (torch.full((pool, capacity, Hk * d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    slots = torch.tensor([3, -1, 0, 4], dtype=torch.int32, device="cuda")
    start = [0, 5, T - 3]                            # steps at which the streams begin
    rows = [0, 2, 3]
    for t in range(T):
        pos = torch.tensor([t - start[0], 7, t - start[1], t - start[2]], dtype=torch.int32, device="cuda")
        pick = lambda x: torch.stack([x[0, t], x[0, t] * float("nan"), x[1, max(0, t - start[1])], x[2, max(0, t - start[2])]])
        o = ttt.window_attention_step(kc, vc, pick(q), pick(k), pick(v), pos, heads=H, key_heads=Hk, slots=slots, block=block,
                                      before=before, sinks=sinks, scale=0.3)
        assert (o[1] == 0).all()
        if t % 5 and t < T - 3:
            continue
        for i in range(n):
            p = t - start[i]
            if p < 0:
                assert (o[rows[i]] == 0).all()
                continue
            ref = step_reference([x[i, :p + 1].double() for x in (k, v)], q[i, p], H, Hk, p, capacity, block, before, sinks, 0.3)
            assert rel(o[rows[i]], ref) <= TOL[dtype], (t, i)
    # what the caches hold
    for i, slot in enumerate((3, 0, 4)):
        p = T - 1 - start[i]
        for j in range(max(0, p - (capacity - sinks) + 1), p + 1):
            assert torch.equal(kc[slot, ring_place(j, capacity, sinks)], k[i, j])
            assert torch.equal(vc[slot, ring_place(j, capacity, sinks)], v[i, j])
    assert kc[1].isnan().all() and vc[2].isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_step_over_a_long_cache(dtype):
    """Enough keys for many ranges of them, against the form for prompts; both caches in one buffer."""
    from test_weight_layers_amd import ttt
    H, Hk, d, T = 4, 2, 64, 5000
    g = torch.Generator().manual_seed(2)
    both = torch.randn(2, T + 1, 2 * Hk * d, generator=g).to(dtype).cuda()
    kc, vc = both[:, :, :Hk * d], both[:, :, Hk * d:]
    q, k, v = (torch.randn(2, h * d, generator=g).to(dtype).cuda() for h in (H, Hk, Hk))
    pos = torch.tensor([T, 1234], dtype=torch.int32, device="cuda")
    old = both.clone()
    o = ttt.window_attention_step(kc, vc, q, k, v, pos, heads=H, key_heads=Hk, block=3, before=1000, sinks=9)
    for i, p in enumerate(pos.tolist()):
        ks, vs = (torch.cat([x[i, :p], y[i:i + 1]]) for x, y in ((old[:, :, :Hk * d], k), (old[:, :, Hk * d:], v)))
        ref, _, _ = reference(q[i:i + 1], ks, vs, H, Hk, [1], [p + 1], (3, 1000, 0, 9))
        assert rel(o[i:i + 1], ref) <= TOL[dtype]
        assert torch.equal(kc[i, p], k[i]) and torch.equal(vc[i, p], v[i])
        old[i, p] = both[i, p]
    assert torch.equal(old, both)
    pair = both.view(2, T + 1, 2, Hk * d).transpose(1, 2).contiguous()       # [pool, k or v, capacity, columns]
    pair.transpose(1, 2).reshape(both.shape).copy_(both)
    o2 = ttt.window_attention_step(pair[:, 0], pair[:, 1], q, k, v, pos, heads=H, key_heads=Hk, block=3, before=1000, sinks=9)
    assert torch.equal(o, o2)


def test_step_rows_of_one_cache():
    """They read the cache as it was; of one place the last row's token stays."""
    from test_weight_layers_amd import ttt
    d, n = 64, 6
    g = torch.Generator().manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()
    kc, vc, q, k, v = rn(2, 20, d), rn(2, 20, d), rn(n, d), rn(n, d), rn(n, d)
    slots = torch.tensor([0, 1, 0, 0, 7, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([10, 10, 10, 11, 10, 10], dtype=torch.int32, device="cuda")
    kc1, vc1 = kc.clone(), vc.clone()
    o = ttt.window_attention_step(kc1, vc1, q, k, v, pos, heads=1, slots=slots)
    for i in range(n):
        a, b = kc.clone(), vc.clone()
        one = ttt.window_attention_step(a, b, q[i:i + 1], k[i:i + 1], v[i:i + 1], pos[i:i + 1], heads=1, slots=slots[i:i + 1])
        assert rel(o[i:i + 1], one) <= 2.0 ** -20      # (other ranges of keys: fp32 sums in another order)
    kc[0, 10], vc[0, 10], kc[0, 11], vc[0, 11], kc[1, 10], vc[1, 10] = k[5], v[5], k[3], v[3], k[1], v[1]
    assert torch.equal(kc, kc1) and torch.equal(vc, vc1)
    # a given output keeps its padded rows
    out = torch.full((n, d), 4.0, device="cuda")
    ttt.window_attention_step(kc1, vc1, q, k, v, pos, heads=1, slots=slots, out=out)
    assert (out[4] == 4.0).all()


# ------------------------------------------------------------------ graphs and streams
def test_replay_and_streams():
    from test_weight_layers_amd import ttt
    H, Hk, d, n = 4, 2, 64, 700
    lens = [300, 0, 400]
    cu = offsets(lens)
    new = lambda seed: [t.cuda() for t in inputs(n, n, H, Hk, d, BF, seed=seed)]
    q, k, v, go = new(1)
    kw = dict(heads=H, key_heads=Hk, before=30, sinks=4, cu_seqlens=cu)
    ttt.window_attention(q, k, v, **kw)
    kc, vc = (torch.randn(3, 50, Hk * d, device="cuda").to(BF) for _ in range(2))
    pos = torch.tensor([7, 60], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    kc0, vc0 = kc.clone(), vc.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = ttt.window_attention(q, k, v, **kw)
        grads = ttt.window_attention_backward(q, k, v, o, lse, go, **kw)
        one = ttt.window_attention_step(kc, vc, q[:2], k[:2], v[:2], pos, heads=H, key_heads=Hk, sinks=2)
    for seed in (2, 3, 4):
        x = new(seed)
        for a, b in zip((q, k, v, go), x):
            a.copy_(b)
        pos += 1
        graph.replay()
        o2, lse2 = ttt.window_attention(*x[:3], **kw)
        grads2 = ttt.window_attention_backward(*x[:3], o2, lse2, x[3], **kw)
        one2 = ttt.window_attention_step(kc0, vc0, x[0][:2], x[1][:2], x[2][:2], pos, heads=H, key_heads=Hk, sinks=2)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(one, one2)
        assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
        assert all(torch.equal(a, b) for a, b in zip(grads, grads2))
    # two calls at once on streams of their own
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s, seed in zip(streams, (5, 6)):
        x = new(seed)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            outs.append((x, ttt.window_attention(*x[:3], **kw)))
    torch.cuda.synchronize()
    for x, (a, b) in outs:
        ref = ttt.window_attention(*x[:3], **kw)
        assert torch.equal(a, ref[0]) and torch.equal(b, ref[1])


def test_refusals():
    from test_weight_layers_amd import ttt
    q = torch.zeros(4, 128, device="cuda")
    k = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError, match="heads"):
        ttt.window_attention(q, k, k, heads=3)
    with pytest.raises(ttt.TTTError, match="d=32"):
        ttt.window_attention(q, q, q.clone(), heads=4)
    with pytest.raises(ValueError, match="k must be"):
        ttt.window_attention(q, k, k, heads=2)
    with pytest.raises(ttt.TTTError, match="block"):
        ttt.window_attention(q, k, k, heads=2, key_heads=1, block=0)
    with pytest.raises(ValueError, match="before"):
        ttt.window_attention(q, k, k, heads=2, key_heads=1, before=-1)
    with pytest.raises(ttt.TTTError, match="scale"):
        ttt.window_attention(q, k, k, heads=2, key_heads=1, scale=0.0)
    with pytest.raises(ttt.TTTError, match="overlap"):
        ttt.window_attention(q, k, k, heads=2, key_heads=1, out=q)
    with pytest.raises(ttt.TTTError, match="cu_seqlens_k"):
        ttt.window_attention(q, torch.zeros(5, 64, device="cuda"), torch.zeros(5, 64, device="cuda"), heads=2, key_heads=1,
                             cu_seqlens=offsets([4]))
    with pytest.raises(ValueError, match="cu_seqlens"):
        ttt.window_attention(q, k, k, heads=2, key_heads=1, cu_seqlens=torch.tensor([0, 4], device="cuda"))
    with pytest.raises(ValueError, match="dtype"):
        ttt.window_attention(q, k.bfloat16(), k, heads=2, key_heads=1)
    with pytest.raises(ttt.TTTError, match="workspace"):
        ttt.window_attention(q, k, k, heads=2, key_heads=1, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    o, lse = ttt.window_attention(q, k, k, heads=2, key_heads=1)
    with pytest.raises(ValueError, match="lse"):
        ttt.window_attention_backward(q, k, k, o, lse.t(), o, heads=2, key_heads=1)
    with pytest.raises(ttt.TTTError, match="overlap"):
        ttt.window_attention_backward(q, k, k, o, lse, o, heads=2, key_heads=1, out=(torch.empty_like(q), k, torch.empty_like(k)))
    cache = torch.zeros(2, 8, 64, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    step = lambda **kw: ttt.window_attention_step(cache, kw.pop("vc", torch.zeros_like(cache)), q, k, k, kw.pop("pos", pos),
                                                  heads=2, key_heads=1, **kw)
    with pytest.raises(ttt.TTTError, match="pool"):
        step()
    with pytest.raises(ttt.TTTError, match="capacity"):
        step(slots=pos, sinks=8)
    with pytest.raises(ttt.TTTError, match="overlap"):
        step(slots=pos, vc=cache)
    with pytest.raises(ValueError, match="positions"):
        step(slots=pos, pos=pos.long())
    with pytest.raises(ValueError, match="slots"):
        step(slots=pos[:3])


@pytest.mark.parametrize("big", [1 << 31, 1 << 32, (1 << 40) + 3])
def test_limits_beyond_32_bits(big):
    """A limit that takes in everything is none: the same bits as without it."""
    from test_weight_layers_amd import ttt
    q, k, v, go = (t.cuda() for t in inputs(70, 300, 2, 1, 64, BF, seed=9))
    for kw, same in ((dict(before=big), dict(before=None)), (dict(before=3, after=big), dict(before=3, after=None)),
                     (dict(before=2, sinks=big), dict(before=2, sinks=(1 << 31) - 1))):
        o, lse = ttt.window_attention(q, k, v, heads=2, key_heads=1, block=5, **kw)
        o2, lse2 = ttt.window_attention(q, k, v, heads=2, key_heads=1, block=5, **same)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        for a, b in zip(ttt.window_attention_backward(q, k, v, o, lse, go, heads=2, key_heads=1, block=5, **kw),
                        ttt.window_attention_backward(q, k, v, o, lse, go, heads=2, key_heads=1, block=5, **same)):
            assert torch.equal(a, b)
    kc, vc = (torch.randn(70, 40, 64, generator=torch.Generator().manual_seed(i)).to(BF).cuda() for i in (1, 2))
    at = torch.arange(70, dtype=torch.int32).cuda()
    step = lambda before: ttt.window_attention_step(kc.clone(), vc.clone(), q, k[:70], v[:70], at, heads=2, key_heads=1, before=before)
    assert torch.equal(step(big), step(None)) and not torch.equal(step(big), step(0))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("pool,more", [(1, 0), (1, 8), (2, 24)], ids=["one", "one with other columns", "entries apart"])
def test_step_halves_of_one_buffer(pool, more, dtype):
    """k and v as column halves of the same rows, of one cache and of entries that are not whole rows apart, round and round:
    the bits of caches of their own."""
    from test_weight_layers_amd import ttt
    H, Hk, d, capacity = 4, 2, 64, 11
    g = torch.Generator().manual_seed(pool)
    width, pad = 2 * Hk * d + (8 if more == 8 else 0), 16 if more == 24 else 0
    flat = torch.full((pool * (capacity * width + pad),), 7.0, dtype=dtype, device="cuda")
    both = flat.as_strided((pool, capacity, width), (capacity * width + pad, width, 1))
    kc, vc = both[:, :, :Hk * d], both[:, :, Hk * d:2 * Hk * d]
    k2, v2 = kc.clone().contiguous(), vc.clone().contiguous()
    expect = flat.clone()
    for p in range(30):
        q, k, v = (torch.randn(pool, h * d, generator=g).to(dtype).cuda() for h in (H, Hk, Hk))
        at = torch.full((pool,), p, dtype=torch.int32, device="cuda")
        kw = dict(heads=H, key_heads=Hk, sinks=3)
        o, o2 = ttt.window_attention_step(kc, vc, q, k, v, at, **kw), ttt.window_attention_step(k2, v2, q, k, v, at, **kw)
        assert torch.equal(o, o2) and torch.equal(kc, k2) and torch.equal(vc, v2), p
    view = expect.as_strided(both.shape, both.stride())
    view[:, :, :Hk * d], view[:, :, Hk * d:2 * Hk * d] = k2, v2
    assert torch.equal(flat, expect)


# Far fewer queries than keys and far fewer keys than queries: what of the other side a walk is cut by, and tiles beyond a window.
UNEQUAL = [
    (8, 2, 128, [64], [4100], (1, None, 0, 0), BF),
    (8, 2, 128, [64], [4100], (1, None, 0, 0), F32),
    (4, 4, 64, [33], [5000], (1, None, None, 0), F32),
    (2, 1, 256, [90], [3000], (1, 700, 0, 4), BF),
    (4, 1, 256, [150], [2000], (10, 30, 0, 70), F32),
    (2, 2, 128, [500], [2500], (1, 100, 100, 0), BF),
    (2, 2, 128, [500], [2500], (7, 10, 10, 30), F32),
    (2, 1, 64, [1], [3000], (1, None, 0, 0), BF),
    (8, 2, 128, [4100], [64], (1, None, None, 0), BF),
    (4, 4, 64, [5000], [33], (1, None, None, 0), F32),
    (2, 1, 256, [2500], [100], (1, None, None, 0), BF),
    (4, 2, 128, [1500], [500], (1, None, 0, 0), BF),              # queries before the first key
    (4, 2, 128, [1500], [500], (8, 5, 60, 20), F32),
    (2, 2, 64, [3000], [1], (1, None, None, 0), BF),
    (8, 4, 64, [70, 0, 1, 200], [2000, 10, 1500, 0], (1, None, 0, 3), BF),
    (4, 4, 64, [3000, 40, 5], [70, 900, 0], (4, None, None, 0), F32),
]


@pytest.mark.parametrize("case", UNEQUAL, ids=str)
def test_unequal_rows(case):
    test_forward_and_gradient(case)
