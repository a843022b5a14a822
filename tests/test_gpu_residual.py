"""Gated residual tail (ttt.gated_residual and its gradient) against the formulas in 64 bits.

Tolerances (relative 2-norm).  Everything is fp32 and rounded once at the end: at most 2^-8 of each bf16
element.  The fp32 arithmetic before it: sums of squares of up to 8192 terms (a wave's tree: 8 terms a
lane, then log2 steps: under 40 roundings of 2^-24), reciprocal, square root, exp2 of a rounded product
(|z| <= 6 here: 9 roundings): below 64 * 2^-24 = 4e-6 for fp32 outputs.  Sums over rows add at most 4000
terms one after another, of random sign: the 2-norm grows with the root, 64 * 2^-24, as well.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 2.0 ** -8, torch.float32: 4e-6}


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


def inputs(n, C, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    d = {x: rn(n, C).to(dtype) for x in ("x", "o", "z", "gy", "gh")}
    for x in ("gamma", "alpha", "gamma_next"):
        d[x] = 1.0 + 0.3 * rn(C)
    return d


def forward(x, o, z, gamma, alpha, gamma_next, eps, norm):
    n, C = o.shape
    og = o.reshape(n, C // norm, norm)
    u = (og / torch.sqrt((og * og).mean(-1, keepdim=True) + eps)).reshape(n, C)
    u = u if gamma is None else u * gamma
    u = u if z is None else u * z * torch.sigmoid(z)
    y = x + (u if alpha is None else alpha * u)
    h = None if gamma_next is None else y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * gamma_next
    return y, h


CASES = [
    # n, channels, norm width, gate, dtype
    (1, 8, 8, True, torch.float32),
    (5, 64, 64, True, torch.bfloat16),
    (37, 64, 16, False, torch.float32),
    (130, 120, 24, True, torch.bfloat16),
    (33, 256, 64, True, torch.float32),
    (70, 504, 504, True, torch.bfloat16),
    (1374, 1024, 256, True, torch.bfloat16),
    (259, 1000, 200, True, torch.float32),
    (64, 1536, 768, False, torch.bfloat16),
    (41, 2048, 64, True, torch.bfloat16),
    (19, 3584, 3584, True, torch.bfloat16),
    (23, 4000, 400, True, torch.float32),
    (9, 8192, 512, True, torch.bfloat16),
    (6, 8192, 4096, True, torch.float32),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradient(case):
    from test_weight_layers_amd import ttt
    n, C, norm, gate, dtype = case
    d = inputs(n, C, dtype)
    if not gate:
        d["z"] = None
    f = {k: None if v is None else v.double() for k, v in d.items()}
    y_ref, h_ref = forward(f["x"], f["o"], f["z"], f["gamma"], f["alpha"], f["gamma_next"], 1e-6, norm)
    g = {k: None if v is None else v.cuda() for k, v in d.items()}
    par = [g[x] for x in ("gamma", "alpha", "gamma_next")]
    y, h = ttt.gated_residual(g["x"], g["o"], g["z"], *par, 1e-6, norm_width=norm)
    assert rel(y, y_ref) <= TOL[dtype] and rel(h, h_ref) <= TOL[dtype]
    x2 = g["x"].clone()
    y2, h2 = ttt.gated_residual(x2, g["o"], g["z"], *par, 1e-6, norm_width=norm, out=x2)
    assert y2 is x2 and torch.equal(y, y2) and torch.equal(h, h2)

    # the gradient at the stored y
    leaf = lambda t: None if t is None else t.clone().requires_grad_(True)
    ys = y.double().cpu().requires_grad_(True)
    gn = leaf(f["gamma_next"])
    hh = ys / torch.sqrt((ys * ys).mean(-1, keepdim=True) + 1e-6) * gn
    dyh, dgn = torch.autograd.grad(hh, (ys, gn), f["gh"])
    gx_ref = f["gy"] + dyh
    o, z, ga, al = leaf(f["o"]), leaf(f["z"]), leaf(f["gamma"]), leaf(f["alpha"])
    out, _ = forward(torch.zeros_like(f["x"]), o, z, ga, al, None, 1e-6, norm)
    refs = torch.autograd.grad(out, [t for t in (o, z, ga, al) if t is not None], gx_ref)
    go_ref, gz_ref = refs[0], refs[1] if gate else None
    gg_ref, ga_ref = refs[-2], refs[-1]
    got = ttt.gated_residual_backward(g["gy"], g["gh"], y, g["o"], g["z"], *par, 1e-6, norm_width=norm)
    again = ttt.gated_residual_backward(g["gy"], g["gh"], y, g["o"], g["z"], *par, 1e-6, norm_width=norm)
    err = {}
    for name, a, b, r in zip(("x", "o", "z", "gamma", "alpha", "gamma_next"), got, again,
                             (gx_ref, go_ref, gz_ref, gg_ref, ga_ref, dgn)):
        if r is None:
            assert a is None
            continue
        assert torch.equal(a, b)
        err[name] = (rel(a, r), TOL[a.dtype])
    print({k: f"{v[0]:.1e}" for k, v in err.items()})
    assert all(a <= b for a, b in err.values()), err


def test_gradient_against_differences():
    """Central differences of the fp32 call: outputs are off by 1e-6 of the loss' terms, over a step of 2^-6;
    the third derivative adds step^2 / 6 of the curvature's size: 2e-3 of the gradient's norm."""
    from test_weight_layers_amd import ttt
    n, C, norm = 17, 96, 32
    g = {k: v.cuda() for k, v in inputs(n, C, torch.float32, seed=3).items()}
    names = ("x", "o", "z", "gamma", "alpha", "gamma_next")
    run = lambda a: ttt.gated_residual(*[a[x] for x in names], 1e-6, norm_width=norm)
    y, _ = run(g)
    grads = ttt.gated_residual_backward(g["gy"], g["gh"], y, *[g[x] for x in names[1:]], 1e-6, norm_width=norm)
    for name, grad in zip(names, grads):
        u = torch.randn(grad.shape, generator=torch.Generator().manual_seed(1)).cuda().double()
        u = u / u.norm() + grad.double() / grad.double().norm()
        u /= u.norm()

        def loss(h):
            y, hh = run({**g, name: (g[name].double() + h * u).float()})
            return ((y.double() * g["gy"]).sum() + (hh.double() * g["gh"]).sum()).item()

        h = 2.0 ** -6
        diff = (loss(h) - loss(-h)) / (2 * h)
        assert abs(diff - (grad.double() * u).sum().item()) <= 2e-3 * grad.norm().item(), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_left_out_parts(dtype):
    from test_weight_layers_amd import ttt
    n, C = 50, 128
    d = inputs(n, C, dtype, seed=4)
    f = {k: v.double() for k, v in d.items()}
    g = {k: v.cuda() for k, v in d.items()}
    y, h = ttt.gated_residual(g["x"], g["o"])
    assert h is None and rel(y, forward(f["x"], f["o"], None, None, None, None, 1e-6, C)[0]) <= TOL[dtype]
    y, h = ttt.gated_residual(g["x"], g["o"], alpha=g["alpha"], gamma_next=g["gamma_next"])
    ref = forward(f["x"], f["o"], None, None, f["alpha"], f["gamma_next"], 1e-6, C)
    assert rel(y, ref[0]) <= TOL[dtype] and rel(h, ref[1]) <= TOL[dtype]
    # no gradient of h, or none of y
    for gy, gh in ((g["gy"], None), (None, g["gh"])):
        got = ttt.gated_residual_backward(gy, gh, y, g["o"], alpha=g["alpha"], gamma_next=g["gamma_next"])
        full = ttt.gated_residual_backward(torch.zeros_like(g["gy"]) if gy is None else gy,
                                           torch.zeros_like(g["gh"]) if gh is None else gh, y, g["o"],
                                           alpha=g["alpha"], gamma_next=g["gamma_next"])
        assert got[2] is None and got[3] is None
        for i in (0, 1, 4, 5):
            assert torch.equal(got[i], full[i])


def test_no_rows_and_zero_rows():
    from test_weight_layers_amd import ttt
    e = torch.empty(0, 64, device="cuda")
    ones = torch.ones(64, device="cuda")
    y, h = ttt.gated_residual(e, e.clone(), gamma_next=ones)
    assert y.shape == (0, 64) and h.shape == (0, 64)
    got = ttt.gated_residual_backward(e, e.clone(), y, e.clone(), gamma=ones, gamma_next=ones)
    assert (got[3] == 0).all() and (got[5] == 0).all()
    z = torch.zeros(3, 64, device="cuda")
    y, h = ttt.gated_residual(z, z.clone(), gamma_next=ones)
    assert (y == 0).all() and (h == 0).all()
    # NaN in one row stays in that row
    x = torch.randn(9, 64, device="cuda")
    o = torch.randn(9, 64, device="cuda")
    ref = ttt.gated_residual(x, o, gamma_next=ones)
    x2 = x.clone()
    x2[4, 7] = float("nan")
    got = ttt.gated_residual(x2, o, gamma_next=ones)
    keep = torch.arange(9, device="cuda") != 4
    assert torch.equal(got[0][keep], ref[0][keep]) and torch.equal(got[1][keep], ref[1][keep])
    assert got[1][4].isnan().all()


def test_strided_rows_and_replay():
    from test_weight_layers_amd import ttt
    n, C = 300, 256
    d = {k: v.cuda() for k, v in inputs(n, C, torch.bfloat16, seed=5).items()}
    wide = torch.full((n, 3 * C + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    x, o, z = wide[:, :C], wide[:, C:2 * C], wide[:, 2 * C:3 * C]
    x.copy_(d["x"]), o.copy_(d["o"]), z.copy_(d["z"])
    par = [d[k] for k in ("gamma", "alpha", "gamma_next")]
    ref = ttt.gated_residual(d["x"], d["o"], d["z"], *par, norm_width=64)
    got = ttt.gated_residual(x, o, z, *par, norm_width=64)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1]) and (wide[:, 3 * C:] == 9.0).all()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = ttt.gated_residual(x, o, z, *par, norm_width=64)
        grads = ttt.gated_residual_backward(d["gy"], d["gh"], y, o, z, *par, norm_width=64)
    for seed in (6, 7, 8):
        new = {k: v.cuda() for k, v in inputs(n, C, torch.bfloat16, seed=seed).items()}
        x.copy_(new["x"]), o.copy_(new["o"]), z.copy_(new["z"])
        graph.replay()
        y2, h2 = ttt.gated_residual(new["x"], new["o"], new["z"], *par, norm_width=64)
        grads2 = ttt.gated_residual_backward(d["gy"], d["gh"], y2, new["o"], new["z"], *par, norm_width=64)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(h, h2)
        assert all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_refusals():
    from test_weight_layers_amd import ttt
    x = torch.zeros(4, 64, device="cuda")
    o = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ttt.TTTError, match="norm_width"):
        ttt.gated_residual(x, o, norm_width=48)
    with pytest.raises(ttt.TTTError, match="channels"):
        ttt.gated_residual(x[:, :60].contiguous(), o[:, :60].contiguous())
    with pytest.raises(ttt.TTTError, match="overlap"):
        ttt.gated_residual(x, o, out=o)
    with pytest.raises(ttt.TTTError, match="eps"):
        ttt.gated_residual(x, o, eps=-1.0)
    with pytest.raises(ttt.TTTError, match="aligned"):
        ttt.gated_residual(torch.zeros(4, 66, device="cuda")[:, 1:65], o)
    with pytest.raises(ValueError, match="gamma"):
        ttt.gated_residual(x, o, gamma=torch.ones(63, device="cuda"))
    with pytest.raises(ValueError, match="dtype"):
        ttt.gated_residual(x, o.bfloat16())
    with pytest.raises(ttt.TTTError, match="gamma_next"):
        ttt.gated_residual_backward(x, x.clone(), x.clone(), o)
