"""Layer norm (ttt.layer_norm and its gradient) against the formulas in 64 bits.

Tolerances (relative 2-norm).  Everything is fp32 and rounded once at the end: at most 2^-8 of each bf16 element.  The
fp32 arithmetic before it: sums of up to 8192 terms (16 a lane, then log2 steps: under 40 roundings of 2^-24), a square
root, a reciprocal and five products: below 64 * 2^-24 = 4e-6.  Sums over rows: at most 6000 terms, of random sign, in
partial sums of a lane, a workgroup and the workgroups: 64 * 2^-24 as well.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 2.0 ** -8, F32: 4e-6}


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


def forward(x, gamma, beta, eps, w):
    x = x.unflatten(1, (-1, w))
    c = x - x.mean(-1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    return ((y if gamma is None else y * gamma) + (0 if beta is None else beta)).flatten(1)


def rows(n, C, dtype, g, mean=0.0):
    """[n, C] rows that begin on 16 bytes, whatever C is."""
    ld = -(-C // 8) * 8
    x = torch.full((n, ld), float("nan"), dtype=dtype)
    x[:, :C] = (mean + torch.randn(n, C, generator=g)).to(dtype)
    return x.cuda()[:, :C]


CASES = [
    # n, channels, norm width, dtype
    (1, 1, 1, F32), (3, 2, 2, BF), (1, 8, 8, F32), (5, 64, 64, BF), (37, 67, 67, F32), (130, 120, 24, BF),
    (33, 256, 64, F32), (70, 504, 504, BF), (1374, 1024, 64, BF), (259, 1000, 1000, F32), (64, 1029, 1029, BF),
    (300, 1536, 768, F32), (41, 2047, 2047, BF), (19, 3584, 3584, BF), (23, 4000, 400, F32), (9, 8192, 8192, BF),
    (7, 8191, 8191, F32), (6000, 72, 72, BF), (2, 12288, 4096, F32),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_gradient(case):
    from test_weight_layers_amd import ttt
    n, C, w, dtype = case
    g = torch.Generator().manual_seed(n)
    x, gy = rows(n, C, dtype, g, 0.5), rows(n, C, dtype, g)
    ga, be = (1.0 + 0.3 * torch.randn(w, generator=g)).cuda(), torch.randn(w, generator=g).cuda()
    xd, gad, bed = (t.double().requires_grad_(True) for t in (x, ga, be))
    ref = forward(xd, gad, bed, 1e-6, w)
    grads_ref = torch.autograd.grad(ref, (xd, gad, bed), gy.double())
    y = ttt.layer_norm(x, ga, be, 1e-6, norm_width=w)
    assert y.shape == x.shape and rel(y, ref.detach()) <= TOL[dtype]
    got = ttt.layer_norm_backward(gy, x, ga, 1e-6, norm_width=w)
    again = ttt.layer_norm_backward(gy, x, ga, 1e-6, norm_width=w)
    for name, a, b, r in zip(("x", "gamma", "beta"), got, again, grads_ref):
        assert torch.equal(a, b) and a.shape == r.shape
        # a vector of one or two elements: its gradient is what eps leaves of terms of the size of gy / sqrt(var)
        base = max(r.norm().item(), 0.1 * gy.double().norm().item() if w <= 2 else 0.0)
        assert (a.double() - r).norm().item() <= TOL[a.dtype] * base, name
    x2, g2 = x.clone(), gy.clone()
    if x2.stride(0) % 8 == 0 or x2.shape[0] == 1 and C % 8 == 0:
        assert torch.equal(ttt.layer_norm(x2, ga, be, 1e-6, norm_width=w, out=x2), y)
        assert torch.equal(ttt.layer_norm_backward(g2, x, ga, 1e-6, norm_width=w, out=g2)[0], got[0])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_large_means(dtype):
    """A mean of 1000 deviations: the squares are taken of what is left of x, which fp32 holds exactly."""
    from test_weight_layers_amd import ttt
    x = rows(64, 1000, dtype, torch.Generator().manual_seed(1), 1000.0)
    assert rel(ttt.layer_norm(x), forward(x.double(), None, None, 1e-6, 1000)) <= TOL[dtype]


def test_left_out_parts_and_no_rows():
    from test_weight_layers_amd import ttt
    g = torch.Generator().manual_seed(2)
    x, gy = rows(50, 128, F32, g), rows(50, 128, F32, g)
    one, zero = torch.ones(128, device="cuda"), torch.zeros(128, device="cuda")
    assert torch.equal(ttt.layer_norm(x), ttt.layer_norm(x, one, zero))
    for a, b in zip(ttt.layer_norm_backward(gy, x), ttt.layer_norm_backward(gy, x, one)):
        assert torch.equal(a, b)
    e = torch.empty(0, 128, device="cuda")
    assert ttt.layer_norm(e).shape == (0, 128)
    gx, gg, gb = ttt.layer_norm_backward(e, e.clone())
    assert gx.shape == (0, 128) and (gg == 0).all() and (gb == 0).all()
    z = torch.zeros(3, 64, device="cuda")
    assert (ttt.layer_norm(z) == 0).all()
    x2 = x.clone()
    x2[4, 7] = float("nan")
    y, y2 = ttt.layer_norm(x), ttt.layer_norm(x2)
    keep = torch.arange(50, device="cuda") != 4
    assert torch.equal(y[keep], y2[keep]) and y2[4].isnan().all()


def test_replay():
    from test_weight_layers_amd import ttt
    g = torch.Generator().manual_seed(3)
    x, gy, ga = rows(3000, 768, BF, g), rows(3000, 768, BF, g), torch.randn(64, generator=g).cuda()
    ttt.layer_norm_backward(gy, x, ga, norm_width=64)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ttt.layer_norm(x, ga, norm_width=64)
        grads = ttt.layer_norm_backward(gy, x, ga, norm_width=64)
    for _ in range(3):
        x.copy_(rows(3000, 768, BF, g))
        graph.replay()
        ref, gref = ttt.layer_norm(x.clone(), ga, norm_width=64), ttt.layer_norm_backward(gy, x.clone(), ga, norm_width=64)
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and all(torch.equal(a, b) for a, b in zip(grads, gref))


def test_refusals():
    from test_weight_layers_amd import ttt
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ttt.TTTError, match="norm_width"):
        ttt.layer_norm(x, norm_width=48)
    with pytest.raises(ttt.TTTError, match="norm_width"):
        ttt.layer_norm(x, norm_width=4)
    with pytest.raises(ttt.TTTError, match="norm_width"):
        ttt.layer_norm(torch.zeros(1, 8200, device="cuda"))
    with pytest.raises(ttt.TTTError, match="aligned"):
        ttt.layer_norm(torch.zeros(4, 63, device="cuda"))
    with pytest.raises(ttt.TTTError, match="eps"):
        ttt.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError, match="gamma"):
        ttt.layer_norm(x, torch.ones(64, device="cuda"), norm_width=32)
    with pytest.raises(ttt.TTTError, match="overlap"):
        ttt.layer_norm_backward(x.clone(), x, out=x)
    with pytest.raises(ValueError, match="grad_y"):
        ttt.layer_norm_backward(x[:3], x)


def test_width_beyond_32_bits():
    """A width of 2^32 + 64 is not one of 64."""
    from test_weight_layers_amd import ttt
    x = torch.zeros(4, 64, device="cuda")
    for width in ((1 << 32) + 64, (1 << 32) + 32, 1 << 31, -(1 << 32) + 64):
        for call in (lambda: ttt.layer_norm(x, norm_width=width), lambda: ttt.layer_norm_backward(x.clone(), x, norm_width=width),
                     lambda: ttt.gated_residual(x, x.clone(), norm_width=width),
                     lambda: ttt.gated_residual_backward(x, None, x.clone(), x.clone(), norm_width=width)):
            with pytest.raises(ValueError, match="norm_width"):
                call()
