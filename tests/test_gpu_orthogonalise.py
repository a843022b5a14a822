"""Newton-Schulz orthogonalisation (ttt.orthogonalise) against the same steps in 64 bits.

Tolerances (relative 2-norm).  Operands carry 22 bits (two fp16 parts; one part, 11 bits, in the last two
steps of bf16 matrices, whose errors grow by 3.4 at most).  The five steps
multiply what is lost along small singular directions by at most 3.4445^5 = 485, while the result's norm
is at least 0.68 sqrt(r) against X's norm 1 before: an error of p in every operand, three products a step,
leaves at most 485 * 3 p / (0.68 sqrt(r)) of it.  With sums of up to c terms (random signs, a root of c
roundings of 2^-24): fp32, r = 16, c = 700: 485 * 3 * 2^-23 / 2.7 = 6.4e-5, worst over directions that
all matrices here fill only in part: held to 1e-5.  bf16: 3.4 * 2^-12 from the last steps, and the result is
rounded by at most 2^-8: held to 2^-8 + 2^-10.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TOL = {torch.bfloat16: 2.0 ** -8 + 2.0 ** -10, torch.float32: 1e-5}


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


def reference(g, steps=5):
    x = g.double().cpu()
    x = x / (x.norm(dim=(-2, -1), keepdim=True) + 1e-7)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT.contiguous() if tall else x
    for _ in range(steps):
        a = x @ x.mT
        x = 3.4445 * x + (-4.7750 * a + 2.0315 * a @ a) @ x
    return x.mT if tall else x


SHAPES = [(1, 1, 1), (1, 1, 9), (2, 16, 16), (3, 63, 65), (1, 64, 64), (2, 130, 70), (1, 33, 700), (1, 700, 96),
          (12, 128, 256), (1, 513, 385), (5, 640, 700), (1, 1100, 2050)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_against_64_bits(shape, dtype):
    from test_weight_layers_amd import ttt
    g = (1e-3 * torch.randn(*shape, generator=torch.Generator().manual_seed(0))).to(dtype)
    ref = reference(g)
    dg = g.cuda()
    out = ttt.orthogonalise(dg)
    err = rel(out, ref)
    print(f"{shape} {dtype}: {err:.2e}")
    assert err <= TOL[dtype]
    assert torch.equal(out, ttt.orthogonalise(dg))
    assert ttt.orthogonalise(dg, out=dg) is dg and torch.equal(dg, out)


@pytest.mark.parametrize("steps", [0, 1, 2, 7])
def test_steps(steps):
    from test_weight_layers_amd import ttt
    g = torch.randn(2, 100, 150, generator=torch.Generator().manual_seed(1))
    assert rel(ttt.orthogonalise(g.cuda(), steps=steps), reference(g, steps)) <= 1e-5


def test_magnitudes_rank_and_zeros():
    from test_weight_layers_amd import ttt
    gen = torch.Generator().manual_seed(2)
    g = torch.randn(90, 120, generator=gen)
    ref = ttt.orthogonalise(g.cuda())
    # the norm is taken out: a power of two changes nothing that 1e-7 beside the norm does not
    for s in (2.0 ** 60, 2.0 ** 100):
        assert rel(ttt.orthogonalise((g * s).cuda()), ref) <= 1e-6
    low = torch.randn(90, 5, generator=gen) @ torch.randn(5, 120, generator=gen)
    assert rel(ttt.orthogonalise(low.cuda()), reference(low)) <= 1e-4   # all but 5 directions hold rounding only
    z = torch.zeros(3, 70, 50, device="cuda")
    z[1] = g[:70, :50].cuda()
    out = ttt.orthogonalise(z)
    assert (out[0] == 0).all() and (out[2] == 0).all() and rel(out[1], reference(g[:70, :50])) <= 1e-5
    bad = z.clone()
    bad[0, 3, 3] = float("nan")
    out2 = ttt.orthogonalise(bad)
    assert out2[0].isnan().all() and torch.equal(out2[1:], out[1:])


def test_strides():
    from test_weight_layers_amd import ttt
    g = torch.randn(4, 80, 60, generator=torch.Generator().manual_seed(3)).cuda()
    ref = ttt.orthogonalise(g)
    wide = torch.full((4, 83, 71), 5.0, device="cuda")
    wide[:, 2:82, 3:63] = g
    assert torch.equal(ttt.orthogonalise(wide[:, 2:82, 3:63]), ref)
    out = torch.full((4, 83, 71), 5.0, device="cuda")
    ttt.orthogonalise(g, out=out[:, 1:81, 7:67])
    assert torch.equal(out[:, 1:81, 7:67], ref)
    out[:, 1:81, 7:67] = 5.0
    assert (out == 5.0).all()
    one = g[:1].expand(3, -1, -1)            # the same matrix three times
    assert torch.equal(ttt.orthogonalise(one), ref[:1].expand(3, -1, -1))
    assert ttt.orthogonalise(g[:0]).shape == (0, 80, 60)


def test_replay():
    from test_weight_layers_amd import ttt
    g = torch.randn(2, 200, 300, device="cuda").bfloat16()
    ttt.orthogonalise(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ttt.orthogonalise(g)
    for seed in range(3):
        new = torch.randn(2, 200, 300, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        g.copy_(new)
        graph.replay()
        ref = ttt.orthogonalise(new)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_refusals():
    from test_weight_layers_amd import ttt
    g = torch.zeros(4, 8, 8, device="cuda")
    with pytest.raises(ValueError, match="stride"):
        ttt.orthogonalise(g.mT[:, :4])
    with pytest.raises(TypeError):
        ttt.orthogonalise(g.half())
    with pytest.raises(ttt.TTTError, match="steps"):
        ttt.orthogonalise(g, steps=-1)
    with pytest.raises(ttt.TTTError, match="overlap"):
        ttt.orthogonalise(g[:2], out=g[1:3])
    with pytest.raises(ttt.TTTError, match="overlap"):
        ttt.orthogonalise(g, out=g[:1].expand(4, -1, -1))
    with pytest.raises(ttt.TTTError, match="workspace"):
        ttt.orthogonalise(g, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="GPU"):
        ttt.orthogonalise(g.cpu())


@pytest.mark.parametrize("shape", [(2, 36, 1216), (1, 1097, 34), (1, 1400, 50), (1, 16, 1400), (200, 64, 100), (200, 100, 64),
                                   (1, 65, 1300), (2, 40, 2048), (1, 8192, 33), (1, 33, 8193), (3, 1, 500)], ids=str)
def test_long_and_narrow(shape):
    """fp32 matrices of few rows or columns, as exact as fp32 steps.  B = a I + b A + c A A is 0.7 where A is
    near I, of terms of 3.4, 4.8 and 2.0, each rounded by 2^-24: 8.7e-7 a step, of which the last two
    remain (an error there is multiplied by about 1).  A's sums of up to 1400 terms are rounded 44 times, a root
    of that at random: 6.6 * 2^-24 * 4.8 / 0.7 = 2.7e-6.  Together below 5e-6."""
    from test_weight_layers_amd import ttt
    g = 1e-3 * torch.randn(*shape, generator=torch.Generator().manual_seed(3))
    err = rel(ttt.orthogonalise(g.cuda()), reference(g))
    print(f"{shape}: {err:.2e}")
    assert err <= 5e-6
    half = g.bfloat16()
    assert rel(ttt.orthogonalise(half.cuda()), reference(half)) <= TOL[torch.bfloat16]
