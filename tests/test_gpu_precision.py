"""How exact the operators beside the layer are beyond the rounding of their outputs.

bf16 outputs are compared with the 64-bit values rounded to bf16.  Before its one rounding a value v is off by
some e: it rounds to another number only where a border lies between, with probability |e| / u for a spacing
u <= 2^-7 |v|, and the difference then is u.  The sum of squares of the differences is at most
sum |e| u <= 2^-7 |e|_2 |v|_2, so arithmetic held to a relative error E leaves at most sqrt(2^-7 E) between the two.
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
    x, ref = x.double(), ref.double()
    assert torch.isfinite(x).all()
    return ((x - ref).norm() / ref.norm()).item()


def borders(x, ref):
    """How far x is from the 64-bit reference rounded as x is."""
    return rel(x, ref.to(x.dtype))


def limit(e):
    return math.sqrt(2.0 ** -7 * e)


# ------------------------------------------------------------------ gated delta rule
def delta_inputs(lens, H, Hk, dk, dv, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)
    n = sum(lens)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    d = dict(q=unit(rn(n, Hk, dk)).reshape(n, -1), k=unit(rn(n, Hk, dk)).reshape(n, -1), v=rn(n, H * dv), go=rn(n, H * dv))
    d = {x: t.bfloat16() for x, t in d.items()}
    d["beta"] = torch.sigmoid(rn(H, n)).float()
    d["decay"] = (-0.05 * torch.exp(rn(H, n))).float()
    for x in ("w", "gw"):
        d[x] = (rn(len(lens), H, dv, dk) / math.sqrt(dk)).float()
    d["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    return d


def delta_reference(d, lens, Hk):
    """Outputs, states and gradients token by token in 64 bits."""
    S, H, dv, dk = d["w"].shape
    n, r = d["q"].shape[0], H // Hk
    heads = lambda t, m: t.double().view(n, -1, m).repeat_interleave(H // (t.shape[1] // m), 1)
    q, k, v, go = heads(d["q"], dk), heads(d["k"], dk), heads(d["v"], dv), heads(d["go"], dv)
    be, a = d["beta"].double().t(), d["decay"].double().exp().t()
    o, dq, dk_, dvv = torch.zeros_like(v), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dbe, dde = torch.zeros_like(be), torch.zeros_like(be)
    wf, gw0 = [], []
    at = 0
    for s in range(S):
        w, kept = d["w"][s].double(), []
        for t in range(at, at + lens[s]):
            kept.append(w * a[t][:, None, None])
            e = v[t] - (kept[-1] * k[t][:, None, :]).sum(-1)
            w = kept[-1] + (be[t][:, None] * e)[:, :, None] * k[t][:, None, :]
            o[t] = (w * q[t][:, None, :]).sum(-1)
        wf.append(w)
        dw = d["gw"][s].double()
        for t in reversed(range(at, at + lens[s])):
            p = kept[t - at]
            e = v[t] - (p * k[t][:, None, :]).sum(-1)
            w = p + (be[t][:, None] * e)[:, :, None] * k[t][:, None, :]
            dq[t] = (go[t][:, :, None] * w).sum(1)
            dw = dw + go[t][:, :, None] * q[t][:, None, :]
            g = (dw * k[t][:, None, :]).sum(-1)
            dbe[t] = (g * e).sum(-1)
            dvv[t] = be[t][:, None] * g
            dk_[t] = ((be[t][:, None] * e)[:, :, None] * dw - dvv[t][:, :, None] * p).sum(1)
            dw = dw - dvv[t][:, :, None] * k[t][:, None, :]
            dde[t] = (dw * p).sum((1, 2))
            dw = dw * a[t][:, None, None]
        gw0.append(dw)
        at += lens[s]
    shared = lambda t: t.view(n, Hk, r, dk).sum(2).reshape(n, -1)
    grads = shared(dq), shared(dk_), dvv.reshape(n, -1), dbe.t(), dde.t(), torch.stack(gw0)
    return o.reshape(n, -1), torch.stack(wf), grads


# The first is cut in segments that run at once, the others are not.
DELTA = [([1100], 4, 4, 64, 256), ([300, 0, 1, 200], 6, 2, 128, 128), ([260, 250], 4, 4, 256, 256)]


@pytest.mark.parametrize("case", DELTA, ids=str)
def test_delta(case):
    """Arithmetic as exact as fp32 has it.  Operands carry 24 bits; a sum of up to 256 products is rounded once a
    matrix instruction, at most 48 times (8 blocks of 32 terms, 6 pairs of parts), of random sign: 7 * 2^-24 =
    4.1e-7, and five such sums follow one another (their errors add as a root): 9.3e-7.  Outputs and states are held to
    1e-6; the gradients pass through the forward's five and the backward's five, 1.4e-6, and of a rate through a
    sum that cancels in part: 2e-6."""
    from test_weight_layers_amd import ttt
    lens, H, Hk, dk, dv = case
    d = delta_inputs(lens, H, Hk, dk, dv, 1)
    o_ref, w_ref, g_ref = delta_reference(d, lens, Hk)
    args = [d[x] for x in ("w", "q", "k", "v", "beta", "decay")]
    o, w = ttt.delta(*args, key_heads=Hk, cu_seqlens=d["cu"])
    grads = ttt.delta_backward(*args, d["go"], d["gw"], key_heads=Hk, cu_seqlens=d["cu"])
    names = ("q", "k", "v", "beta", "decay", "w")
    got = {"o": (borders(o, o_ref), limit(1e-6)), "states": (rel(w, w_ref), 1e-6)}
    for x, g, r in zip(names, grads, g_ref):
        got["grad " + x] = (borders(g, r), limit(2e-6)) if x in "qkv" else (rel(g, r), 2e-6)
    print({x: f"{a:.2e} of {b:.2e}" for x, (a, b) in got.items()})
    assert all(a <= b for a, b in got.values()), got


def test_delta_gradients_inside_a_chunk():
    """Sequences of one chunk from zero states, whose final states count for nothing: the gradients of q and k are
    those of the 64 x 64 terms alone.  Roundings on the way, counted as above: of K K^T and Q K^T 8 instructions (1.7e-7),
    of D 2^-23, of a substitution over 64 tokens 64 (4.8e-7), of T R, A^T go and T^T dU 6 to 12 (1.5e-7 to 2.1e-7), of
    go U^T and dR U^T 6 to 12, of the last sums 6 each.  For q the root of their squares' sum is below 7e-7, for k,
    which takes the substitution twice, below 9e-7."""
    from test_weight_layers_amd import ttt
    lens, H = [64] * 12 + [50] * 4, 4
    d = delta_inputs(lens, H, H, 256, 64, 2)
    d["w"].zero_(), d["gw"].zero_()
    ref = delta_reference(d, lens, H)[2]
    got = ttt.delta_backward(*[d[x] for x in ("w", "q", "k", "v", "beta", "decay")], d["go"], None, cu_seqlens=d["cu"])
    off = borders(got[0], ref[0]), borders(got[1], ref[1])
    print(f"q {off[0]:.2e} of {limit(7e-7):.2e}, k {off[1]:.2e} of {limit(9e-7):.2e}")
    assert off[0] <= limit(7e-7) and off[1] <= limit(9e-7)


# ------------------------------------------------------------------ gated residual tail
def test_gate_of_fp32_rows():
    """o = +-1 and no eps: the norm is exactly 1, and y is the gate alone, z / (1 + e^-z): an exponential (2^-23),
    a sum, a quotient and a product (2^-24 each), and the square root's and quotient's of the norm: 8 * 2^-24 of every
    element.  The gradient of z adds the sigmoid of -z, two products and a sum: 16 * 2^-24, its largest being
    1.1."""
    from test_weight_layers_amd import ttt
    C = 256
    z = torch.linspace(-80.0, 80.0, 64 * C, device="cuda").view(64, C)
    o = torch.where(torch.arange(C, device="cuda") % 3 == 0, -1.0, 1.0).expand(64, C).contiguous()
    y, _ = ttt.gated_residual(torch.zeros_like(z), o, z, eps=0.0)
    zd = z.double()
    s = torch.sigmoid(zd)
    ref = o.double() * zd * s
    off = ((y.double() - ref).abs() / ref.abs()).max().item()
    gz = ttt.gated_residual_backward(torch.ones_like(z), None, y, o, z, eps=0.0)[2]
    want = o.double() * s * (1 + zd * (1 - s))
    goff = (gz.double() - want).abs().max().item()
    print(f"gate {off:.2e}, gradient {goff:.2e}")
    assert off <= 8 * 2.0 ** -24 and goff <= 16 * 2.0 ** -24
    # beyond what an exponential reaches: z itself, 0, infinity, and not a number only where it stands
    far = torch.tensor([200.0, 3e38, math.inf, -200.0, -3e38, math.nan, 0.0, 1.0], device="cuda")[None]
    y, _ = ttt.gated_residual(torch.zeros_like(far), torch.ones_like(far), far, eps=0.0)
    assert torch.equal(y[0, :5], torch.tensor([200.0, 3e38, math.inf, 0.0, 0.0], device="cuda"))
    assert y[0, 5].isnan() and y[0, 6] == 0 and abs(y[0, 7].item() - 1 / (1 + math.exp(-1))) <= 8 * 2.0 ** -24
    gz = ttt.gated_residual_backward(torch.ones_like(far), None, y, torch.ones_like(far), far, eps=0.0)[2]
    assert torch.equal(gz[0, [0, 1, 3, 4, 6]], torch.tensor([1.0, 1.0, 0.0, 0.0, 0.5], device="cuda")) and gz[0, 5].isnan()


@pytest.mark.parametrize("C,norm", [(8192, 4096), (8176, 4088), (2048, 1024)], ids=str)
def test_wide_groups(C, norm):
    """One element of eight is 3967 / 2048, whose square is exact: added one after another the squares of 512 such
    round the same way again and again (7.6e-6 of the sum).  40 roundings in a row at most, halved by the root, and
    8 after it: 28 * 2^-24."""
    from test_weight_layers_amd import ttt
    o = torch.zeros(3, C, device="cuda")
    o[:, ::8] = 3967 / 2048
    y, _ = ttt.gated_residual(torch.zeros_like(o), o, eps=0.0, norm_width=norm)
    off = (y[:, ::8].double() / math.sqrt(8.0) - 1.0).abs().max().item()
    print(f"{off:.2e}")
    assert off <= 28 * 2.0 ** -24


@pytest.mark.parametrize("C,norm", [(8176, 4088), (6144, 2048), (7200, 2400), (2048, 1024), (4096, 1024), (2040, 680),
                                    (600, 120)], ids=str)
def test_groups_of_many_lanes(C, norm):
    """Values and gradients against the formula, the groups apart from one another.  Under 64 roundings of 2^-24 in a
    row: 8 squares of a lane, two levels of at most 23 sums, the root, a quotient and the products."""
    from test_weight_layers_amd import ttt
    gen = torch.Generator(device="cuda").manual_seed(8)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    n = 5
    x, z, gy = rn(n, C), rn(n, C), rn(n, C)
    # each group of a size of its own
    o = rn(n, C) * torch.logspace(-2, 2, n * (C // norm), device="cuda").view(n, -1).repeat_interleave(norm, 1)
    y, _ = ttt.gated_residual(x, o, z, norm_width=norm)
    od, zd = o.double().requires_grad_(True), z.double().requires_grad_(True)
    og = od.view(n, -1, norm)
    u = (og / torch.sqrt((og * og).mean(-1, keepdim=True) + 1e-6)).view(n, C) * zd * torch.sigmoid(zd)
    go_ref, gz_ref = torch.autograd.grad(u, (od, zd), gy.double())
    got = ttt.gated_residual_backward(gy, None, y, o, z, norm_width=norm)
    scale = o.double().abs()        # the gradient of a group is as large as its o is small
    off = rel(y, x.double() + u.detach()), rel(got[1].double() * scale, go_ref * scale), rel(got[2], gz_ref)
    print([f"{e:.1e}" for e in off])
    assert max(off) <= 64 * 2.0 ** -24


# ------------------------------------------------------------------ orthogonalisation
def orth_reference(g, steps):
    x = g.double()
    x = x / (x.norm(dim=(-2, -1), keepdim=True) + 1e-7)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT.contiguous() if tall else x
    for _ in range(steps):
        a = torch.matmul(x, x.mT.contiguous())
        x = 3.4445 * x + torch.matmul(-4.7750 * a + 2.0315 * torch.matmul(a, a), x)
    return x.mT if tall else x


@pytest.mark.parametrize("steps", [1, 2, 3, 5])
@pytest.mark.parametrize("shape", [(5, 200, 300), (2, 700, 400)], ids=str)
def test_orthogonalise_bf16(shape, steps):
    """As exact as fp32 matrices are (1e-5), then one rounding."""
    from test_weight_layers_amd import ttt
    g = (1e-3 * torch.randn(*shape, generator=torch.Generator().manual_seed(5))).bfloat16().cuda()
    off = borders(ttt.orthogonalise(g, steps=steps), orth_reference(g, steps))
    print(f"{off:.2e} of {limit(1e-5):.2e}")
    assert off <= limit(1e-5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(3, 100, 200), (1, 300, 280)], ids=str)
def test_orthogonalise_small_directions_beside_a_large_one(shape, dtype):
    """A matrix of rank one and noise of a hundredth of its size, which the steps multiply by up to 3.4445^5 = 485
    while the large direction stays near 1: what is lost of the large elements shows in the noise.  With p lost of
    every operand (22 bits: 2^-23), three products a step and a result of norm 0.25 sqrt(r) at least, off by
    485 * 3 p / (0.25 sqrt(r)): 6.9e-5 for r = 100, 4.1e-5 for 280."""
    from test_weight_layers_amd import ttt
    b, r, c = shape
    gen = torch.Generator().manual_seed(6)
    rn = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    g = (rn(b, r, 1) * rn(b, 1, c) + 1e-2 * rn(b, r, c)).to(dtype).cuda()
    ref = orth_reference(g, 5)
    assert ref.norm() >= 0.25 * math.sqrt(b * min(r, c))
    got, e = ttt.orthogonalise(g), 485 * 3 * 2.0 ** -23 / (0.25 * math.sqrt(min(r, c)))
    off, most = (borders(got, ref), limit(e)) if dtype == torch.bfloat16 else (rel(got, ref), e)
    print(f"{off:.2e} of {most:.2e}")
    assert off <= most


def test_orthogonalise_elements_of_bf16():
    """Diagonal matrices, whose elements stay apart: each is a product of numbers of 22 bits, off by at most 3 * 2^-22
    in each of the six products of two steps (4.3e-6, held to 1e-5) before it is rounded, by at most half a spacing."""
    from test_weight_layers_amd import ttt
    d = (0.5 + 0.5 * torch.rand(3000, 100, generator=torch.Generator().manual_seed(7))).bfloat16().cuda()
    got = ttt.orthogonalise(torch.diag_embed(d), steps=2)
    x = d.double() / (d.double().norm(dim=1, keepdim=True) + 1e-7)
    for _ in range(2):
        x = x * (3.4445 - 4.7750 * x ** 2 + 2.0315 * x ** 4)
    half = 2.0 ** (torch.floor(torch.log2(x)) - 8)
    off = (got.diagonal(dim1=1, dim2=2).double() - x).abs() - half
    print(f"{(off > 1e-5 * x).sum().item()} of {x.numel()} elements, {(off / x).max().item():.1e}")
    assert (off <= 1e-5 * x).all()
    assert got.count_nonzero() == x.numel()


# Every pair of tile sizes: of B X, and of the symmetric A and B.
TILES = [((3, 200, 300), 64, 64), ((120, 100, 120), 64, 128), ((5, 1300, 1390), 128, 128), ((30, 250, 1000), 128, 64),
         ((2, 1300, 5100), 256, 128), ((2, 5100, 1300), 256, 128), ((3, 200, 20000), 256, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape,tile,sym", TILES, ids=str)
def test_orthogonalise_tiles(shape, tile, sym, dtype):
    """Each step has products of its own (X enters the first in one part where it is bf16, the last writes the result):
    1, 2 and 5 of them.  Sizes leave a part of the last tile empty.  fp32 is held to 1e-5."""
    from test_weight_layers_amd import ttt
    b, r, c = shape
    # the tiles are chosen as the padded sizes in the workspace say
    pad = max(tile, sym)
    rp, cp = (-(-x // pad) * pad for x in (min(r, c), max(r, c)))
    up = lambda x: -(-x // 256) * 256
    blocks = min(256, -(-r * c // 4096))
    assert ttt.orthogonalise_workspace_bytes(r, c, b, dtype) == (up(b * blocks * 8) + up(b * 4) + 4 * up(rp * cp * 4 * b)
                                                                 + 2 * up(rp * rp * 4 * b))
    g = torch.randn(*shape, generator=torch.Generator().manual_seed(9)).to(dtype).cuda()
    for steps in (1, 2, 5):
        ref = orth_reference(g, steps)
        got = ttt.orthogonalise(g, steps=steps)
        off, most = (borders(got, ref), limit(1e-5)) if dtype == torch.bfloat16 else (rel(got, ref), 1e-5)
        print(f"{steps}: {off:.2e} of {most:.2e}")
        assert off <= most
        assert torch.equal(got, ttt.orthogonalise(g, steps=steps))
