"""AdamW over many tensors (ttt.adamw_tensors, ttt.adamw_step) against its formula.

32-bit states and weights in fp64: four roundings of 2^-24 each for m and v (relative to terms that do not cancel in the
2-norm), under ten for the weight's step, which is small beside the weight: 8 * 2^-24; bf16 params are the masters (or the
stepped weight) rounded, 2^-8.  8-bit states: the codes are those of the formula in fp32, step by step as documented:
equal; the values that they stand for are off by at most half a code's distance.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
BETAS, LR, EPS, WD = (0.9, 0.99), 1e-2, 1e-8, 0.1


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


def make(sizes, dtype, bits, master, seed=0, offset=0):
    """Tensors of the sizes; offset: elements by which their storage begins off 16 bytes."""
    g = torch.Generator().manual_seed(seed)

    def new(n, dt, fill=None):
        t = torch.empty(n + offset, dtype=dt, device="cuda")[offset:]
        return t.zero_() if fill is None else t.copy_(fill.to(dt))

    rn = lambda n: torch.randn(n, generator=g)
    s = dict(p=[new(n, dtype, rn(n)) for n in sizes])
    if master:
        s["master"] = [new(n, F32, rn(n)) for n in sizes]
    if bits == 32:
        s["m"], s["v"] = [new(n, F32) for n in sizes], [new(n, F32) for n in sizes]
    else:
        s["m"], s["v"] = [new(n, torch.int8) for n in sizes], [new(n, torch.uint8) for n in sizes]
        s["ms"], s["vs"] = ([new(-(-n // 256), F32) for n in sizes] for _ in range(2))
    return s, lambda: [new(n, dtype, rn(n) * torch.exp(rn(n))) for n in sizes]


def handle(s):
    from test_weight_layers_amd import ttt
    return ttt.adamw_tensors(s["p"], s["m"], s["v"], master=s.get("master"), exp_avg_scales=s.get("ms"), exp_avg_sq_scales=s.get("vs"))


def values(c, s, top):
    """What 8-bit codes stand for, in the kernel's order of fp32 operations."""
    c = c.int()
    return (c * c.abs()).float() * (1.0 / top ** 2) * s.repeat_interleave(256)[:c.numel()]


def codes(x, top):
    """The codes of x and their scales."""
    n = x.numel()
    b = torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256)
    s = b.abs().amax(1)
    r = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    c = torch.round(((b.abs() * r[:, None]).sqrt()) * float(top)) * torch.sign(b)
    return c.view(-1)[:n], s


def reference(w, g, m, v, t, scale=1.0):
    g = g * scale
    m = m * BETAS[0] + g * (1 - BETAS[0])
    v = v * BETAS[1] + (g * g) * (1 - BETAS[1])
    c1, c2 = LR / (1 - BETAS[0] ** t), 1 / math.sqrt(1 - BETAS[1] ** t)
    return w * (1 - LR * WD) - (m * c1) / (v.sqrt() * c2 + EPS), m, v


SIZES = [1, 7, 8, 255, 256, 257, 2048, 2049, 5000, 100003]
MANY = [3 + 37 * i for i in range(130)]          # more tensors than one launch takes


@pytest.mark.parametrize("sizes", [SIZES, MANY], ids=["sizes", "many"])
@pytest.mark.parametrize("dtype,master", [(F32, False), (BF, False), (BF, True)], ids=["f32", "bf16", "master"])
@pytest.mark.parametrize("offset", [0, 1], ids=["aligned", "offset"])
def test_32_bit_states(sizes, dtype, master, offset):
    from test_weight_layers_amd import ttt
    s, grads = make(sizes, dtype, 32, master, offset=offset)
    h = handle(s)
    w = [x.double() for x in s["master" if master else "p"]]
    m, v = [torch.zeros_like(x) for x in w], [torch.zeros_like(x) for x in w]
    for t in (1, 2, 3):
        g = grads()
        old = [x.double() for x in s["p"]]
        ttt.adamw_step(h, g, step=t, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD)
        for i in range(len(sizes)):
            # (params without a master are rounded every step: each step is compared from where it began)
            start = w[i] if master or dtype == F32 else old[i]
            w[i], m[i], v[i] = reference(start, g[i].double(), m[i], v[i], t)
            assert rel(s["m"][i], m[i]) <= 2.0 ** -21 and rel(s["v"][i], v[i]) <= 2.0 ** -21, (t, sizes[i])
            if master:
                assert rel(s["master"][i], w[i]) <= 2.0 ** -21 and torch.equal(s["p"][i], s["master"][i].to(dtype)), sizes[i]
            else:
                assert rel(s["p"][i], w[i]) <= (2.0 ** -21 if dtype == F32 else 2.0 ** -8), sizes[i]


@pytest.mark.parametrize("sizes", [SIZES, MANY], ids=["sizes", "many"])
@pytest.mark.parametrize("dtype,master", [(F32, False), (BF, True)], ids=["f32", "master"])
@pytest.mark.parametrize("offset", [0, 1], ids=["aligned", "offset"])
def test_8_bit_states(sizes, dtype, master, offset):
    from test_weight_layers_amd import ttt
    s, grads = make(sizes, dtype, 8, master, offset=offset)
    h = handle(s)
    for t in (1, 2, 3):
        g = grads()
        before = {k: [x.clone() for x in s[k]] for k in s}
        ttt.adamw_step(h, g, step=t, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD)
        for i in range(len(sizes)):
            m, r = values(before["m"][i], before["ms"][i], 127), values(before["v"][i], before["vs"][i], 255)
            w = before["master" if master else "p"][i].float()
            w, m, v = reference(w, g[i].float(), m, r * r, t)
            cm, ms = codes(m, 127)
            cv, vs = codes(v.sqrt(), 255)
            assert torch.equal(s["ms"][i], ms) and torch.equal(s["vs"][i], vs), (t, sizes[i])
            assert torch.equal(s["m"][i].float(), cm) and torch.equal(s["v"][i].float(), cv), (t, sizes[i])
            got = s["master" if master else "p"][i]
            assert torch.equal(got, w.to(got.dtype)), (t, sizes[i])
            # a code stands for a value at most half the way to its neighbour from it: (2 c + 1) / 2 of s / top^2 away
            held, c = values(s["m"][i], ms, 127).double(), s["m"][i].double().abs()
            step = (c + 0.5) * 1.0001 / 127 ** 2 * ms.double().repeat_interleave(256)[:sizes[i]]
            assert ((held - m.double()).abs() <= step).all()


def test_scale_step_and_rate_on_the_gpu():
    from test_weight_layers_amd import ttt
    sizes = [300, 4097]
    s, grads = make(sizes, F32, 32, False)
    s2, _ = make(sizes, F32, 32, False)
    h, h2 = handle(s), handle(s2)
    step, lr = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, device="cuda")
    gs = torch.ones(1, device="cuda")
    g = grads()
    torch.cuda.synchronize()
    start = [x.clone() for x in s["p"]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        ttt.adamw_step(h, g, step=step, lr=lr, betas=BETAS, eps=EPS, weight_decay=WD, grad_scale=gs)
    assert all(torch.equal(a, b) for a, b in zip(s["p"], start))
    for t in (1, 2, 3, 4):
        new, scale = grads(), 0.25 * t
        for a, b in zip(g, new):
            a.copy_(b)
        lr.fill_(LR / t), gs.fill_(scale)
        graph.replay()
        # (the rate as the GPU has it: rounded to fp32)
        ttt.adamw_step(h2, [x * scale for x in new], step=t, lr=float(lr.item()), betas=BETAS, eps=EPS, weight_decay=WD)
        torch.cuda.synchronize()
        for k in ("p", "m", "v"):
            for a, b in zip(s[k], s2[k]):
                assert rel(a, b) <= 2.0 ** -22        # (the host's and the GPU's power differ in a last digit)


@pytest.mark.parametrize("bits", [32, 8])
def test_what_is_not_finite_stays_where_it_is(bits):
    from test_weight_layers_amd import ttt
    sizes = [1000, 500]
    s, grads = make(sizes, F32, bits, False)
    s2, _ = make(sizes, F32, bits, False)
    h, h2 = handle(s), handle(s2)
    g = grads()
    bad = [x.clone() for x in g]
    bad[0][300] = float("nan")
    bad[0][700] = float("inf")
    for t in (1, 2):
        ttt.adamw_step(h, g, step=t, lr=LR)
        ttt.adamw_step(h2, bad, step=t, lr=LR)
    keep = torch.ones(1000, dtype=torch.bool, device="cuda")
    for i in (300, 700):
        keep[(slice(i, i + 1) if bits == 32 else slice(i // 256 * 256, i // 256 * 256 + 256))] = False
    assert torch.equal(s["p"][1], s2["p"][1]) and torch.equal(s["p"][0][keep], s2["p"][0][keep])
    assert s2["p"][0][300].isnan() and not torch.isfinite(s2["p"][0][700])
    if bits == 8:                                    # (the second step reads a state that is not finite)
        assert not torch.isfinite(s2["p"][0][256:512]).any()


def test_empty_tensors_and_zero_gradients():
    from test_weight_layers_amd import ttt
    for bits in (32, 8):
        s, grads = make([0, 5, 0, 300], F32, bits, False)
        h = handle(s)
        start = [x.clone() for x in s["p"]]
        ttt.adamw_step(h, [torch.zeros_like(x) for x in s["p"]], step=1, lr=LR)
        assert all(torch.equal(a, b) for a, b in zip(s["p"], start))
        assert all((x == 0).all() for k in ("m", "v") for x in s[k])


def test_refusals():
    from test_weight_layers_amd import ttt
    s, grads = make([300, 20], F32, 32, False)
    h, g = handle(s), grads()
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        ttt.adamw_step(h, [g[0], g[1].bfloat16()], step=1, lr=LR)
    with pytest.raises(ValueError, match="grads must hold"):
        ttt.adamw_step(h, g[:1], step=1, lr=LR)
    with pytest.raises(ttt.TTTError, match="step"):
        ttt.adamw_step(h, g, step=0, lr=LR)
    with pytest.raises(ttt.TTTError, match="beta"):
        ttt.adamw_step(h, g, step=1, lr=LR, betas=(1.0, 0.9))
    with pytest.raises(ttt.TTTError, match="lr"):
        ttt.adamw_step(h, g, step=1, lr=float("nan"))
    with pytest.raises(ValueError, match="step must be"):
        ttt.adamw_step(h, g, step=torch.ones(1, device="cuda"), lr=LR)
    with pytest.raises(ttt.TTTError, match="overlap"):
        ttt.adamw_tensors([s["p"][0], s["p"][0]], [s["m"][0], s["v"][0]], [x.clone() for x in (s["m"][0], s["v"][0])])
    with pytest.raises(ttt.TTTError, match="overlap"):
        ttt.adamw_tensors(s["p"], s["m"], s["m"])
    with pytest.raises(ValueError, match="scales"):
        ttt.adamw_tensors(s["p"], s["m"], s["v"], exp_avg_scales=s["m"])
    with pytest.raises(ValueError, match="exp_avg"):
        ttt.adamw_tensors(s["p"], s["m"][:1], s["v"])
    with pytest.raises(ValueError, match="contiguous"):
        ttt.adamw_tensors([torch.zeros(4, 8, device="cuda").t()], [torch.zeros(32, device="cuda")], [torch.zeros(32, device="cuda")])


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_empty_tensors_beside_masters(dtype, bits):
    """A table with empty tensors steps the others as the table without them does: the same bits."""
    from test_weight_layers_amd import ttt
    sizes = [0, 300, 0, 0, 1029, 0]
    s, grads = make(sizes, dtype, bits, True)
    assert s["master"][0].data_ptr() == 0
    full = [i for i, n in enumerate(sizes) if n]
    alone = {k: [x[i].clone() for i in full] for k, x in s.items()}
    h, h2 = handle(s), handle(alone)
    for step in (1, 2, 3):
        g = grads()
        ttt.adamw_step(h, g, step=step, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD)
        ttt.adamw_step(h2, [g[i] for i in full], step=step, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD)
    for k, x in s.items():
        assert all(torch.equal(x[i], y) for i, y in zip(full, alone[k])), k
    assert s["m"][1].any() and not torch.equal(s["master"][1], make(sizes, dtype, bits, True)[0]["master"][1])


@pytest.mark.parametrize("name", ["p", "master"])
def test_moved_tensors_are_refused(name):
    """A tensor whose data is set anew is not stepped where it was."""
    from test_weight_layers_amd import ttt
    s, grads = make([300, 20], BF, 32, True)
    h, g = handle(s), grads()
    ttt.adamw_step(h, g, step=1, lr=LR)
    held = s[name][1].detach()
    s[name][1].data = s[name][1].clone()
    before = held.clone()
    with pytest.raises(ValueError, match="moved"):
        ttt.adamw_step(h, g, step=2, lr=LR)
    assert torch.equal(held, before) and torch.equal(s[name][1], before)
    ttt.adamw_step(handle(s), g, step=2, lr=LR)
    s2, grads2 = make([300, 20], BF, 32, True)
    h2, g2 = handle(s2), grads2()
    for step in (1, 2):
        ttt.adamw_step(h2, g2, step=step, lr=LR)
    assert all(torch.equal(a, b) for k in s for a, b in zip(s[k], s2[k])) and not torch.equal(held, s[name][1])
