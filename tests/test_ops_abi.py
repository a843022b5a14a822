"""Argument checks and workspace queries of the delta-rule, gated-residual and orthogonalisation entry
points, without a GPU.  Made-up addresses are passed only where no GPU is visible, and every check
rejects them before any launch."""
import ctypes
import os

import pytest
import torch

from test_weight_layers_amd import ttt

F32, BF16 = ttt.TTT_F32, ttt.TTT_BF16
BIG = 1 << 40
cpu_only = pytest.mark.skipif(torch.cuda.device_count() > 0,
                              reason="passes made-up device addresses; CPU-only by design")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ttt.LIB_PATH):
        pytest.fail("libttt.so is not built; run __graft_entry__.build()")
    return ttt.load()


def ws(lib, fn, *args):
    out = ctypes.c_size_t()
    return getattr(lib, fn)(*args, ctypes.byref(out)), out.value


def test_delta_workspace(lib):
    st, f = ws(lib, "ttt_delta_workspace_bytes", 4, 2, 128, 192, 1000, 3, BF16, 0)
    assert st == 0 and f > 0
    st, b = ws(lib, "ttt_delta_workspace_bytes", 4, 2, 128, 192, 1000, 3, BF16, 1)
    # the states and their gradients: 18 chunks at most
    assert st == 0 and b > f + 2 * 18 * 4 * 128 * 192 * 4
    assert ws(lib, "ttt_delta_workspace_bytes", 4, 4, 64, 64, 0, 1, F32, 1)[0] == 0


@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("H,dk,dv,nseq", [(1, 64, 64, 1), (4, 256, 256, 1), (2, 128, 192, 3), (1, 256, 64, 2), (8, 128, 128, 1)])
def test_delta_workspace_grows_with_rows(lib, H, dk, dv, nseq, backward):
    """A workspace for more rows serves fewer."""
    last = 0
    for n in list(range(nseq, 9000, 61)) + [20000, 44000, 100000, 1000000]:
        st, b = ws(lib, "ttt_delta_workspace_bytes", H, H, dk, dv, n, nseq, BF16, backward)
        assert st == 0 and b >= last, n
        last = b


def test_delta_launches_fit(lib):
    """Workgroups of 512: 2^23 of them and more are refused, one fewer is not."""
    assert ws(lib, "ttt_delta_workspace_bytes", 1, 1, 64, 1024, 10, 1 << 17, BF16, 0)[0] == -2
    assert ws(lib, "ttt_delta_workspace_bytes", 1, 1, 64, 1024, 10, (1 << 17) - 1, BF16, 0)[0] == 0


@pytest.mark.parametrize("args,code", [
    ((4, 3, 64, 64, 10, 1, BF16, 0), -1),         # heads not a multiple of key heads
    ((0, 1, 64, 64, 10, 1, BF16, 0), -1),
    ((4, 4, 96, 64, 10, 1, BF16, 0), -2),         # dk
    ((4, 4, 64, 96, 10, 1, BF16, 0), -2),         # dv
    ((4, 4, 64, 1088, 10, 1, BF16, 0), -2),
    ((4, 4, 64, 64, -1, 1, BF16, 0), -1),
    ((4, 4, 64, 64, 10, 0, BF16, 0), -1),         # no sequence
    ((4, 4, 64, 64, 10, 1, 5, 0), -2),            # dtype
    ((4, 4, 64, 64, 1 << 31, 1, BF16, 0), -2),    # rows
    ((4, 4, 64, 64, 1 << 30, 1, BF16, 0), -2),    # chunks x heads
    ((64, 64, 64, 1024, 1000, 5000, BF16, 0), -2),   # sequences x heads x slices
])
def test_delta_workspace_refusals(lib, args, code):
    assert ws(lib, "ttt_delta_workspace_bytes", *args)[0] == code
    assert len(lib.ttt_last_error()) > 0


def _delta(lib, w=1 << 20, w_out=2 << 20, q=4 << 20, k=5 << 20, v=6 << 20, beta=7 << 20, bhs=10, o=8 << 20, ld=64, n=10,
           cu=None, nseq=1, scale=1.0, flags=0, work=1 << 30, size=BIG, ld_q=None):
    return lib.ttt_delta(1, 1, 64, 64, w, w_out, q, ld_q or ld, k, ld, v, ld, beta, bhs, None, 0, o, ld, n, cu, nseq, scale, F32,
                         flags, work, size, None)


@cpu_only
def test_delta_refusals(lib):
    for kw, code, text in (
            (dict(w=None), -1, b"w is null"), (dict(w_out=None), -1, b"w_out"), (dict(q=None), -1, b"q is null"),
            (dict(q=(4 << 20) + 4), -1, b"aligned"), (dict(ld=60), -1, b"ld"), (dict(ld_q=66), -1, b"aligned"),
            (dict(beta=None), -1, b"beta"), (dict(bhs=-1), -1, b"stride"), (dict(nseq=2), -1, b"sequences"),
            (dict(scale=float("nan")), -1, b"scale"), (dict(flags=2), -1, b"flag"), (dict(work=None), -3, b"workspace"),
            (dict(size=64), -3, b"workspace"), (dict(work=(1 << 30) + 8), -1, b"aligned"),
            (dict(w_out=(1 << 20) + 64), -1, b"overlap"), (dict(o=(4 << 20) + 256), -1, b"overlap"),
            (dict(ld=1 << 24), -2, b"stride")):
        assert _delta(lib, **kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())


@cpu_only
def test_delta_backward_refusals(lib):
    def call(gq=8 << 20, gk=9 << 20, gv=10 << 20, gb=11 << 20, gd=None, gw=12 << 20, decay=None, ldg=64):
        return lib.ttt_delta_backward(1, 1, 64, 64, 1 << 20, 4 << 20, 64, 5 << 20, 64, 6 << 20, 64, 7 << 20, 10, decay, 0,
                                      3 << 20, 64, None, gq, ldg, gk, ldg, gv, ldg, gb, gd, gw, 10, None, 1, 1.0, F32,
                                      1 << 30, BIG, None)
    for kw, text in ((dict(gq=None), b"grad_q"), (dict(gb=None), b"grad_beta"), (dict(gw=None), b"grad_w"),
                     (dict(gd=13 << 20), b"grad_decay"), (dict(decay=14 << 20), b"grad_decay"),
                     (dict(gq=6 << 20), b"overlap"), (dict(gk=(8 << 20) + 64), b"overlap"), (dict(gw=1 << 20), b"overlap")):
        assert call(**kw) == -1, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())


@cpu_only
def test_delta_step_refusals(lib):
    def call(w=1 << 30, pool=4, slots=3 << 20, n=10, o=8 << 20, flags=0, beta=7 << 20):
        return lib.ttt_delta_step(1, 1, 64, 64, w, pool, slots, 4 << 20, 64, 5 << 20, 64, 6 << 20, 64, beta, 10, None, 0, o,
                                  64, n, 1.0, F32, flags, None)
    for kw, code, text in ((dict(w=None), -1, b"w is null"), (dict(slots=None), -1, b"slots"), (dict(pool=0), -1, b"pool"),
                           (dict(n=-1), -1, b"n must"), (dict(o=4 << 20), -1, b"overlap"), (dict(flags=4), -1, b"flag"),
                           (dict(w=4 << 20), -1, b"overlap"), (dict(n=1 << 24), -2, b"rows"), (dict(beta=None), -1, b"beta")):
        assert call(**kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())
    assert call(n=0) == 0


@cpu_only
def test_delta_step_of_too_many_slots(lib):
    """Rows of one state are looked for among all slots: more than 2^42 looks, seconds of work, are refused."""
    def call(n, slots, dv=64):
        # (no q: the last check before a launch would refuse it)
        return lib.ttt_delta_step(1, 1, 64, dv, 1 << 30, 1 << 30, slots, None, 64, 5 << 20, 64, 6 << 20, dv, 7 << 20, 10, None, 0,
                                  8 << 20, dv, n, 1.0, F32, 0, None)
    assert call((1 << 21) + 1, 3 << 20) == -2 and b"slots" in lib.ttt_last_error()
    assert call((1 << 20) + 1, 3 << 20, 256) == -2 and b"slots" in lib.ttt_last_error()
    for n, slots, dv in ((1 << 21, 3 << 20, 64), (1 << 20, 3 << 20, 256), ((1 << 21) + 1, None, 64)):
        assert call(n, slots, dv) == -1 and b"q is null" in lib.ttt_last_error()


@cpu_only
def test_gated_residual_refusals(lib):
    def call(C=64, norm=64, x=1 << 20, o=2 << 20, z=None, gamma=None, gn=None, eps=1e-6, y=3 << 20, h=None, ld=64, n=10):
        return lib.ttt_gated_residual(C, norm, x, ld, o, ld, z, ld, gamma, None, gn, eps, y, ld, h, ld, n, F32, None)
    for kw, code, text in ((dict(C=60), -2, b"channels"), (dict(C=8200, ld=8200), -2, b"channels"),
                           (dict(norm=48), -2, b"norm_width"), (dict(norm=4), -2, b"norm_width"),
                           (dict(eps=-1.0), -1, b"eps"), (dict(eps=float("inf")), -1, b"eps"), (dict(x=None), -1, b"x is null"),
                           (dict(y=2 << 20), -1, b"overlap"), (dict(gn=5 << 20), -1, b"gamma_next"), (dict(h=5 << 20), -1, b"gamma_next"),
                           (dict(gamma=(5 << 20) + 4), -1, b"gamma"), (dict(o=(2 << 20) + 4), -1, b"aligned"), (dict(n=-1), -1, b"n must"),
                           (dict(ld=32), -1, b"ld")):
        assert call(**kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())
    assert call(n=0) == 0
    st, b = ws(lib, "ttt_gated_residual_backward_workspace_bytes", 64, 10)
    assert st == 0 and b >= 2 * 64 * 4
    assert ws(lib, "ttt_gated_residual_backward_workspace_bytes", 60, 10)[0] == -2

    def back(gh=None, gn=None, z=None, gz=None, gx=6 << 20, go=7 << 20, size=BIG):
        return lib.ttt_gated_residual_backward(64, 64, 1 << 20, 64, gh, 64, 2 << 20, 64, 3 << 20, 64, z, 64, None, None, gn, 1e-6,
                                               gx, 64, go, 64, gz, 64, None, None, None, 10, F32, 1 << 30, size, None)
    for kw, code, text in ((dict(gh=8 << 20), -1, b"gamma_next"), (dict(z=8 << 20), -1, b"grad_z"), (dict(gz=8 << 20), -1, b"grad_z"),
                           (dict(go=6 << 20), -1, b"overlap"), (dict(gx=3 << 20), -1, b"overlap"), (dict(size=16), -3, b"workspace")):
        assert back(**kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())


@cpu_only
def test_orthogonalise_refusals(lib):
    def call(r=8, c=8, b=2, g=1 << 20, ld=8, bs=64, out=2 << 20, steps=5, dt=F32, size=BIG):
        return lib.ttt_orthogonalise(r, c, b, g, ld, bs, out, ld, bs, steps, dt, 1 << 30, size, None)
    for kw, code, text in ((dict(r=0), -1, b"rows"), (dict(c=70000, ld=70000), -2, b"65536"), (dict(b=-1), -1, b"batch"),
                           (dict(dt=9), -2, b"dtype"), (dict(steps=-1), -1, b"steps"), (dict(ld=7), -1, b"ld"),
                           (dict(bs=60), -1, b"overlap"), (dict(g=None), -1, b"null"), (dict(out=(1 << 20) + 4), -1, b"overlap"),
                           (dict(size=16), -3, b"workspace")):
        assert call(**kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())
    assert call(b=0) == 0
    st, n = ws(lib, "ttt_orthogonalise_workspace_bytes", 100, 200, 3, BF16)
    assert st == 0 and n > 3 * 100 * 200 * 4


@pytest.mark.parametrize("rows,cols,batch,rp,cp", [
    (128, 1024, 64, 128, 1024), (768, 128, 96, 128, 768), (128, 16384, 4, 128, 16384), (100, 120, 200, 128, 128),
    (300, 1024, 64, 320, 1024), (190, 1000, 50, 192, 1024),           # a larger tile would be mostly padding
    (768, 2048, 8, 768, 2048), (1300, 5100, 2, 1536, 5120), (4096, 1024, 4, 1024, 4096)])
def test_orthogonalise_is_not_mostly_padding(lib, rows, cols, batch, rp, cp):
    """The workspace holds two X and X^T and one A and B of padded sizes, two fp16 parts each."""
    up = lambda x: -(-x // 256) * 256
    st, b = ws(lib, "ttt_orthogonalise_workspace_bytes", rows, cols, batch, BF16)
    blocks = min(256, -(-rows * cols // 4096))
    assert st == 0
    assert b == up(batch * blocks * 8) + up(batch * 4) + 4 * up(rp * cp * 4 * batch) + 2 * up(rp * rp * 4 * batch)


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, 64)
    w = torch.zeros(1, 1, 64, 64)
    rate = torch.zeros(1, 4)
    for call in (lambda: ttt.delta(w, t, t, t, rate), lambda: ttt.delta_backward(w, t, t, t, rate, None, t),
                 lambda: ttt.delta_step(w, t[:1], t[:1], t[:1], rate), lambda: ttt.gated_residual(t, t),
                 lambda: ttt.gated_residual_backward(t, None, t, t), lambda: ttt.orthogonalise(t)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call()


def test_rates_are_refused_by_their_names():
    good = torch.zeros(2, 5)
    for name in ("beta", "decay"):
        for t in (good.double(), good, good[:, :3], good.t(), good[None]):
            with pytest.raises(ValueError, match=f"^{name} must be"):
                ttt._rate(t, 2, 4, 0, name)
    with pytest.raises(ValueError, match="^eta must be float32"):
        ttt._eta_stride(good.double(), 2, 4, None)
