"""Argument checks and workspace queries of the windowed-attention, layer-norm and AdamW entry points, without a GPU.
Made-up addresses are passed only where no GPU is visible, and every check rejects them before any launch."""
import ctypes
import os

import pytest
import torch

from test_weight_layers_amd import ttt

F32, BF16 = ttt.TTT_F32, ttt.TTT_BF16
BIG = 1 << 40
MB = 1 << 20
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


ATT = "ttt_window_attention_workspace_bytes"


def test_attention_workspace(lib):
    # heads, key heads, d, nq, nk, sequences, block, before, after, sinks, dtype, backward
    st, b = ws(lib, ATT, 4, 2, 64, 1000, 1000, 3, 1, 99, 0, 4, BF16, 1)
    assert st == 0 and b >= 4 * 1000 * 4                                    # delta
    st, b = ws(lib, ATT, 2, 2, 128, 3, 100000, 1, 1, -1, 0, 0, BF16, 0)
    assert st == 0 and b >= 2 * 2 * 3 * 128 * 4                             # ranges of keys
    st, b = ws(lib, ATT, 1, 1, 64, 30000, 30000, 1, 1, 63, 0, 4, BF16, 1)
    assert st == 0 and b >= 30000 * 4 + 3 * 128 * 2 * 64 * 4                # a tile of sinks, in ranges of queries
    st, b = ws(lib, ATT, 1, 1, 64, 5000, 5000, 500, 1, -1, 0, 0, F32, 0)
    assert st == 0 and b >= 501 * 24                                        # the table of sequences
    for args in ((4, 4, 64, 0, 0, 1, 1, -1, -1, 0, F32, 1), (4, 4, 64, 0, 10, 1, 1, -1, -1, 0, F32, 1)):
        assert ws(lib, ATT, *args)[0] == 0


def test_attention_workspace_of_sinks(lib):
    assert ws(lib, ATT, 2, 1, 64, 1000, 0, 1, 1, 10, 0, 4, BF16, 1)[0] == 0               # sinks, but no keys
    st, b = ws(lib, ATT, 16, 8, 128, 500000, 500000, 10000, 1, 63, 0, 4, BF16, 1)         # of many sequences
    assert st == 0 and b < 200 * MB


@pytest.mark.parametrize("args,code", [
    ((4, 3, 64, 10, 10, 1, 1, -1, 0, 0, BF16, 0), -1),          # heads not a multiple of key heads
    ((0, 1, 64, 10, 10, 1, 1, -1, 0, 0, BF16, 0), -1),
    ((4, 4, 96, 10, 10, 1, 1, -1, 0, 0, BF16, 0), -2),          # d
    ((4, 4, 64, -1, 10, 1, 1, -1, 0, 0, BF16, 0), -1),
    ((4, 4, 64, 10, 10, 0, 1, -1, 0, 0, BF16, 0), -1),          # no sequence
    ((4, 4, 64, 10, 10, 1, 0, -1, 0, 0, BF16, 0), -1),          # block
    ((4, 4, 64, 10, 10, 1, 1, -1, 0, -2, BF16, 0), -1),         # sinks
    ((4, 4, 64, 10, 10, 1, 1, -1, 0, 0, 7, 0), -2),             # dtype
    ((4, 4, 64, 1 << 31, 10, 1, 1, -1, 0, 0, BF16, 0), -2),     # rows
    ((64, 64, 64, 1 << 30, 10, 1, 1, -1, 0, 0, BF16, 0), -2),   # tiles x heads
    ((64, 64, 256, 10, 1 << 30, 1, 1, -1, 0, 0, BF16, 1), -2),
])
def test_attention_workspace_refusals(lib, args, code):
    assert ws(lib, ATT, *args)[0] == code
    assert len(lib.ttt_last_error()) > 0


@cpu_only
def test_attention_refusals(lib):
    def call(q=1 * MB, k=2 * MB, v=3 * MB, o=4 * MB, ld=64, ld_q=None, nq=10, nk=10, cu=None, cu_k=None, nseq=1, block=1,
             sinks=0, scale=0.1, flags=0, work=1 << 30, size=BIG):
        return lib.ttt_window_attention(1, 1, 64, q, ld_q or ld, k, ld, v, ld, o, ld, None, nq, nk, cu, cu_k, nseq, block, -1, 0,
                                        sinks, scale, F32, flags, work, size, None)
    for kw, code, text in (
            (dict(q=None), -1, b"q is null"), (dict(k=2 * MB + 4), -1, b"aligned"), (dict(ld=60), -1, b"ld"),
            (dict(ld_q=66), -1, b"aligned"), (dict(nseq=2), -1, b"cu_seqlens"), (dict(cu_k=5 * MB), -1, b"cu_seqlens_k"),
            (dict(cu=5 * MB, nk=12), -1, b"cu_seqlens_k"), (dict(block=-3), -1, b"block"), (dict(sinks=-1), -1, b"sinks"),
            (dict(scale=float("nan")), -1, b"scale"), (dict(scale=-1.0), -1, b"scale"), (dict(flags=2), -1, b"flag"),
            (dict(work=None), -3, b"workspace"), (dict(size=64), -3, b"workspace"), (dict(work=(1 << 30) + 8), -1, b"aligned"),
            (dict(o=1 * MB + 256), -1, b"overlap"), (dict(o=3 * MB), -1, b"overlap"), (dict(ld=1 << 24), -2, b"stride")):
        assert call(**kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())
    assert call(nq=0, q=None, o=None) == 0


@cpu_only
def test_attention_backward_refusals(lib):
    def call(lse=5 * MB, go=6 * MB, gq=7 * MB, gk=8 * MB, gv=9 * MB, o=4 * MB, ldg=64, nk=10):
        return lib.ttt_window_attention_backward(1, 1, 64, 1 * MB, 64, 2 * MB, 64, 3 * MB, 64, o, 64, lse, go, 64, gq, ldg, gk, ldg,
                                                 gv, ldg, 10, nk, None, None, 1, 1, -1, 0, 0, 0.1, F32, 1 << 30, BIG, None)
    for kw, text in ((dict(lse=None), b"lse"), (dict(go=None), b"grad_o"), (dict(gq=None), b"grad_q"), (dict(gv=None), b"grad_v"),
                     (dict(o=None), b"o is null"), (dict(gq=1 * MB), b"overlap"), (dict(gk=7 * MB + 256), b"overlap"),
                     (dict(gv=2 * MB), b"overlap"), (dict(gk=6 * MB), b"overlap"), (dict(ldg=60), b"ld")):
        assert call(**kw) == -1, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())


@cpu_only
def test_attention_step_refusals(lib):
    def call(kc=100 * MB, vc=101 * MB, ldc=64, stride=20 * 64, pool=4, cap=20, slots=5 * MB, pos=6 * MB, o=4 * MB, n=10, block=1,
             sinks=0, scale=0.1, flags=0, size=BIG, work=1 << 30, q=1 * MB):
        return lib.ttt_window_attention_step(1, 1, 64, kc, vc, ldc, stride, pool, cap, slots, pos, q, 64, 2 * MB, 64, 3 * MB, 64,
                                             o, 64, n, block, -1, sinks, scale, F32, flags, work, size, None)
    for kw, code, text in (
            (dict(kc=None), -1, b"k_cache is null"), (dict(vc=100 * MB), -1, b"overlap"), (dict(vc=100 * MB + 256 * 20), -1, b"overlap"),
            (dict(ldc=60), -1, b"ld of k_cache"), (dict(stride=19 * 64), -1, b"pool_stride"), (dict(pool=0), -1, b"pool"),
            (dict(cap=0), -1, b"capacity"), (dict(sinks=20), -1, b"capacity"), (dict(slots=None), -1, b"slots"),
            (dict(pos=None), -1, b"positions"), (dict(o=1 * MB), -1, b"overlap"), (dict(o=100 * MB), -1, b"overlap"),
            (dict(q=101 * MB), -1, b"overlap"), (dict(block=0), -1, b"block"), (dict(scale=float("inf")), -1, b"scale"),
            (dict(flags=8), -1, b"flag"), (dict(n=-1), -1, b"n must"), (dict(n=(1 << 21) + 1), -2, b"slots"),
            (dict(size=16), -3, b"workspace")):
        assert call(**kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())
    assert call(n=0) == 0
    # the halves of rows, or of entries, of one buffer may be given: refused only for what comes after
    for kw in (dict(vc=100 * MB + 256, ldc=128, stride=20 * 128), dict(vc=100 * MB + 256 * 20, stride=40 * 64)):
        assert call(**kw, work=None) == -3, kw


@cpu_only
def test_layer_norm_refusals(lib):
    def call(C=64, w=64, x=1 * MB, ld=64, gamma=None, beta=None, eps=1e-6, y=2 * MB, n=10, dtype=F32):
        return lib.ttt_layer_norm(C, w, x, ld, gamma, beta, eps, y, ld, n, dtype, None)
    for kw, code, text in ((dict(w=0), -2, b"norm_width"), (dict(C=8200, w=8200, ld=8200), -2, b"norm_width"), (dict(w=48), -1, b"norm_width"),
                           (dict(w=4), -2, b"norm_width"), (dict(C=32, w=64), -1, b"norm_width"), (dict(n=-1), -1, b"n must"),
                           (dict(eps=float("nan")), -1, b"eps"), (dict(gamma=5 * MB + 4), -1, b"gamma"), (dict(beta=5 * MB + 8), -1, b"beta"),
                           (dict(x=None), -1, b"x is null"), (dict(y=1 * MB + 64), -1, b"overlap"), (dict(ld=32), -1, b"ld"),
                           (dict(ld=65), -1, b"aligned"), (dict(dtype=4), -2, b"dtype")):
        assert call(**kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())
    assert call(n=0) == 0
    st, b = ws(lib, "ttt_layer_norm_backward_workspace_bytes", 64, 64, 10)
    assert st == 0 and b >= 2 * 64 * 4
    assert ws(lib, "ttt_layer_norm_backward_workspace_bytes", 64, 48, 10)[0] == -1

    def back(gx=3 * MB, size=BIG, gy=2 * MB):
        return lib.ttt_layer_norm_backward(64, 64, gy, 64, 1 * MB, 64, None, 1e-6, gx, 64, None, None, 10, F32, 1 << 30, size, None)
    for kw, code, text in ((dict(gx=1 * MB), -1, b"overlap"), (dict(gx=2 * MB + 256), -1, b"overlap"), (dict(gy=None), -1, b"grad_y"),
                           (dict(size=16), -3, b"workspace")):
        assert back(**kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())


def table(*tensors):
    t = (ttt._AdamwTensor * len(tensors))()
    for x, kw in zip(t, tensors):
        for k, v in {**dict(param=1 * MB, grad=2 * MB, exp_avg=3 * MB, exp_avg_sq=4 * MB, n=100), **kw}.items():
            setattr(x, k, v)
    return t


@cpu_only
def test_adamw_refusals(lib):
    def call(t, count=None, step=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, bits=32, dtype=F32, dev_step=None, work=None, gs=None):
        return lib.ttt_adamw_step(t, len(t) if count is None else count, step, dev_step, lr, None, b1, b2, eps, wd, gs, bits, dtype,
                                  work, BIG, None)
    one = table({})
    for t, kw, code, text in (
            (one, dict(bits=16), -2, b"bits"), (one, dict(dtype=5), -2, b"dtype"), (one, dict(count=-1), -1, b"count"),
            (one, dict(step=0), -1, b"step"), (one, dict(lr=-1.0), -1, b"lr"), (one, dict(lr=float("nan")), -1, b"lr"),
            (one, dict(b1=1.0), -1, b"beta"), (one, dict(b2=-0.1), -1, b"beta"), (one, dict(eps=-1.0), -1, b"eps"),
            (one, dict(wd=float("inf")), -1, b"weight_decay"), (one, dict(bits=8), -1, b"scales"),
            (one, dict(dev_step=8 * MB), -3, b"workspace"), (one, dict(dev_step=8 * MB + 4, work=1 << 30), -1, b"aligned"),
            (one, dict(gs=8 * MB + 2), -1, b"aligned"), (table(dict(param=None)), {}, -1, b"null"), (table({}, dict(grad=None)), {}, -1, b"tensor 1"),
            (table(dict(n=-1)), {}, -1, b"n must"), (table(dict(exp_avg=3 * MB + 2)), {}, -1, b"aligned"),
            (table({}, dict(master=5 * MB)), {}, -1, b"master"), (table(dict(exp_avg_scale=5 * MB, exp_avg_sq_scale=6 * MB)), {}, -1, b"scales")):
        assert call(t, **kw) == code, kw
        assert text in lib.ttt_last_error(), (kw, lib.ttt_last_error())
    assert call(one, count=0) == 0 and call(table(dict(n=0))) == 0


def test_adamw_check(lib):
    ok = lambda *t, bits=32: lib.ttt_adamw_check(table(*t), len(t), bits, F32)
    assert ok({}) == 0
    assert ok({}, dict(param=5 * MB, exp_avg=6 * MB, exp_avg_sq=7 * MB)) == 0                   # gradients may be shared
    assert ok({}, {}) == -1 and b"overlap" in lib.ttt_last_error()
    assert ok(dict(exp_avg=4 * MB)) == -1 and ok(dict(exp_avg=4 * MB - 396)) == -1 and ok(dict(exp_avg=4 * MB - 400)) == 0
    assert ok(dict(grad=1 * MB + 396)) == -1 and ok(dict(grad=1 * MB - 396)) == -1 and ok(dict(grad=1 * MB + 400)) == 0
    scales = dict(exp_avg_scale=5 * MB, exp_avg_sq_scale=5 * MB + 4)
    assert ok(scales, bits=8) == 0 and ok(dict(scales, n=257), bits=8) == -1
    assert ok(dict(n=0, param=None, exp_avg=None, exp_avg_sq=None)) == 0


def test_binding_refuses_host_tensors():
    t = torch.zeros(4, 64)
    lse, pos = torch.zeros(1, 4), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: ttt.window_attention(t, t, t, heads=1), lambda: ttt.window_attention_backward(t, t, t, t, lse, t, heads=1),
                 lambda: ttt.window_attention_step(t[None], t[None], t, t, t, pos, heads=1), lambda: ttt.layer_norm(t),
                 lambda: ttt.layer_norm_backward(t, t), lambda: ttt.adamw_tensors([t], [t], [t])):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call()


def test_limits_beyond_32_bits():
    """Limits that take in everything mean that, whatever their size; they do not wrap."""
    def ask(before, after=0, sinks=0, block=1, backward=False):
        return ttt.window_attention_workspace_bytes(8, 2, 128, 1374, 43968, 1, block, before, after, sinks, torch.bfloat16, backward)
    most = (1 << 31) - 1
    assert ask(0) != ask(None) and ask(0, sinks=0) != ask(0, sinks=most)
    for big in (1 << 31, 1 << 32, (1 << 32) + 5, 1 << 40, 1 << 62, 1 << 70):
        assert ttt._limit(big, "before") == -1 and ttt._sinks(big) == most
        for backward in (False, True):
            assert ask(big, backward=backward) == ask(None, backward=backward)
            assert ask(3, after=big, backward=backward) == ask(3, after=None, backward=backward)
            assert ask(3, sinks=big, backward=backward) == ask(3, sinks=most, backward=backward)
        for bad in (dict(block=big), dict(block=-big), dict(block=1 - big), dict(before=-big), dict(after=1 - big), dict(sinks=-big)):
            with pytest.raises((ValueError, ttt.TTTError)):
                ask(**{"before": 3, **bad})
    for name, fn in (("block", ttt._int32), ("before", ttt._limit)):
        with pytest.raises(ValueError, match=name):
            fn(-(1 << 32), name)


@cpu_only
@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_empty_tensors_beside_masters(lib, bits):
    """An empty tensor has no master, nor any other array: its pointers are null, wherever it stands in the table."""
    none = dict(param=None, grad=None, exp_avg=None, exp_avg_sq=None, n=0)
    scales = dict(exp_avg_scale=8 * MB, exp_avg_sq_scale=9 * MB) if bits == 8 else {}
    first = dict(scales, master=5 * MB)
    other = dict(param=11 * MB, exp_avg=13 * MB, exp_avg_sq=14 * MB, master=15 * MB,
                 **{k: v + 10 * MB for k, v in scales.items()})
    for t in ((first, none), (none, first), (none, first, none, other, none), (none,), (none, dict(none, master=7 * MB))):
        assert lib.ttt_adamw_check(table(*t), len(t), bits, BF16) == 0, (t, lib.ttt_last_error())
    bare = {k: v for k, v in other.items() if k != "master"}
    for t, at in (((none, first, bare), b"tensor 2"), ((none, bare, first), b"tensor 2"), ((first, none, bare), b"tensor 2")):
        assert lib.ttt_adamw_check(table(*t), len(t), bits, BF16) == -1
        assert at in lib.ttt_last_error() and b"master" in lib.ttt_last_error()


@cpu_only
def test_attention_step_cache_layouts(lib):
    """k and v in one buffer, for pools of one cache and of more: apart by columns or by entries, or refused."""
    def call(x, pool, ldc=128, stride=0, cap=20):
        return lib.ttt_window_attention_step(1, 1, 64, 100 * MB, 100 * MB + x, ldc, stride, pool, cap, 5 * MB, 6 * MB, 1 * MB, 64,
                                             2 * MB, 64, 3 * MB, 64, 4 * MB, 64, 10, 1, -1, 0, 0.1, F32, 0, None, 0, None)
    # rows of 64 fp32 values: 256 bytes, 512 from row to row
    for pool in (1, 2, 4):
        tight, wide = 20 * 128, 20 * 128 + 64           # entries back to back, and 256 bytes apart
        for stride in (tight, wide):
            for x in (256, -256):                       # column halves of the same rows
                assert call(x, pool, stride=stride) == -3, (pool, stride, x, lib.ttt_last_error())
            for x in (0, 128, -128, 384, -64):          # columns that both have
                assert call(x, pool, stride=stride) == -1 and b"overlap" in lib.ttt_last_error(), (pool, stride, x)
        # halves of the rows of different entries, or of rows further down
        assert call(tight * 4 + 256, pool, stride=tight) == -3
        assert call(5 * 512 + 256, pool, stride=tight) == -3
        # rows moved down in entries that are not whole rows apart: the next entry's columns are others (but for a pool of one)
        assert call(5 * 512 + 256, pool, stride=wide) == (-3 if pool == 1 else -1)
        # one cache after the other in each entry
        assert call(20 * 512, pool, stride=40 * 128) == -3
        assert call(20 * 512 - 256, pool, stride=40 * 128) == -3          # (its last row ends at 19 * 512 + 256)
        assert call(20 * 512 - 384, pool, stride=40 * 128) == -1
    for cap in (1, 2):
        assert call(256, 1, cap=cap) == -3 and call(128, 1, cap=cap) == -1


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("nq,nk,seqs,heads,key_heads,d,before,after", [
    (64, 8192, 1, 8, 2, 128, -1, 0), (1374, 43968, 1, 8, 8, 128, -1, 0), (256, 131072, 1, 32, 8, 128, -1, 0),
    (64, 8192, 1, 8, 8, 64, -1, -1), (1, 5000, 1, 8, 2, 128, -1, 0), (986, 603660, 2, 64, 16, 256, -1, 0),
    (65536, 512, 1, 8, 8, 64, -1, -1), (8192, 64, 1, 8, 2, 128, -1, -1), (5000, 1, 1, 8, 2, 128, -1, -1), (40000, 500, 2, 8, 2, 64, -1, -1)])
def test_attention_gradient_ranges_of_unequal_rows(lib, nq, nk, seqs, heads, key_heads, d, before, after, dtype):
    """A few queries are not cut in ranges because there are many keys, nor a few keys because there are many queries: a range
    holds fp32 gradients of all keys (of all queries), and two take twice that."""
    st, b = ws(lib, ATT, heads, key_heads, d, nq, nk, seqs, 1, before, after, 0, dtype, 1)
    keys, queries = nk * key_heads * 2 * d * 4, nq * heads * d * 4
    assert st == 0 and b < 2 * max(keys, queries), (b, keys, queries)


def test_attention_gradient_ranges_of_equal_rows(lib):
    """Where both walks are long both are cut, as they were."""
    for dtype, most in ((BF16, 28), (F32, 47)):
        st, b = ws(lib, ATT, 2, 1, 128, 2048, 2048, 1, 1, -1, 0, 0, dtype, 1)
        assert st == 0 and 2 * 2048 * 2 * 128 * 4 < b < most * 10 ** 6


@pytest.mark.parametrize("nq,nk,seqs,heads,key_heads,d", [(100, 198494, 70, 64, 4, 128), (91, 7644, 70, 64, 1, 128), (207, 137547, 500, 64, 1, 128),
                                                          (89, 85264, 70, 64, 2, 256), (57, 18522, 70, 64, 1, 128)])
def test_attention_ranges_of_few_queries(lib, nq, nk, seqs, heads, key_heads, d):
    """A few queries in many sequences are a tile each, and so many tiles need no ranges of keys: what they would take is many
    times the tensors."""
    for dtype, size in ((F32, 4), (BF16, 2)):
        st, b = ws(lib, ATT, heads, key_heads, d, nq, nk, seqs, 1, -1, 0, 0, dtype, 0)
        assert st == 0 and b < 2 * (nq * heads + nk * key_heads) * d * size
