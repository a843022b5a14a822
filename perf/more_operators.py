"""Timed cases of windowed attention (prompts, gradients, single tokens over a rolling cache), layer norm with its
gradient and AdamW over many tensors, each in elementary torch operations beside the library's calls.

``own`` selects which of the two ``run`` computes.  ``exact`` states every operator once more in 64 bits, from its
definition (whole masks, differentiation, token by token).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SCORES = 1 << 28                            # scores that the plain attention holds at once
BLOCK8 = 256                                # elements that share a scale of 8-bit optimiser states


# ------------------------------------------------------------------ cases
def listed():
    return [
        # attention inside one 518 x 518 frame (37 x 37 patches + 5 tokens), 16 heads of 64
        dict(name="attention frame", op="attention", nq=1374, nk=1374, seqs=1, cut=0, heads=16, key_heads=16, d=64,
             block=1374, before=0, after=0, sinks=0, dtype="bf16"),
        # eight frames of a stream against the 32 so far: each frame sees itself, five before it and the first one
        dict(name="attention stream chunk", op="attention", nq=10992, nk=43968, seqs=1, cut=0, heads=8, key_heads=8, d=128,
             block=1374, before=5, after=0, sinks=1374, dtype="bf16"),
        # training on eight object views of 1024 tokens, width 768, keys shared by three heads, a window of tokens
        dict(name="attention train views", op="attention_backward", nq=8192, nk=8192, seqs=8, cut=0, heads=12, key_heads=4,
             d=64, block=1, before=511, after=0, sinks=4, dtype="bf16"),
        # fp32 training on packed sequences of uneven lengths, one of them empty and one a single token
        dict(name="attention train ragged", op="attention_backward", nq=2731, nk=2731, seqs=6, cut=2, heads=4, key_heads=4,
             d=128, block=37, before=9, after=1, sinks=5, dtype="f32"),
        # one token of one sequence: what a stream pays per query
        dict(name="attention step one", op="attention_step", n=1, pool=2, capacity=4100, heads=16, key_heads=16, d=64,
             block=1, before=4095, sinks=4, dtype="bf16"),
        # one token for each of 64 sequences of uneven age out of a pool of 80 caches
        dict(name="attention step pool", op="attention_step", n=64, pool=80, capacity=4096, heads=16, key_heads=4, d=128,
             block=1, before=-1, sinks=64, dtype="bf16"),
        # the norm of one frame before attention
        dict(name="norm frame", op="norm", n=1374, width=1024, norm=1024, dtype="bf16"),
        # the norm of every head's queries over 100 frames
        dict(name="norm 100 frames", op="norm", n=137400, width=1024, norm=64, dtype="bf16"),
        # gradients over one 32-frame chunk
        dict(name="norm train chunk", op="norm_backward", n=43968, width=1024, norm=1024, dtype="bf16"),
        # gradients in fp32
        dict(name="norm train f32", op="norm_backward", n=8192, width=768, norm=768, dtype="f32"),
        # one block of width 768, fp32 with 32-bit states
        dict(name="adamw block", op="adamw", layers=1, cut=0, width=768, bits=32, dtype="f32"),
        # twelve blocks of width 1024, bf16 with fp32 masters, 8-bit states
        dict(name="adamw 12 blocks", op="adamw", layers=12, cut=0, width=1024, bits=8, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attention", "attention_backward", "attention_step", "norm", "norm_backward", "adamw"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op.startswith("attention"):
        heads = rng.choice((1, 2, 3, 4, 6, 8, 12))
        key_heads = rng.choice([k for k in range(1, heads + 1) if heads % k == 0])
        d = rng.choice((64, 64, 128, 256))
        block = rng.choice((1, 1, 1, 16, _log(rng, 2, 1500)))
        c = dict(op=op, heads=heads, key_heads=key_heads, d=d, block=block, sinks=rng.choice((0, 0, 4, _log(rng, 1, 300))),
                 dtype=dtype)
        if op == "attention_step":
            capacity = c["sinks"] + _log(rng, 1, 6000)
            n = min(_log(rng, 1, 200), max(1, (1 << 17) // capacity))
            return dict(c, n=n, pool=n + rng.randrange(0, 20), capacity=capacity,
                        before=rng.choice((-1, rng.randrange(0, 1 + capacity // block))))
        # where every query sees one key alone its gradient is zero: a window of two tokens at least
        n = _log(rng, 1, 6000) if op == "attention" else _log(rng, 64, 3000)
        least = 1 if op == "attention_backward" else 0
        more = 0 if op != "attention" else rng.choice((0, 0, _log(rng, 1, 6000)))
        return dict(c, nq=n, nk=n + more, seqs=rng.choice((1, 1, 2, 3, 5, 9)) if more == 0 else 1, cut=rng.randrange(1, 1 << 20),
                    before=rng.choice((-1, rng.randrange(least, 2 + n // block))), after=rng.choice((0, 0, -1, rng.randrange(0, 3))))
    if op.startswith("norm"):
        norm, groups = (8 * rng.randrange(1, 65), rng.choice((1, 2, 3, 8))) if rng.random() < 0.5 else (_log(rng, 1, 8192), 1)
        return dict(op=op, n=max(1, min(_log(rng, 1, 40000), (1 << 26) // (norm * groups))), width=norm * groups, norm=norm,
                    dtype=dtype)
    return dict(op=op, layers=0, cut=rng.randrange(1, 1 << 20), width=_log(rng, 1, 60), bits=rng.choice((8, 32)), dtype=dtype)


def _lengths(case):
    """Token counts of the packed sequences.  cut = 0: even; else uneven, and from four sequences on one is
    empty and one a single token."""
    n, s = case["nq"], case["seqs"]
    if s == 1 or case["cut"] == 0:
        return [(n + i) // s for i in range(s)]
    g = torch.Generator().manual_seed(case["cut"])
    fixed = [0, 1] if s >= 4 and n > 1 else []
    left = n - sum(fixed)
    cuts = sorted(torch.randint(0, left + 1, (s - len(fixed) - 1,), generator=g).tolist())
    lens = [b - a for a, b in zip([0] + cuts, cuts + [left])]
    return lens[:1] + fixed + lens[1:]


def _sizes(case):
    """Shapes of the optimised tensors: whole blocks of a width, or `width` tensors of any sizes."""
    if case["layers"]:
        C = case["width"]
        one = [(C,), (C,), (3 * C, C), (3 * C,), (C, C), (C,), (C,), (C,), (4 * C, C), (4 * C,), (C, 4 * C), (C,)]
        return [math.prod(s) for s in one] * case["layers"]
    g = torch.Generator().manual_seed(case["cut"])
    return [max(1, int(math.exp(x * math.log(1 << 21)))) for x in torch.rand(case["width"], generator=g).tolist()]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)
    op, st, dt = case["op"], dict(case), DT[case["dtype"]]
    if op == "attention_step":
        n, H, Hk, d = case["n"], case["heads"], case["key_heads"], case["d"]
        st["q"], st["k"], st["v"] = rn(n, H * d).to(dt), rn(n, Hk * d).to(dt), rn(n, Hk * d).to(dt)
        st["k_cache"] = torch.randn(case["pool"], case["capacity"], Hk * d, generator=g, device=dev, dtype=dt)
        st["v_cache"] = torch.randn(case["pool"], case["capacity"], Hk * d, generator=g, device=dev, dtype=dt)
        st["slots"] = torch.randperm(case["pool"], generator=g, device=dev)[:n].to(torch.int32)
        # sequences of any age: some have just begun, some went round their cache many times
        age = torch.exp(torch.rand(n, generator=g, device=dev) * math.log(20.0 * case["capacity"]))
        st["positions"] = (age if n > 1 else age.clamp(min=case["capacity"])).to(torch.int32)
    elif op.startswith("attention"):
        H, Hk, d = case["heads"], case["key_heads"], case["d"]
        st["q"], st["k"], st["v"] = (rn(m, h * d).to(dt) for m, h in ((case["nq"], H), (case["nk"], Hk), (case["nk"], Hk)))
        st["lens"] = _lengths(case)
        more = case["nk"] - case["nq"]              # of one sequence
        st["lens_k"] = [x + more for x in st["lens"]]
        st["cu"] = torch.tensor([0] + st["lens"], device=dev).cumsum(0).to(torch.int32)
        st["cu_k"] = torch.tensor([0] + st["lens_k"], device=dev).cumsum(0).to(torch.int32)
        if op == "attention_backward":
            # the forward's outputs, which training keeps
            st["o"], st["lse"] = _attention(st)
            st["do"] = rn(case["nq"], H * d).to(dt)
    elif op.startswith("norm"):
        n, C, w = case["n"], case["width"], case["norm"]
        st["x"] = (0.5 + 2.0 * rn(n, C)).to(dt)
        if C * st["x"].element_size() % 16:         # rows begin on 16 bytes
            st["x"] = torch.nn.functional.pad(st["x"], (0, -C % 8))[:, :C]
        st["gamma"], st["beta"] = 1.0 + 0.1 * rn(w), 0.1 * rn(w)
        if op == "norm_backward":
            st["dy"] = torch.empty_strided(st["x"].shape, st["x"].stride(), dtype=dt, device=dev).copy_(rn(n, C))
    else:
        sizes = _sizes(case)
        at, total = [], 0
        for s in sizes:                             # one buffer, each tensor from a multiple of a state's block on
            at.append(total)
            total += -(-s // BLOCK8) * BLOCK8
        live = torch.zeros(total, dtype=torch.bool, device=dev)
        for a, s in zip(at, sizes):
            live[a:a + s] = True
        flat = lambda t: t.masked_fill_(~live, 0.0)
        p = flat(0.02 * rn(total))
        st["p"], st["master"] = p.to(dt), p if dt == torch.bfloat16 else None
        st["g"] = flat(1e-3 * rn(total) * torch.exp(rn(total))).to(dt)
        m, v = flat(1e-3 * rn(total)), flat(1e-6 * torch.exp(rn(total)))
        if case["bits"] == 8:
            st["m"], st["ms"] = _quantise(m, 127)
            st["v"], st["vs"] = _quantise(v.sqrt_(), 255)
        else:
            st["m"], st["v"] = m, v
        views = lambda t: [t[a:a + s] for a, s in zip(at, sizes)]
        scales = lambda t: [t[a // BLOCK8:(a + s + BLOCK8 - 1) // BLOCK8] for a, s in zip(at, sizes)]
        st["lists"] = {k: scales(st[k]) if k in ("ms", "vs") else views(st[k])
                       for k in ("p", "master", "g", "m", "v", "ms", "vs") if st.get(k) is not None}
        st["step"], st["lr"], st["betas"], st["eps"], st["decay"] = 1000, 3e-4, (0.9, 0.999), 1e-8, 0.05
    return st


# ------------------------------------------------------------------ the plain forms
def _pad(rows, lens, cu):
    """Packed rows -> [seqs, longest, width] in fp32."""
    if len(lens) == 1:
        return rows.float()[None]
    t = torch.arange(max(lens), device=rows.device)
    idx = (cu[:-1, None].long() + t).clamp_(max=max(0, rows.shape[0] - 1))
    return rows.float()[idx] * (t < (cu[1:] - cu[:-1])[:, None])[..., None]


def _packed(x, lens, cu):
    """The reverse of _pad."""
    if len(lens) == 1:
        return x[0]
    t = torch.arange(max(lens), device=x.device)
    return x[t < (cu[1:] - cu[:-1])[:, None]]


def _steps(st):
    """The queries in chunks: (first, last, first key, last key, leading keys beside them, mask [seqs, 1, queries, keys])."""
    lens, lens_k, block, before, after, sinks = (st[x] for x in ("lens", "lens_k", "block", "before", "after", "sinks"))
    T, K = max(lens), max(lens_k)
    off = [b - a for a, b in zip(lens, lens_k)]
    wide = K if before < 0 or after < 0 else min(K, (before + after + 2) * block + sinks)
    rows = max(16, min(T, SCORES // (len(lens) * st["heads"] * max(1, wide))))
    t_off = torch.tensor(off, device=st["q"].device)[:, None]
    t_len = torch.tensor(lens_k, device=st["q"].device)[:, None, None]
    for a in range(0, T, rows):
        b = min(T, a + rows)
        first = 0 if before < 0 else max(0, ((a + min(off)) // block - before) * block)
        last = K if after < 0 else min(K, ((b - 1 + max(off)) // block + after + 1) * block)
        first = min(first, max(last, 0))
        last = max(first, last)
        lead = min(sinks, first)
        j = torch.cat([torch.arange(lead, device=t_off.device), torch.arange(first, last, device=t_off.device)])
        bl = torch.div(t_off + torch.arange(a, b, device=t_off.device), block, rounding_mode="floor")[..., None]
        ok = j < t_len
        if after >= 0:
            ok = ok & (j < (bl + after + 1) * block)
        if before >= 0:
            ok = ok & ((j >= (bl - before) * block) | (j < sinks))
        yield a, b, first, last, lead, ok.expand(len(lens), b - a, j.numel())[:, None]


def _heads(st):
    """q [seqs, key heads, group, longest, d] and k, v [seqs, key heads, longest, d]."""
    Hk, d, G = st["key_heads"], st["d"], st["heads"] // st["key_heads"]
    q = _pad(st["q"], st["lens"], st["cu"]).unflatten(-1, (Hk, G, d)).permute(0, 2, 3, 1, 4).contiguous()
    k, v = (_pad(st[x], st["lens_k"], st["cu_k"]).unflatten(-1, (Hk, d)).transpose(1, 2).contiguous() for x in "kv")
    return q, k, v, d ** -0.5


def _part(x, first, last, lead):
    return x[:, :, first:last] if lead == 0 else torch.cat([x[:, :, :lead], x[:, :, first:last]], 2)


def _rows(x, lens, cu):
    """[seqs, heads.., longest, d] -> packed rows."""
    x = x.flatten(1, -3).transpose(1, 2)
    return _packed(x.flatten(2), lens, cu)


def _attention(st):
    q, k, v, scale = _heads(st)
    out, lse = torch.zeros_like(q), q.new_full(q.shape[:-1], -math.inf)
    for a, b, first, last, lead, ok in _steps(st):
        if not ok.shape[-1]:
            continue
        kc, vc, qc = _part(k, first, last, lead), _part(v, first, last, lead), q[:, :, :, a:b]
        s = (qc.flatten(2, 3) @ kc.transpose(-1, -2)).view(*qc.shape[:-1], -1) * scale
        s.masked_fill_(~ok[:, :, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        m.masked_fill_(m == -math.inf, 0.0)
        e = s.sub_(m).exp_()
        l = e.sum(-1, keepdim=True)
        lse[:, :, :, a:b] = (m + l.log())[..., 0]
        e /= l.masked_fill(l == 0, 1.0)
        out[:, :, :, a:b] = (e.flatten(2, 3) @ vc).view(qc.shape)
    return (_rows(out, st["lens"], st["cu"]).to(st["q"].dtype),
            _packed(lse.flatten(1, 2).transpose(1, 2), st["lens"], st["cu"]).t().contiguous())


def _attention_backward(st):
    q, k, v, scale = _heads(st)
    Hk, d = st["key_heads"], st["d"]
    grouped = lambda x: _pad(x, st["lens"], st["cu"]).unflatten(-1, (Hk, q.shape[2], -1)).permute(0, 2, 3, 1, 4)
    do, o, lse = grouped(st["do"]).contiguous(), grouped(st["o"]), grouped(st["lse"].t())
    delta = (do * o).sum(-1, keepdim=True)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for a, b, first, last, lead, ok in _steps(st):
        if not ok.shape[-1]:
            continue
        kc, vc, qc, dc = _part(k, first, last, lead), _part(v, first, last, lead), q[:, :, :, a:b], do[:, :, :, a:b]
        qf, df = qc.flatten(2, 3), dc.flatten(2, 3)
        s = (qf @ kc.transpose(-1, -2)).view(*qc.shape[:-1], -1) * scale
        p = s.sub_(lse[:, :, :, a:b]).exp_().masked_fill_(~ok[:, :, None], 0.0)
        ds = (df @ vc.transpose(-1, -2)).view(p.shape).sub_(delta[:, :, :, a:b]).mul_(p)
        p, ds = p.flatten(2, 3), ds.flatten(2, 3) * scale
        dq[:, :, :, a:b] = (ds @ kc).view(qc.shape)
        for whole, part in ((dk, ds.transpose(-1, -2) @ qf), (dv, p.transpose(-1, -2) @ df)):
            whole[:, :, :lead] += part[:, :, :lead]
            whole[:, :, first:last] += part[:, :, lead:]
    dt = st["q"].dtype
    return (_rows(dq, st["lens"], st["cu"]).to(dt), _rows(dk, st["lens_k"], st["cu_k"]).to(dt),
            _rows(dv, st["lens_k"], st["cu_k"]).to(dt))


def _attention_step(st):
    n, Hk, d, G, C, sinks, block = (st["n"], st["key_heads"], st["d"], st["heads"] // st["key_heads"], st["capacity"],
                                    st["sinks"], st["block"])
    slots, p = st["slots"].long(), st["positions"].long()
    ring = C - sinks
    place = torch.where(p < sinks, p, sinks + (p - sinks).clamp(min=0) % ring)
    st["k_cache"][slots, place], st["v_cache"][slots, place] = st["k"], st["v"]
    # the position that each place of the cache holds
    c = torch.arange(C, device=p.device)
    held = torch.where(c < sinks, c, p[:, None] - (p[:, None] - c) % ring)
    ok = (held >= 0) & (held <= p[:, None]) & ((c < sinks) | (held >= sinks))
    if st["before"] >= 0:
        ok &= (held >= ((p // block - st["before"]) * block)[:, None]) | (c < sinks)
    q = st["q"].float().view(n, Hk, G, d)
    k, v = (st[x][slots].float().view(n, C, Hk, d).permute(0, 2, 1, 3) for x in ("k_cache", "v_cache"))
    s = (q @ k.transpose(-1, -2)) * d ** -0.5
    s.masked_fill_(~ok[:, None, None], -math.inf)
    e = (s - s.amax(-1, keepdim=True)).exp_()
    o = (e @ v) / e.sum(-1, keepdim=True)
    return o.reshape(n, -1).to(st["q"].dtype), st["k_cache"], st["v_cache"]


def _norm(st):
    x = st["x"].float().unflatten(1, (-1, st["norm"]))
    x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * st["gamma"] + st["beta"]
    return y.flatten(1).to(st["x"].dtype)


def _norm_backward(st):
    x, dy = (st[k].float().unflatten(1, (-1, st["norm"])) for k in ("x", "dy"))
    x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    xn, t = x * r, dy * st["gamma"]
    dx = r * (t - t.mean(-1, keepdim=True) - xn * (t * xn).mean(-1, keepdim=True))
    return dx.flatten(1).to(st["x"].dtype), (dy * xn).sum((0, 1)), dy.sum((0, 1))


def _quantise(x, top):
    """Codes c of blocks: x = s c |c| / top^2 with s the block's largest |x|."""
    b = x.view(-1, BLOCK8)
    s = b.abs().amax(-1, keepdim=True)
    r = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    c = torch.round((b.abs() * r).sqrt() * float(top)) * torch.sign(b)
    return c.to(torch.int8 if top == 127 else torch.uint8).view(-1), s.view(-1).contiguous()


def _values(c, s, top):
    c = c.view(-1, BLOCK8).int()
    return ((c * c.abs()).float() * (1.0 / (top * top)) * s[:, None]).view(-1)


def _adamw(st):
    b1, b2 = st["betas"]
    w = st["master"] if st["master"] is not None else st["p"]
    g = st["g"].float()
    if st["bits"] == 8:
        m, v = _values(st["m"], st["ms"], 127), _values(st["v"], st["vs"], 255)
        v = v * v
    else:
        m, v = st["m"], st["v"]
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    r = v.sqrt()
    c1, c2 = st["lr"] / (1 - b1 ** st["step"]), 1 / math.sqrt(1 - b2 ** st["step"])
    w.copy_(w * (1 - st["lr"] * st["decay"]) - (m * c1) / (r * c2 + st["eps"]))
    if st["master"] is not None:
        st["p"].copy_(w)
    if st["bits"] == 8:
        (m, ms), (r, vs) = _quantise(m, 127), _quantise(r, 255)
        for x, y in (("m", m), ("ms", ms), ("v", r), ("vs", vs)):
            st[x].copy_(y)
    else:
        st["m"].copy_(m), st["v"].copy_(v)


def _adamw_outputs(st):
    if st["bits"] == 8:
        root = _values(st["v"], st["vs"], 255)
        return st["p"], st["master"], _values(st["m"], st["ms"], 127), root * root
    return st["p"], st["master"], st["m"], st["v"]


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    none = lambda x: None if x < 0 else x
    if own:
        from test_weight_layers_amd import ttt

        if op == "attention_step":
            o = ttt.window_attention_step(st["k_cache"], st["v_cache"], st["q"], st["k"], st["v"], st["positions"],
                                          heads=st["heads"], key_heads=st["key_heads"], slots=st["slots"],
                                          block=st["block"], before=none(st["before"]), sinks=st["sinks"])
            return o, st["k_cache"], st["v_cache"]
        if op.startswith("attention"):
            how = dict(heads=st["heads"], key_heads=st["key_heads"], block=st["block"], before=none(st["before"]),
                       after=none(st["after"]), sinks=st["sinks"], cu_seqlens=st["cu"], cu_seqlens_k=st["cu_k"])
            if op == "attention":
                return ttt.window_attention(st["q"], st["k"], st["v"], **how)
            return ttt.window_attention_backward(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], **how)
        if op == "norm":
            return ttt.layer_norm(st["x"], st["gamma"], st["beta"], 1e-6, norm_width=st["norm"])
        if op == "norm_backward":
            return ttt.layer_norm_backward(st["dy"], st["x"], st["gamma"], 1e-6, norm_width=st["norm"])
        if "handle" not in st:                      # made once, as a training program does
            l = st["lists"]
            st["handle"] = ttt.adamw_tensors(l["p"], l["m"], l["v"], master=l.get("master"), exp_avg_scales=l.get("ms"),
                                             exp_avg_sq_scales=l.get("vs"))
        ttt.adamw_step(st["handle"], st["lists"]["g"], step=st["step"], lr=st["lr"], betas=st["betas"], eps=st["eps"],
                       weight_decay=st["decay"])
        return _adamw_outputs(st)
    if op == "attention":
        return _attention(st)
    if op == "attention_backward":
        return _attention_backward(st)
    if op == "attention_step":
        return _attention_step(st)
    if op == "norm":
        return _norm(st)
    if op == "norm_backward":
        return _norm_backward(st)
    _adamw(st)
    return _adamw_outputs(st)


def _pairs(case):
    """Visible (query, key) pairs of the packed sequences."""
    total, B, before, after, sinks = 0, case["block"], case["before"], case["after"], case["sinks"]
    for lq in _lengths(case):
        lk = lq + case["nk"] - case["nq"]
        b = torch.div(torch.arange(lk - lq, lk), B, rounding_mode="floor")
        hi = torch.full_like(b, lk) if after < 0 else ((b + after + 1) * B).clamp(0, lk)
        lo = torch.zeros_like(b) if before < 0 else ((b - before) * B).clamp(min=0)
        lo = torch.minimum(lo, hi)
        total += int((hi - lo + lo.clamp(max=sinks)).sum())
    return total


def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("attention"):
        H, Hk, d = case["heads"], case["key_heads"], case["d"]
        if op == "attention_step":
            seen = case["capacity"] if case["before"] < 0 else min(case["capacity"], case["before"] * case["block"] + 1 + case["sinks"])
            rows = case["n"] * min(case["capacity"], max(1, seen))
            return {"bytes": 2 * rows * Hk * d * es + case["n"] * (2 * H + 4 * Hk) * d * es, "flops": 4 * rows * H * d}
        rq, rk, lse = case["nq"] * H * d * es, case["nk"] * Hk * d * es, case["nq"] * H * 4
        pairs = _pairs(case) * H * d
        if op == "attention":
            return {"bytes": 2 * rq + 2 * rk + lse, "flops": 4 * pairs}
        return {"bytes": 4 * rq + 4 * rk + lse, "flops": 10 * pairs}
    if op.startswith("norm"):
        rows, w = case["n"] * case["width"], case["norm"]
        if op == "norm":
            return {"bytes": 2 * rows * es + 8 * w, "flops": 8 * rows}
        return {"bytes": 3 * rows * es + 12 * w, "flops": 16 * rows}
    n = sum(_sizes(case))
    state = 4 * (1 + 4 / BLOCK8) if case["bits"] == 8 else 16
    return {"bytes": n * (3 * es + (8 if case["dtype"] == "bf16" else 0) + state), "flops": 20 * n}


# ------------------------------------------------------------------ in 64 bits
def _exact_attention(st, backward):
    """Sequence by sequence, rows of the whole mask at a time."""
    H, Hk, d = st["heads"], st["key_heads"], st["d"]
    q, k, v = (st[x].double() for x in "qkv")
    out, lse = torch.zeros_like(q), torch.full((H, q.shape[0]), -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    q0 = k0 = 0
    for lq, lk in zip(st["lens"], st["lens_k"]):
        each = lambda x, a, b: x[a:b].reshape(b - a, x.shape[1] // d, d).transpose(0, 1).contiguous()
        ks, vs = each(k, k0, k0 + lk), each(v, k0, k0 + lk)
        step = max(1, (1 << 27) // max(1, H * lk))
        for a in range(0, lq, step):
            b = min(lq, a + step)
            pos = torch.arange(a, b, device=q.device)[:, None] + lk - lq
            j = torch.arange(lk, device=q.device)[None, :]
            own_block = torch.floor(pos.double() / st["block"])
            away = torch.floor(j.double() / st["block"]) - own_block        # blocks from the query's
            see = torch.ones_like(away, dtype=torch.bool)
            if st["before"] >= 0:
                see = (away >= -st["before"]) | (j < st["sinks"])
            if st["after"] >= 0:
                see &= away <= st["after"]
            qs = each(q, q0 + a, q0 + b)
            leaves = [x.repeat_interleave(r, 0).requires_grad_(backward) for x, r in ((qs, 1), (ks, H // Hk), (vs, H // Hk))]
            s = (leaves[0] @ leaves[1].transpose(1, 2) / math.sqrt(d)).masked_fill(~see, -math.inf)
            any_key = see.any(1)
            w = torch.softmax(s[:, any_key], -1)
            o = w @ leaves[2]
            if not backward:
                out[q0 + a:q0 + b][any_key] = o.transpose(0, 1).reshape(-1, H * d)
                lse[:, q0 + a:q0 + b] = torch.logsumexp(s, -1)
            elif w.numel():
                g = torch.autograd.grad(o, leaves, each(st["do"].double(), q0 + a, q0 + b)[:, any_key])
                dq[q0 + a:q0 + b] += g[0].transpose(0, 1).reshape(b - a, -1)
                for to, x in ((dk, g[1]), (dv, g[2])):
                    to[k0:k0 + lk] += x.view(Hk, -1, lk, d).sum(1).transpose(0, 1).reshape(lk, -1)
        q0, k0 = q0 + lq, k0 + lk
    return (dq, dk, dv) if backward else (out, lse)


def _exact_step(st):
    n, H, Hk, d, C, sinks = (st[x] for x in ("n", "heads", "key_heads", "d", "capacity", "sinks"))
    o = torch.zeros(n, H, d, dtype=torch.float64, device=st["q"].device)
    ring = C - sinks
    for i, (slot, p) in enumerate(zip(st["slots"].tolist(), st["positions"].tolist())):
        lo = 0 if st["before"] < 0 else max(0, (p // st["block"] - st["before"]) * st["block"])
        lo = max(lo, p + 1 - ring if p + 1 > C else 0)
        js = torch.cat([torch.arange(min(sinks, lo, p + 1)), torch.arange(lo, p + 1)])
        at = torch.where(js < sinks, js, sinks + (js - sinks) % ring).to(o.device)
        ks, vs = st["k_cache"][slot, at].double(), st["v_cache"][slot, at].double()
        ks[-1], vs[-1] = st["k"][i].double(), st["v"][i].double()
        st["k_cache"][slot, at[-1]], st["v_cache"][slot, at[-1]] = st["k"][i], st["v"][i]
        ks, vs = (x.view(-1, Hk, d).repeat_interleave(H // Hk, 1) for x in (ks, vs))
        w = torch.softmax(torch.einsum("hd,jhd->hj", st["q"][i].double().view(H, d), ks) / math.sqrt(d), -1)
        o[i] = torch.einsum("hj,jhd->hd", w, vs)
    return o.view(n, -1), None, None


def exact(case, seed):
    op, st = case["op"], prepare(case, seed)
    if op == "attention_step":
        return _exact_step(st)
    if op.startswith("attention"):
        return _exact_attention(st, op == "attention_backward")
    if op.startswith("norm"):
        w = st["norm"]
        leaf = lambda t: t.double().detach().requires_grad_(op == "norm_backward")
        x, ga, be = leaf(st["x"]), leaf(st["gamma"]), leaf(st["beta"])
        y = torch.nn.functional.layer_norm(x.unflatten(1, (-1, w)), (w,), ga, be, 1e-6).flatten(1)
        return y if op == "norm" else torch.autograd.grad(y, (x, ga, be), st["dy"].double())
    b1, b2 = st["betas"]
    if st["bits"] == 8:
        held = lambda c, s, top: (c.double() / top) ** 2 * torch.sign(c.double()) * s.double().repeat_interleave(BLOCK8)
        m, v = held(st["m"], st["ms"], 127), held(st["v"], st["vs"], 255) ** 2
    else:
        m, v = st["m"].double(), st["v"].double()
    p = (st["p"] if st["master"] is None else st["master"]).double()
    g, t = st["g"].double(), st["step"]
    m = torch.lerp(g, m, b1)
    v = torch.lerp(g.square(), v, b2)
    p = p - st["lr"] * (st["decay"] * p + (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + st["eps"]))
    states = (None, None) if st["bits"] == 8 else (m, v)
    return (p, None if st["master"] is None else p, *states)
