"""Timed cases of the gated delta rule, the gated residual tail of a block and Newton-Schulz
orthogonalisation, with each operator in elementary torch operations beside the library's call.

``own`` selects which of the two ``run`` computes.  ``exact`` states every operator once more in
64 bits, from its definition (token by token, by differentiation, from the other side).
"""
import math

import torch

own = False

CHUNK = 64                                  # tokens per chunk of the plain chunked form
NS = (3.4445, -4.7750, 2.0315)              # Muon's quintic
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one 518 x 518 frame (37 x 37 patches + 5 tokens) through a layer of four 256-wide heads
        dict(name="delta frame", op="delta", n=1374, seqs=1, cut=0, heads=4, key_heads=4, dk=256, dv=256, dtype="bf16"),
        # one 32-frame chunk of a causal stream, the state carried in and out
        dict(name="delta stream chunk", op="delta", n=43968, seqs=1, cut=0, heads=4, key_heads=4, dk=256, dv=256,
             dtype="bf16"),
        # training on eight object views of 1024 tokens, token width 768, keys shared by three heads
        dict(name="delta train views", op="delta_backward", n=8192, seqs=8, cut=0, heads=6, key_heads=2, dk=128, dv=128,
             dtype="bf16"),
        # fp32 training on packed sequences of uneven lengths, one of them empty and one a single token
        dict(name="delta train ragged", op="delta_backward", n=2731, seqs=6, cut=2, heads=4, key_heads=4, dk=64, dv=128,
             dtype="f32"),
        # one token of one sequence: what a stream pays per query
        dict(name="delta step one", op="delta_step", n=1, slots=4, heads=4, key_heads=4, dk=256, dv=256, dtype="bf16"),
        # one token for each of 300 sequences out of a pool of 512 states
        dict(name="delta step pool", op="delta_step", n=300, slots=512, heads=8, key_heads=4, dk=128, dv=128,
             dtype="bf16"),
        # the tail of a block on one frame, norm over each head
        dict(name="residual frame", op="residual", n=1374, width=1024, norm=256, gate=True, dtype="bf16"),
        # the same on 100 frames
        dict(name="residual 100 frames", op="residual", n=137400, width=1024, norm=256, gate=True, dtype="bf16"),
        # gradients over one 32-frame chunk
        dict(name="residual train chunk", op="residual_backward", n=43968, width=1024, norm=256, gate=True,
             dtype="bf16"),
        # gradients in fp32, norm over the row, no gate: the plain scaled residual
        dict(name="residual train f32", op="residual_backward", n=8192, width=768, norm=768, gate=False, dtype="f32"),
        # the fast-weight gradients of four heads (three matrices each)
        dict(name="orthogonalise heads", op="orthogonalise", batch=12, rows=512, cols=256, dtype="f32"),
        # projections of four blocks
        dict(name="orthogonalise projections", op="orthogonalise", batch=4, rows=4096, cols=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("delta", "delta_backward", "delta_step", "residual", "residual_backward", "orthogonalise"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op.startswith("delta"):
        heads = rng.choice((1, 2, 3, 4, 6, 8))
        key_heads = rng.choice([k for k in range(1, heads + 1) if heads % k == 0])
        dk = rng.choice((64, 128, 256))
        dv = rng.choice((64, 128, 192, 256))
        if op == "delta_step":
            n = _log(rng, 1, 300)
            return dict(op=op, n=n, slots=n + rng.randrange(0, 200), heads=heads, key_heads=key_heads, dk=dk, dv=dv,
                        dtype=dtype)
        n = _log(rng, 1, 20000) if op == "delta" else _log(rng, 1, 6000)
        return dict(op=op, n=n, seqs=rng.choice((1, 1, 2, 3, 5, 9)), cut=rng.randrange(1, 1 << 20), heads=heads,
                    key_heads=key_heads, dk=dk, dv=dv, dtype=dtype)
    if op.startswith("residual"):
        norm = 8 * rng.randrange(1, 65)
        width = norm * rng.choice((1, 2, 3, 4))
        n = _log(rng, 1, 40000)
        return dict(op=op, n=n, width=width, norm=norm, gate=rng.random() < 0.7, dtype=dtype)
    return dict(op=op, batch=rng.choice((1, 2, 3, 5)), rows=_log(rng, 16, 1400), cols=_log(rng, 16, 1400), dtype=dtype)


def _lengths(case):
    """Token counts of the packed sequences.  cut = 0: even; else uneven, and from four sequences on one is
    empty and one a single token."""
    n, s = case["n"], case["seqs"]
    if case["cut"] == 0:
        return [(n + i) // s for i in range(s)]
    g = torch.Generator().manual_seed(case["cut"])
    fixed = [0, 1] if s >= 4 and n > 1 else []
    left = n - sum(fixed)
    cuts = sorted(torch.randint(0, left + 1, (s - len(fixed) - 1,), generator=g).tolist())
    lens = [b - a for a, b in zip([0] + cuts, cuts + [left])]
    return lens[:1] + fixed + lens[1:]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)
    op, st = case["op"], dict(case)
    dt = DT[case["dtype"]]
    if op.startswith("delta"):
        n, H, Hk, dk, dv = case["n"], case["heads"], case["key_heads"], case["dk"], case["dv"]
        unit = lambda t: t / t.norm(dim=-1, keepdim=True)
        st["q"] = unit(rn(n, Hk, dk)).reshape(n, Hk * dk).to(dt)
        st["k"] = unit(rn(n, Hk, dk)).reshape(n, Hk * dk).to(dt)
        st["v"] = rn(n, H * dv).to(dt)
        st["beta"] = torch.sigmoid(rn(H, n))
        # heads forget over 2 to 1000 tokens
        rate = torch.exp(torch.linspace(math.log(1e-3), math.log(0.5), H, device=dev))[:, None]
        st["decay"] = -rate * torch.exp(0.5 * rn(H, n))
        if op == "delta_step":
            st["w"] = rn(case["slots"], H, dv, dk) / math.sqrt(dk)
            st["slots"] = torch.randperm(case["slots"], generator=g, device=dev)[:n].to(torch.int32)
        else:
            lens = _lengths(case)
            st["lens"] = lens
            st["cu"] = torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)
            st["w"] = rn(len(lens), H, dv, dk) / math.sqrt(dk)
            if op == "delta_backward":
                st["do"] = rn(n, H * dv).to(dt)
                st["dw"] = rn(len(lens), H, dv, dk) / math.sqrt(dk)
    elif op.startswith("residual"):
        n, C = case["n"], case["width"]
        st["x"] = (4.0 * rn(n, C)).to(dt)
        st["o"] = (0.3 * rn(n, C)).to(dt)
        st["z"] = rn(n, C).to(dt) if case["gate"] else None
        st["gamma"], st["gamma_next"] = 1.0 + 0.1 * rn(C), 1.0 + 0.1 * rn(C)
        st["alpha"] = 0.1 + 0.05 * rn(C)
        if op == "residual_backward":
            st["dy"], st["dh"] = rn(n, C).to(dt), rn(n, C).to(dt)
            # the forward's output, which training keeps
            st["y"] = _residual(st, torch.float64)[0].to(dt)
    else:
        st["g"] = (1e-3 * rn(case["batch"], case["rows"], case["cols"])).to(dt)
    return st


# ------------------------------------------------------------------ the plain forms
def _blocks(st, rows, width):
    """Packed rows [n, heads * width] -> zero-padded fp32 chunks [seqs, heads, chunks, CHUNK, width]."""
    lens, cu = st["lens"], st["cu"].long()
    T = max(1, -(-max(lens) // CHUNK)) * CHUNK
    t = torch.arange(T, device=rows.device)
    ok = t < (cu[1:] - cu[:-1])[:, None]
    idx = (cu[:-1, None] + t).clamp_(max=max(0, rows.shape[0] - 1))
    x = rows.float()[idx] * ok[..., None]
    return x.view(len(lens), T // CHUNK, CHUNK, -1, width).permute(0, 3, 1, 2, 4).contiguous()


def _rows(st, x):
    """The reverse of _blocks: the packed rows of [seqs, heads, chunks, CHUNK, width]."""
    B, H, N, C, w = x.shape
    cu = st["cu"].long()
    t = torch.arange(N * C, device=x.device)
    ok = t < (cu[1:] - cu[:-1])[:, None]
    return x.permute(0, 2, 3, 1, 4).reshape(B, N * C, H * w)[ok]


def _chunk_terms(st):
    """What every chunk has before the state is known."""
    H, Hk, dk, dv, r = st["heads"], st["key_heads"], st["dk"], st["dv"], st["heads"] // st["key_heads"]
    c = {}
    c["q"] = _blocks(st, st["q"], dk).repeat_interleave(r, 1)
    c["k"] = _blocks(st, st["k"], dk).repeat_interleave(r, 1)
    c["v"] = _blocks(st, st["v"], dv)
    c["beta"] = _blocks(st, st["beta"].t(), 1)
    gam = _blocks(st, st["decay"].t(), 1)[..., 0].double().cumsum(-1)
    c["eg"] = gam.exp().float()[..., None]
    c["el"] = (gam[..., -1:] - gam).exp().float()[..., None]
    c["eC"] = gam[..., -1].exp().float()[..., None, None]
    tri = torch.ones(CHUNK, CHUNK, device=gam.device, dtype=torch.bool).tril()
    c["D"] = (gam[..., :, None] - gam[..., None, :]).masked_fill(~tri, -math.inf).exp().float()
    c["kk"] = c["k"] @ c["k"].transpose(-1, -2)
    c["A"] = (c["q"] @ c["k"].transpose(-1, -2)) * c["D"]
    c["BD"] = (c["beta"] * c["D"]).tril(-1)
    L = c["BD"] * c["kk"]
    # (I + L)^-1 row by row: powers of L lose every digit where keys repeat, substitution does not
    T = torch.eye(CHUNK, device=L.device).expand_as(L).contiguous()
    for i in range(1, CHUNK):
        T[..., i, :i] = -(L[..., i, None, :i] @ T[..., :i, :i])[..., 0, :]
    c["T"], c["L"] = T, L
    return c


def _delta(st):
    c = _chunk_terms(st)
    u0 = c["T"] @ (c["beta"] * c["v"])
    wd = c["T"] @ (c["beta"] * c["eg"] * c["k"])
    s = st["w"].transpose(-1, -2)                       # [seqs, heads, dk, dv]
    qg, kl = c["q"] * c["eg"], (c["k"] * c["el"]).transpose(-1, -2)
    outs = []
    for i in range(u0.shape[2]):
        u = u0[:, :, i] - wd[:, :, i] @ s
        outs.append(qg[:, :, i] @ s + c["A"][:, :, i] @ u)
        s = c["eC"][:, :, i] * s + kl[:, :, i] @ u
    return _rows(st, torch.stack(outs, 2)).to(st["q"].dtype), s.transpose(-1, -2).contiguous()


def _delta_backward(st):
    c = _chunk_terms(st)
    q, k, v, beta, eg, el, eC, T, A = (c[x] for x in ("q", "k", "v", "beta", "eg", "el", "eC", "T", "A"))
    do = _blocks(st, st["do"], st["dv"])
    N = q.shape[2]
    s, S, E, U = st["w"].transpose(-1, -2), [], [], []
    for i in range(N):
        S.append(s)
        e = v[:, :, i] - eg[:, :, i] * (k[:, :, i] @ s)
        u = T[:, :, i] @ (beta[:, :, i] * e)
        s = eC[:, :, i] * s + (k[:, :, i] * el[:, :, i]).transpose(-1, -2) @ u
        E.append(e)
        U.append(u)
    S, E, U = torch.stack(S, 2), torch.stack(E, 2), torch.stack(U, 2)
    du0 = A.transpose(-1, -2) @ do
    qdo = (q * eg).transpose(-1, -2) @ do
    ds, dS, dR = st["dw"].transpose(-1, -2), [], []
    for i in reversed(range(N)):
        dS.append(ds)
        du = du0[:, :, i] + el[:, :, i] * (k[:, :, i] @ ds)
        dr = T[:, :, i].transpose(-1, -2) @ du
        ds = eC[:, :, i] * ds + qdo[:, :, i] - k[:, :, i].transpose(-1, -2) @ (beta[:, :, i] * eg[:, :, i] * dr)
        dR.append(dr)
    dS, dR = torch.stack(dS[::-1], 2), torch.stack(dR[::-1], 2)
    dp = -beta * eg * dR
    dA, dL = do @ U.transpose(-1, -2), -(dR @ U.transpose(-1, -2))
    X = dA * c["D"]
    Y = dL * c["BD"]
    dq = eg * (do @ S.transpose(-1, -2)) + X @ k
    dk = (dp @ S.transpose(-1, -2) + el * (U @ dS.transpose(-1, -2)) + X.transpose(-1, -2) @ q
          + (Y + Y.transpose(-1, -2)) @ k)
    dbeta = (dR * E).sum(-1) + (dL * c["D"].tril(-1) * c["kk"]).sum(-1)
    M = dA * A + dL * c["L"]
    last = el[..., 0] * (U * (k @ dS)).sum(-1)
    dgam = ((eg * do) * (q @ S)).sum(-1) + (dp * (k @ S)).sum(-1) + M.sum(-1) - M.sum(-2) - last
    dgam[..., -1] += eC[..., 0, 0] * (S * dS).sum((-1, -2)) + last.sum(-1)
    ddecay = dgam.flip(-1).cumsum(-1).flip(-1)
    r = st["heads"] // st["key_heads"]
    group = lambda t: t.unflatten(1, (-1, r)).sum(2)
    dt = st["q"].dtype
    heads = lambda t: _rows(st, t[..., None]).t().contiguous()
    return (_rows(st, group(dq)).to(dt), _rows(st, group(dk)).to(dt), _rows(st, beta * dR).to(dt), heads(dbeta),
            heads(ddecay), ds.transpose(-1, -2).contiguous())


def _delta_step(st):
    H, Hk, dk, dv, n = st["heads"], st["key_heads"], st["dk"], st["dv"], st["n"]
    slots = st["slots"].long()
    q = st["q"].float().view(n, Hk, dk).repeat_interleave(H // Hk, 1)[:, :, None, :]
    k = st["k"].float().view(n, Hk, dk).repeat_interleave(H // Hk, 1)[:, :, None, :]
    p = st["w"][slots] * st["decay"].t().exp()[..., None, None]
    e = st["v"].float().view(n, H, dv) - (p * k).sum(-1)
    w = p + (st["beta"].t()[..., None] * e)[..., None] * k
    o = (w * q).sum(-1).reshape(n, H * dv).to(st["q"].dtype)
    st["w"][slots] = w
    return o, st["w"]


def _residual(st, f):
    x, o = st["x"].to(f), st["o"].to(f)
    n, C = x.shape
    w = st["norm"]
    og = o.view(n, C // w, w)
    u = (og * torch.rsqrt((og * og).mean(-1, keepdim=True) + 1e-6)).view(n, C) * st["gamma"].to(f)
    if st["z"] is not None:
        z = st["z"].to(f)
        u = u * (z / (1 + torch.exp(-z)))
    y = x + st["alpha"].to(f) * u
    h = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * st["gamma_next"].to(f)
    return y, h


def _residual_backward(st):
    y, o, dy, dh = (st[x].float() for x in ("y", "o", "dy", "dh"))
    n, C = y.shape
    w = st["norm"]
    r2 = torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
    yn, t = y * r2, dh * st["gamma_next"]
    dx = dy + r2 * (t - yn * (t * yn).mean(-1, keepdim=True))
    og = o.view(n, C // w, w)
    r1 = torch.rsqrt((og * og).mean(-1, keepdim=True) + 1e-6)
    on = (og * r1).view(n, C)
    sil, dz = 1.0, None
    if st["z"] is not None:
        z = st["z"].float()
        sg = 1 / (1 + torch.exp(-z))
        sil = z * sg
        dz = (dx * st["alpha"] * st["gamma"] * on * sg * (1 + z * (1 - sg))).to(st["y"].dtype)
    ws = (dx * sil * on).sum(0)
    t = (dx * sil * (st["alpha"] * st["gamma"])).view(n, C // w, w)
    ong = on.view(n, C // w, w)
    do = (r1 * (t - ong * (t * ong).mean(-1, keepdim=True))).view(n, C)
    dt = st["y"].dtype
    return (dx.to(dt), do.to(dt), dz, st["alpha"] * ws, st["gamma"] * ws, (dh * yn).sum(0))


def _orthogonalise(st):
    g = st["g"].float()
    tall = g.shape[1] > g.shape[2]
    x = g.transpose(1, 2).contiguous() if tall else g
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + 1e-7)
    a, b, c = NS
    for _ in range(5):
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    return (x.transpose(1, 2).contiguous() if tall else x).to(st["g"].dtype)


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["op"]
    if own:
        from test_weight_layers_amd import ttt

        if op == "delta":
            return ttt.delta(st["w"], st["q"], st["k"], st["v"], st["beta"], st["decay"], key_heads=st["key_heads"],
                             cu_seqlens=st["cu"])
        if op == "delta_backward":
            return ttt.delta_backward(st["w"], st["q"], st["k"], st["v"], st["beta"], st["decay"], st["do"], st["dw"],
                                      key_heads=st["key_heads"], cu_seqlens=st["cu"])
        if op == "delta_step":
            return ttt.delta_step(st["w"], st["q"], st["k"], st["v"], st["beta"], st["decay"],
                                  key_heads=st["key_heads"], slots=st["slots"]), st["w"]
        if op == "residual":
            return ttt.gated_residual(st["x"], st["o"], st["z"], st["gamma"], st["alpha"], st["gamma_next"], 1e-6,
                                      norm_width=st["norm"])
        if op == "residual_backward":
            return ttt.gated_residual_backward(st["dy"], st["dh"], st["y"], st["o"], st["z"], st["gamma"], st["alpha"],
                                               st["gamma_next"], 1e-6, norm_width=st["norm"])
        return ttt.orthogonalise(st["g"])
    if op == "delta":
        return _delta(st)
    if op == "delta_backward":
        return _delta_backward(st)
    if op == "delta_step":
        return _delta_step(st)
    if op == "residual":
        y, h = _residual(st, torch.float32)
        return y.to(st["x"].dtype), h.to(st["x"].dtype)
    if op == "residual_backward":
        return _residual_backward(st)
    return _orthogonalise(st)


def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("delta"):
        n, H, Hk, dk, dv = case["n"], case["heads"], case["key_heads"], case["dk"], case["dv"]
        key, val, rate, state = n * Hk * dk * es, n * H * dv * es, n * H * 4, H * dk * dv * 4
        if op == "delta_step":
            return {"bytes": 2 * key + 2 * val + 2 * rate + 2 * n * state + 4 * n, "flops": 6 * n * H * dk * dv}
        if op == "delta":
            return {"bytes": 2 * key + 2 * val + 2 * rate + 2 * case["seqs"] * state, "flops": 6 * n * H * dk * dv}
        return {"bytes": 4 * key + 3 * val + 4 * rate + 3 * case["seqs"] * state, "flops": 18 * n * H * dk * dv}
    if op.startswith("residual"):
        rows = case["n"] * case["width"] * es
        if op == "residual":
            return {"bytes": (5 if case["gate"] else 4) * rows + 12 * case["width"], "flops": 20 * case["n"] * case["width"]}
        return {"bytes": (8 if case["gate"] else 6) * rows + 24 * case["width"], "flops": 40 * case["n"] * case["width"]}
    r, c = sorted((case["rows"], case["cols"]))
    # the products A = X X^T and A A are symmetric: half of each
    return {"bytes": 2 * case["batch"] * r * c * es, "flops": 5 * case["batch"] * (3 * r * r * c + r ** 3)}


# ------------------------------------------------------------------ in 64 bits
def _tokens64(st):
    """[longest, seqs * heads, ...] of every token-wise input in fp64, and which of them are tokens."""
    H, r = st["heads"], st["heads"] // st["key_heads"]
    lens, cu = st["lens"], [0]
    for x in lens:
        cu.append(cu[-1] + x)
    T = max(1, max(lens))

    def pad(rows, width):
        x = rows.new_zeros(T, len(lens), rows.shape[1], dtype=torch.float64)
        for b, m in enumerate(lens):
            x[:m, b] = rows[cu[b]:cu[b + 1]].double()
        x = x.view(T, len(lens), -1, width)
        return x.repeat_interleave(H // x.shape[2], 2).reshape(T, -1, width)

    ins = [pad(st["q"], st["dk"]), pad(st["k"], st["dk"]), pad(st["v"], st["dv"]), pad(st["beta"].t(), 1),
           pad(st["decay"].t(), 1)]

    def rows(x):
        x = x.view(T, len(lens), -1)
        return torch.cat([x[:m, b] for b, m in enumerate(lens)])

    return ins, pad, rows, r


def _exact_delta(st):
    (q, k, v, be, de), _, rows, _ = _tokens64(st)
    w = st["w"].double().flatten(0, 1)
    out = torch.empty_like(v)
    a = de.exp()[..., None]
    for t in range(q.shape[0]):
        w = w * a[t]
        e = be[t] * torch.baddbmm(v[t, :, :, None], w, k[t, :, :, None], alpha=-1)[..., 0]
        w = torch.baddbmm(w, e[:, :, None], k[t, :, None, :])
        out[t] = (w @ q[t, :, :, None])[..., 0]
    return rows(out), w.view(st["w"].shape)


def _exact_delta_backward(st):
    (q, k, v, be, de), pad, rows, r = _tokens64(st)
    do = pad(st["do"], st["dv"])
    w, dw = st["w"].double().flatten(0, 1), st["dw"].double().flatten(0, 1)
    T, a, step = q.shape[0], de.exp()[..., None], 128
    kept = []
    forward = lambda p, t: p + (be[t] * (v[t] - (p @ k[t, :, :, None])[..., 0]))[:, :, None] * k[t, :, None, :]
    for t in range(T):
        if t % step == 0:
            kept.append(w)
        w = forward(w * a[t], t)
    dq, dk, dv, dbe, dde = (torch.zeros_like(x) for x in (q, k, v, be, de))
    for s in reversed(range(0, T, step)):
        w, ps = kept[s // step], []
        for t in range(s, min(T, s + step)):
            ps.append(w * a[t])
            w = forward(ps[-1], t)
        for t in reversed(range(s, min(T, s + step))):
            p = ps[t - s]
            e = v[t] - (p @ k[t, :, :, None])[..., 0]
            w = p + (be[t] * e)[:, :, None] * k[t, :, None, :]
            dq[t] = (do[t, :, None, :] @ w)[:, 0]
            dw = dw + do[t, :, :, None] * q[t, :, None, :]
            g = (dw @ k[t, :, :, None])[..., 0]
            dbe[t] = (g * e).sum(-1, keepdim=True)
            dv[t] = be[t] * g
            dk[t] = ((be[t] * e)[:, None, :] @ dw - dv[t, :, None, :] @ p)[:, 0]
            dw = dw - dv[t, :, :, None] * k[t, :, None, :]
            dde[t] = (dw * p).sum((1, 2))[:, None]
            dw = dw * a[t]
    shared = lambda x: rows(x.view(T, -1, r, x.shape[-1]).sum(2))
    return (shared(dq), shared(dk), rows(dv), rows(dbe).t().contiguous(), rows(dde).t().contiguous(),
            dw.view(st["w"].shape))


def _exact_delta_step(st):
    n, H, r = st["n"], st["heads"], st["heads"] // st["key_heads"]
    d = lambda x, width: x.double().view(n, -1, width).repeat_interleave(H // (x.shape[1] // width), 1)
    q, k, v = d(st["q"], st["dk"]), d(st["k"], st["dk"]), d(st["v"], st["dv"])
    w = st["w"].double()
    p = w[st["slots"].long()] * st["decay"].double().t().exp()[..., None, None]
    e = v - torch.einsum("nhvk,nhk->nhv", p, k)
    p = p + torch.einsum("nh,nhv,nhk->nhvk", st["beta"].double().t(), e, k)
    w[st["slots"].long()] = p
    return torch.einsum("nhvk,nhk->nhv", p, q).reshape(n, -1), w


def _exact_residual_backward(st):
    leaf = lambda t: t.double().detach().requires_grad_(True)
    C, w = st["width"], st["norm"]
    o, ga, al, gn = leaf(st["o"]), leaf(st["gamma"]), leaf(st["alpha"]), leaf(st["gamma_next"])
    z = leaf(st["z"]) if st["z"] is not None else None
    y = leaf(st["y"])
    h = torch.nn.functional.rms_norm(y, (C,), gn, 1e-6)
    dyh, dgn = torch.autograd.grad(h, (y, gn), st["dh"].double())
    dx = dyh + st["dy"].double()
    u = torch.nn.functional.rms_norm(o.view(-1, C // w, w), (w,), None, 1e-6).view(-1, C) * ga
    if z is not None:
        u = u * torch.nn.functional.silu(z)
    gr = torch.autograd.grad(al * u, (o, ga, al) + ((z,) if z is not None else ()), dx)
    return dx, gr[0], gr[3] if z is not None else None, gr[1], gr[2], dgn


def _exact_orthogonalise(st):
    x = st["g"].double()
    x = x / (x.flatten(1).norm(dim=1)[:, None, None] + 1e-7)
    a, b, c = NS
    wide = x.shape[2] >= x.shape[1]
    n = min(x.shape[1:])
    eye = torch.eye(n, device=x.device, dtype=x.dtype)
    for _ in range(5):
        xt = x.transpose(1, 2).contiguous()
        s = x @ xt if wide else xt @ x
        p = a * eye + s @ (b * eye + c * s)
        x = p @ x if wide else x @ p
    return x


def exact(case, seed):
    op = case["op"]
    if op == "delta_backward" and case["n"] > 20000:
        return None
    st = prepare(case, seed)
    if op == "delta":
        return _exact_delta(st)
    if op == "delta_backward":
        return _exact_delta_backward(st)
    if op == "delta_step":
        return _exact_delta_step(st)
    if op == "residual":
        x, o, C, w = st["x"].double(), st["o"].double(), st["width"], st["norm"]
        rms = torch.nn.functional.rms_norm
        u = rms(o.view(-1, C // w, w), (w,), None, 1e-6).view(-1, C) * st["gamma"]
        y = x + st["alpha"] * (u if st["z"] is None else u * torch.nn.functional.silu(st["z"].double()))
        return y, rms(y, (C,), st["gamma_next"].double(), 1e-6)
    if op == "residual_backward":
        return _exact_residual_backward(st)
    return _exact_orthogonalise(st)
