"""The training operators beside the attention forward pass: cases, plain forms and exact values.

  attention's backward pass   dq, dk, dv from q, k, v, out, lse and the gradient of out; the probabilities are
                              recomputed from lse.  Key-only padding, a general bit mask, cross-attention.
  layer norm                  forward (y, mean, rstd) and backward (dx, dweight, dbias); with or without the mean
                              (center), one weight vector or one per batch entry (a DiT block's modulation).
  rotary positions            interleaved and half layouts, part of the head, one to three position axes, scaled
                              frequencies, far positions; forward and inverse (the gradient).

`run` computes the plain form with elementary torch operations in 32 bits (angles in 64), or, with `own` set,
makes the calls a user makes of the library.
"""
import math

import torch

own = False
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # attention backward: the `tiny` workload, where launches and latency count
        _attn("attn_bwd_tiny", B=1, Nq=1024, Nkv=1024, H=2, D=64),
        # a quarter of the LTX-2-shaped padded sequence (24,576 / 4 tokens, 24,200 / 4 valid) with a quarter of its heads
        _attn("attn_bwd_ltx2_quarter", B=1, Nq=6144, Nkv=6144, H=8, D=128, valid=6050, fused=True),
        # one key chunk of the ring-style workload (16,384 keys) against as many queries: the largest call
        _attn("attn_bwd_ring_chunk", B=1, Nq=16384, Nkv=16384, H=8, D=128),
        # video queries over a short, ragged text: few key rows, a long sum for each
        _attn("attn_bwd_cross_text", B=2, Nq=11040, Nkv=241, H=16, D=64),
        # frame-local attention with a general mask: most tiles empty
        _attn("attn_bwd_frames", B=2, Nq=4096, Nkv=4096, H=4, D=128, valid=4000, frame=500),
        # a block's pre-attention norm with modulation per batch entry, 32 heads of 128: forward and backward
        _norm("norm_fwd_block", B=2, N=12288, H=1, C=4096, per_batch=True),
        _norm("norm_bwd_block", B=2, N=12288, H=1, C=4096, per_batch=True, backward=True),
        # a single request's few tokens in the forward pass of a small step
        _norm("norm_fwd_few_rows", B=1, N=31, H=1, C=2048),
        # q's head-wise RMS norm, read in place from the fused projection: many short rows, one weight of 128
        _norm("norm_bwd_heads", B=1, N=11040, H=16, C=128, center=False, bias=False, backward=True, strided=True),
        # q and k of the fused projection rotated by three position axes (16 x 32 x 48 latent grid)
        _rope("rope_video_grid", B=1, N=24576, H=64, D=128, R=128, axes=3, strided=True),
        # the gradient in the half layout, a quarter of the head left alone, positions far out on a scaled schedule
        _rope("rope_half_long", B=2, N=5001, H=16, D=128, R=96, half=True, far=1_000_000, scaled=8.0, inverse=True),
        # one new token for each of 48 sequences
        _rope("rope_single_token", B=48, N=1, H=32, D=64, R=64, half=True, far=131_072),
    ]


def _attn(name, *, B, Nq, Nkv, H, D, valid=-1, frame=0, fused=False):
    return {"name": name, "op": "attn_bwd", "B": B, "Nq": Nq, "Nkv": Nkv, "H": H, "D": D,
            "valid": Nkv if valid < 0 else valid, "frame": frame, "fused": fused}


def _norm(name, *, B, N, H, C, center=True, bias=True, per_batch=False, backward=False, strided=False, fp32=False):
    return {"name": name, "op": "norm", "B": B, "N": N, "H": H, "C": C, "center": center, "bias": bias,
            "per_batch": per_batch, "backward": backward, "strided": strided, "fp32": fp32}


def _rope(name, *, B, N, H, D, R, half=False, axes=1, far=0, scaled=1.0, inverse=False, strided=False, fp32=False):
    return {"name": name, "op": "rope", "B": B, "N": N, "H": H, "D": D, "R": R, "half": half, "axes": axes, "far": far,
            "scaled": scaled, "inverse": inverse, "strided": strided, "fp32": fp32}


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(("attn", "norm", "rope"))
    if kind == "attn":
        D = rng.choice((64, 128))
        nq, nkv = _spread(rng, 1, 16384), _spread(rng, 16, 16384)  # (a few keys' gradients are differences of like values)
        form = rng.choice(("plain", "padded", "self", "frames"))
        if form in ("self", "frames"):
            nkv = nq = max(nq, nkv)
        heads = max(1, min(64, (1 << 31) // (nq * nkv)))
        B = rng.randint(1, min(3, heads))
        H = _spread(rng, 1, max(1, min(24, heads // B)))
        valid = nkv if form == "plain" else rng.randint(nkv - nkv // 8, nkv)
        frame = _spread(rng, 16, nkv) if form == "frames" else 0
        c = _attn("", B=B, Nq=nq, Nkv=nkv, H=H, D=D, valid=valid, frame=frame, fused=form == "self" and rng.random() < 0.5)
    elif kind == "norm":
        H = rng.choice((1, 1, rng.randint(2, 24)))
        C = _spread(rng, 16, 8192) if H == 1 else rng.choice((64, 80, 128))
        rows = _spread(rng, 1, max(1, min(200_000, 24576 * 4096 // C)))
        B = rng.randint(1, min(4, rows))
        c = _norm("", B=B, N=max(1, rows // (B * H)), H=H, C=C, center=rng.random() < 0.7, bias=rng.random() < 0.7,
                  per_batch=rng.random() < 0.4, backward=rng.random() < 0.5, strided=rng.random() < 0.4, fp32=rng.random() < 0.2)
    else:
        D = 8 * _spread(rng, 4, 32)
        R = min(D, 2 * rng.randint(4, D // 2)) if rng.random() < 0.6 else D
        H = _spread(rng, 1, 80)
        B = rng.randint(1, 64)
        N = _spread(rng, 1, max(1, 24576 * 64 * 128 // (B * H * D)))
        c = _rope("", B=B, N=N, H=H, D=D, R=R, half=rng.random() < 0.5, axes=rng.choice((1, 1, 2, 3)),
                  far=rng.choice((0, 4096, 131_072, 1_000_000)), scaled=rng.choice((1.0, 4.0, 32.0)),
                  inverse=rng.random() < 0.4, strided=rng.random() < 0.4, fp32=rng.random() < 0.2)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _normal(shape, gen, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    return {"attn_bwd": _prepare_attn, "norm": _prepare_norm, "rope": _prepare_rope}[case["op"]](dict(case), gen)


def _prepare_attn(c, gen):
    B, Nq, Nkv, H, D, valid = c["B"], c["Nq"], c["Nkv"], c["H"], c["D"], c["valid"]
    if c["fused"]:
        qkv = _normal((B, Nq, 3, H, D), gen)
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    else:
        q, k, v = _normal((B, Nq, H, D), gen, 1.5), _normal((B, Nkv, H, D), gen), _normal((B, Nkv, H, D), gen)
    s = {"c": c, "q": q, "k": k, "v": v, "dout": _normal((B, Nq, H, D), gen, 0.25), "scale": D ** -0.5, "bits": None}
    if c["frame"]:  # queries attend their own frame and the frame of the first token; frames start at a seeded offset
        off = int(torch.randint(0, c["frame"], (1,), generator=gen, device=DEV))
        f = (torch.arange(valid, device=DEV) + off) // c["frame"]
        allow = (f[:, None] == f[None, :]) | (f[None, :] == f[0])
        words = 4 * ((valid + 127) // 128)
        padded = torch.zeros((valid, words * 32), dtype=torch.int64, device=DEV)
        padded[:, :valid] = allow
        w = (padded.view(valid, words, 32) << torch.arange(32, device=DEV)).sum(-1)
        s["bits"] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)[None]
    # the forward pass' results, as the program has them before it goes backward
    out, lse = torch.empty((B, Nq, H, D), dtype=torch.bfloat16, device=DEV), torch.empty((B, H, Nq), device=DEV)
    for b in range(B):
        for h in range(H):
            x = (q[b, :, h].float() @ k[b, :valid, h].float().T).mul_(s["scale"])
            if c["frame"]:
                x[:valid].masked_fill_(~allow, -math.inf)
            lse[b, h] = torch.logsumexp(x, 1)
            out[b, :, h] = (torch.exp(x.sub_(lse[b, h][:, None])) @ v[b, :valid, h].float()).to(torch.bfloat16)
    s["out"], s["lse"] = out, lse
    return s


def _prepare_norm(c, gen):
    B, N, H, C = c["B"], c["N"], c["H"], c["C"]
    dtype = torch.float32 if c["fp32"] else torch.bfloat16
    whole = _normal((B, N, 3 * H if c["strided"] else H, C), gen, 2.0, dtype)
    whole += torch.randn((C,), generator=gen, device=DEV).to(dtype)  # channels with means of their own
    x = whole[:, :, :H]
    shape = (B, C) if c["per_batch"] else (C,)
    s = {"c": c, "x": x, "weight": 1 + 0.3 * torch.randn(shape, generator=gen, device=DEV),
         "bias": 0.2 * torch.randn(shape, generator=gen, device=DEV) if c["bias"] else None, "eps": 1e-6}
    if c["backward"]:
        s["dy"] = _normal((B, N, H, C), gen, 0.5, dtype)
        f = x.float()
        mu = f.mean(-1)
        s["mean"] = mu if c["center"] else None
        if c["center"]:
            f = f - mu[..., None]
        s["rstd"] = (f.square().mean(-1) + s["eps"]).rsqrt()
    return s


def _prepare_rope(c, gen):
    B, N, H, D, R, A = c["B"], c["N"], c["H"], c["D"], c["R"], c["axes"]
    dtype = torch.float32 if c["fp32"] else torch.bfloat16
    x = _normal((B, N, H + H // 2 + 1 if c["strided"] else H, D), gen, 1.0, dtype)[:, :, :H]
    # the plan a program keeps: the pairs of each axis and their angles per step, slow pairs slowed for long contexts
    P = R // 2
    pairs = [P // A + (1 if a < P % A else 0) for a in range(A)] if A > 1 else [P]
    freq = []
    for n in pairs:
        for i in range(n):
            f = 10000.0 ** (-i / n)
            ramp = min(1.0, max(0.0, (i / n - 0.25) * 2.0))
            freq.append(f * (1.0 - ramp) + f / c["scaled"] * ramp)
    if A == 1:
        start = torch.randint(0, c["far"] + 1, (B, 1, 1), generator=gen, device=DEV)
        pos = start + torch.arange(N, device=DEV)[None, :, None]
    else:
        pos = torch.randint(0, max(64, c["far"]), (1, N, A), generator=gen, device=DEV)
    return {"c": c, "x": x, "pos": pos.to(torch.int32), "pairs": tuple(pairs), "freq": torch.tensor(freq, dtype=torch.float64),
            "freq_dev": torch.tensor(freq, dtype=torch.float64, device=DEV),
            "axis_dev": torch.tensor([a for a, n in enumerate(pairs) for _ in range(n)], device=DEV),
            "mscale": 1.0 if c["scaled"] == 1.0 else 0.1 * math.log(c["scaled"]) + 1.0}


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["c"]["op"]
    if own:
        return _own(state, op)
    if op == "attn_bwd":
        return _plain_attn(state)
    if op == "norm":
        return _plain_norm_bwd(state) if state["c"]["backward"] else _plain_norm_fwd(state)
    return _plain_rope(state)


def _own(s, op):
    import dit_long_sequence_gb300 as dl
    c = s["c"]
    if op == "attn_bwd":
        if s["bits"] is not None:
            return dl.attn_bwd_masked(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["bits"],
                                      key_valid_len=c["valid"], scale=s["scale"])
        return dl.attn_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], key_valid_len=c["valid"], scale=s["scale"])
    if op == "norm":
        if c["backward"]:
            got = dl.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"], has_bias=c["bias"])
        else:
            got = dl.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=s["eps"], center=c["center"])
        return tuple(t for t in got if t is not None)
    return dl.rope(s["x"], s["freq"], s["pos"], layout="half" if c["half"] else "interleaved", axis_pairs=s["pairs"],
                   mscale=s["mscale"], inverse=c["inverse"])


def _plain_attn(s):
    c, scale = s["c"], s["scale"]
    valid, Nq, Nkv = c["valid"], c["Nq"], c["Nkv"]
    q, dout, out = (s[n].float().transpose(1, 2) for n in ("q", "dout", "out"))  # [B, H, N, D]
    k, v = (s[n][:, :valid].float().transpose(1, 2) for n in ("k", "v"))
    p = (q @ k.transpose(-1, -2)).mul_(scale).sub_(s["lse"][..., None]).exp_()
    if s["bits"] is not None:
        at = torch.arange(valid, device=q.device)
        allow = (s["bits"][0][:, at >> 5] >> (at & 31)) & 1
        p[:, :, :valid].masked_fill_(allow == 0, 0.0)  # rows past the mask attend every valid key
    dv = p.transpose(-1, -2) @ dout
    delta = (dout * out).sum(-1, keepdim=True)
    ds = (dout @ v.transpose(-1, -2)).sub_(delta).mul_(p)
    del p
    dq = (ds @ k) * scale
    dk = (ds.transpose(-1, -2) @ q) * scale
    pad = (0, 0, 0, Nkv - valid)  # keys that nobody attends have no gradient
    return tuple(torch.nn.functional.pad(g, p_).transpose(1, 2).to(torch.bfloat16)
                 for g, p_ in ((dq, (0, 0)), (dk, pad), (dv, pad)))


def _rows(p):
    """A parameter [C] or [B, C] beside [B, N, H, C]."""
    return p if p.dim() == 1 else p[:, None, None]


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(-1) if s["c"]["center"] else None
    d = x - mean[..., None] if mean is not None else x
    rstd = (d.square().mean(-1) + s["eps"]).rsqrt()
    y = d * rstd[..., None] * _rows(s["weight"])
    if s["bias"] is not None:
        y = y + _rows(s["bias"])
    y = y.to(s["x"].dtype)
    return (y, rstd) if mean is None else (y, mean, rstd)


def _plain_norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][..., None]
    xh = (x - s["mean"][..., None] if s["mean"] is not None else x) * rstd
    g = dy * _rows(s["weight"])
    dx = g - xh * (g * xh).mean(-1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - g.mean(-1, keepdim=True)
    over = (1, 2) if s["c"]["per_batch"] else (0, 1, 2)
    dweight = (dy * xh).sum(over)
    got = ((dx * rstd).to(s["x"].dtype), dweight)
    return got + (dy.sum(over),) if s["c"]["bias"] else got


def _plain_rope(s):
    c = s["c"]
    ang = s["pos"].double()[..., s["axis_dev"]] * s["freq_dev"]  # [B or 1, N, R/2]
    cos, sin = ((f(ang) * s["mscale"]).float()[:, :, None] for f in (torch.cos, torch.sin))
    sin = -sin if c["inverse"] else sin
    x = s["x"].float()
    r, rest = x[..., :c["R"]], x[..., c["R"]:]
    if c["half"]:
        a, b = r[..., :c["R"] // 2], r[..., c["R"] // 2:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((r, rest), -1).to(s["x"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "attn_bwd":
        B, Nq, Nkv, H, D, valid = c["B"], c["Nq"], c["Nkv"], c["H"], c["D"], c["valid"]
        pairs = Nq * valid
        if c["frame"]:  # own frame and the first frame, at most; the rows past the mask attend every key
            pairs = valid * min(valid, 2 * c["frame"]) + (Nq - valid) * valid
        rows_q, rows_k = B * H * Nq, B * H * valid
        n_bytes = 2 * D * (4 * rows_q + 2 * rows_k) + 2 * D * 2 * B * H * Nkv + 4 * rows_q  # q out dout dq, k v, dk dv, lse
        if c["frame"]:
            n_bytes += valid * valid // 8
        return {"bytes": n_bytes, "flops": 10 * B * H * D * pairs}
    e = 4 if c["fp32"] else 2
    if c["op"] == "norm":
        rows, C = c["B"] * c["N"] * c["H"], c["C"]
        params = (c["B"] if c["per_batch"] else 1) * C * 4
        stats = rows * (8 if c["center"] else 4)
        if c["backward"]:
            return {"bytes": 3 * e * rows * C + stats + params * (3 if c["bias"] else 2), "flops": 12 * rows * C}
        return {"bytes": 2 * e * rows * C + stats + params * (2 if c["bias"] else 1), "flops": 7 * rows * C}
    rows = c["B"] * c["N"]
    return {"bytes": 2 * e * rows * c["H"] * c["D"] + 4 * c["axes"] * (rows if c["axes"] == 1 else c["N"]),
            "flops": 3 * rows * c["H"] * c["R"]}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn_bwd": _exact_attn, "norm": _exact_norm, "rope": _exact_rope}[case["op"]](s)


def _exact_attn(s):
    """sum_j L(p) by the chain rule, one head at a time: P_ij = exp(scale q_i.k_j - lse_i)."""
    c, n, scale = s["c"], s["c"]["valid"], s["scale"]
    if s["bits"] is not None:
        allow = torch.ones((c["Nq"], n), dtype=torch.float64, device=DEV)
        word = s["bits"][0].to(torch.int64) & 0xFFFFFFFF
        for bit in range(32):
            cols = torch.arange(bit, n, 32, device=DEV)
            allow[:n, cols] = ((word[:, :len(cols)] >> bit) & 1).double()
    grads = [torch.zeros(s[x].shape, dtype=torch.float64, device=DEV) for x in ("q", "k", "v")]
    for b in range(c["B"]):
        for h in range(c["H"]):
            q, o, go = (s[x][b, :, h].double() for x in ("q", "out", "dout"))
            k, v = (s[x][b, :n, h].double() for x in ("k", "v"))
            prob = torch.exp(torch.addmm(-s["lse"][b, h].double()[:, None], q, k.t(), alpha=scale))
            if s["bits"] is not None:
                prob = prob * allow
            grads[2][b, :n, h] = torch.mm(prob.t(), go)
            gs = scale * prob * (torch.mm(go, v.t()) - torch.einsum("id,id->i", go, o)[:, None])
            grads[0][b, :, h] = torch.mm(gs, k)
            grads[1][b, :n, h] = torch.mm(gs.t(), q)
    return tuple(grads)


def _exact_norm(s):
    c = s["c"]
    x = s["x"].double()
    C = c["C"]
    w = s["weight"].double()
    w = w.view(c["B"], 1, 1, C) if c["per_batch"] else w.view(1, 1, 1, C)
    if not c["backward"]:
        mu = x.sum(-1, keepdim=True) / C if c["center"] else torch.zeros_like(x[..., :1])
        rstd = 1 / torch.sqrt(((x - mu) ** 2).sum(-1, keepdim=True) / C + s["eps"])
        y = (x - mu) * rstd * w
        if s["bias"] is not None:
            b = s["bias"].double()
            y = y + (b.view(c["B"], 1, 1, C) if c["per_batch"] else b)
        return (y, mu[..., 0], rstd[..., 0]) if c["center"] else (y, rstd[..., 0])
    rstd, go = s["rstd"].double().unsqueeze(-1), s["dy"].double()
    z = rstd * (x - s["mean"].double().unsqueeze(-1)) if c["center"] else rstd * x
    g = go * w
    gx = rstd * (g - z * torch.einsum("bnhc,bnhc->bnh", g, z)[..., None] / C)
    if c["center"]:
        gx = gx - rstd * g.sum(-1, keepdim=True) / C
    gw = torch.einsum("bnhc,bnhc->bc", go, z)
    gb = torch.einsum("bnhc->bc", go)
    if not c["per_batch"]:
        gw, gb = gw.sum(0), gb.sum(0)
    return (gx, gw, gb) if c["bias"] else (gx, gw)


def _exact_rope(s):
    """Each pair as a complex number, turned by exp(+-i angle)."""
    c, R = s["c"], s["c"]["R"]
    y = s["x"].double().clone()
    turn = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device=DEV),
                       (-1.0 if c["inverse"] else 1.0) * s["pos"].double()[..., s["axis_dev"]] * s["freq_dev"])[:, :, None]
    first, second = (slice(0, R // 2), slice(R // 2, R)) if c["half"] else (slice(0, R, 2), slice(1, R, 2))
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y
