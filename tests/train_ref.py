"""64-bit references of the training operators and the error bounds their
kernels' arithmetic allows (torch, any device).

Roundings counted: half a step of the type, 2^-8 of the value for bf16, 2^-24 for
fp32.  EPS32 terms are chains of fp32 operations; the tensor cores' fp32
accumulation is given a whole step (2^-23) an addition.
"""
import math

import torch

BF16 = 2.0 ** -8
EPS32 = 2.0 ** -23


def attn_forward(q, k, v, scale, allow):
    """fp64 O [B, Nq, H, D] and LSE [B, H, Nq] over the keys `allow` [B, 1, Nq, Nkv] permits."""
    q, k, v = (t.double().transpose(1, 2) for t in (q, k, v))
    s = (q @ k.transpose(-1, -2)) * scale
    s = s.masked_fill(~allow, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None].masked_fill(torch.isinf(lse)[..., None], 0.0))
    return (p @ v).transpose(1, 2), lse


def attn_bwd(q, k, v, out, lse, dout, scale, allow, dlse=None, grad_bf16=True):
    """(dq, dk, dv) in fp64 from the same inputs the kernel gets, and the bound on
    each element's error.

    P and dS enter the products rounded to bf16 (half a step each), so
      |err dV| <= (2^-8 + e_p) sum_i P |dO|,
      |err dQ| <= scale ((2^-8 + e_p) sum_j |dS| |K| + sum_j P e_d |K|)   (dK alike),
    e_p: relative error of P from fp32 scores (D additions of |q k| at most, the
    product with scale log2 e and the LSE's, each carried into the exponent) and
    the exponential (2^-22); e_d: error of dP - delta from two fp32 sums of D
    terms.  Sums over n terms in fp32 add n steps of sum |terms|; the result is
    rounded once (2^-8 of itself in bf16)."""
    B, Nq, H, D = q.shape
    Nkv = k.shape[1]
    q, k, v, o, go = (t.double().transpose(1, 2) for t in (q, k, v, out, dout))
    lse = lse.double()
    s = (q @ k.transpose(-1, -2)) * scale
    keep = allow & ~torch.isinf(lse)[..., None]
    p = torch.exp((s - lse[..., None]).masked_fill(~keep, -math.inf))
    dp = go @ v.transpose(-1, -2)
    delta = (go * o).sum(-1, keepdim=True)
    if dlse is not None:
        delta = delta - dlse.double()[..., None]
    ds = p * (dp - delta)
    dq, dk, dv = (ds @ k) * scale, (ds.transpose(-1, -2) @ q) * scale, p.transpose(-1, -2) @ go

    sabs = ((q.abs() @ k.abs().transpose(-1, -2)) * scale).masked_fill(~keep, 0.0)
    labs = lse.masked_fill(torch.isinf(lse), 0.0).abs()[..., None]
    e_p = EPS32 * (sabs * (D + 2) + 3 * labs + 8)
    e_d = EPS32 * (D + 2) * (go.abs() @ v.abs().transpose(-1, -2) + (go * o).abs().sum(-1, keepdim=True))
    if dlse is not None:
        e_d = e_d + EPS32 * dlse.double().abs()[..., None]
    # The exponential and fp32 / bf16 products flush results below 2^-126 to zero:
    # P is off by up to 2^-126 besides, twice with its own rounding, and so is dS
    # by that times |dP - delta| and by 2^-126 itself.
    tiny = 2.0 ** -125
    pe = p * (BF16 + e_p) + tiny
    dse = ds.abs() * (BF16 + 2 * e_p + 4 * EPS32) + p * e_d + tiny * ((dp - delta).abs() + 1)
    rnd = BF16 if grad_bf16 else EPS32
    bq = scale * (dse @ k.abs() + EPS32 * Nkv * (ds.abs() @ k.abs())) + rnd * dq.abs()
    bk = scale * (dse.transpose(-1, -2) @ q.abs() + EPS32 * Nq * (ds.abs().transpose(-1, -2) @ q.abs())) + rnd * dk.abs()
    bv = pe.transpose(-1, -2) @ go.abs() + EPS32 * Nq * (p.transpose(-1, -2) @ go.abs()) + rnd * dv.abs()
    # the bounds' own roundings (a rounded value is rounded again): (1 + 2^-8)^2, and the result's own flush
    return [(g.transpose(1, 2), 1.01 * b.transpose(1, 2) + tiny) for g, b in ((dq, bq), (dk, bk), (dv, bv))]


def layer_norm(x, weight, bias, eps, center):
    """fp64 (y, mean, rstd, bound of y without its own rounding) of [B, N, H, C].

    A mean is a chain of at most 64 fp32 additions (16 channels a thread, 5
    shuffles, 16 warps), so its error is below 64 * 2^-24 mean |x|; the
    deviation, rstd (from a sum alike), weight and bias add a few steps more:
    128 * 2^-24 of ((|x| + mean |x|) rstd |w| + |b|) covers them."""
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros_like(w) if bias is None else bias.double()
    if w.dim() == 2:
        w = w[:, None, None]
    if b.dim() == 2:
        b = b[:, None, None]
    mean = x.mean(-1, keepdim=True) if center else torch.zeros_like(x[..., :1])
    rstd = ((x - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    y = (x - mean) * rstd * w + b
    bound = 64 * EPS32 * ((x.abs() + x.abs().mean(-1, keepdim=True)) * rstd * w.abs() + b.abs())
    return y, mean[..., 0], rstd[..., 0], bound


def layer_norm_bwd(dy, x, mean, rstd, weight, chain):
    """fp64 (dx, dweight, dbias) per parameter set and their bounds; `chain`: the
    longest chain of fp32 additions of the sums over rows.  dx: two means of C
    terms (chains of at most 64) and some ten operations more."""
    B, C = x.shape[0], x.shape[-1]
    x, dy, r = x.double(), dy.double(), rstd.double()[..., None]
    mu = 0.0 if mean is None else mean.double()[..., None]
    w = torch.ones(C, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    per_batch = w.dim() == 2
    if per_batch:
        w = w[:, None, None]
    xh = (x - mu) * r
    xa = (x.abs() + (mu.abs() if mean is not None else 0.0)) * r       # |xh| before cancellation
    g = dy * w
    c2 = (g * xh).mean(-1, keepdim=True)
    c1 = g.mean(-1, keepdim=True) if mean is not None else torch.zeros_like(c2)
    dx = r * (g - c1 - xh * c2)
    bx = 64 * EPS32 * r * (g.abs() + g.abs().mean(-1, keepdim=True) + 2 * xa * (g.abs() * xa).mean(-1, keepdim=True))
    over = (1, 2) if per_batch else (0, 1, 2)
    dw, db = (dy * xh).sum(over), dy.sum(over)
    bw, bb = EPS32 * (chain + 4) * (dy.abs() * xa).sum(over), EPS32 * chain * dy.abs().sum(over)
    return (dx, bx), (dw, bw), (db, bb)


def rope(x, inv_freq, pos, pairs, half, mscale, inverse):
    """fp64 rotation of [B, N, H, D] and its bound without y's rounding: the
    angle, an integer of 2^-32 turns, becomes an fp32 number of at most an eighth
    turn (2^-25 of it) times 2 pi (another), and the polynomials' results are good
    to a few steps, then four operations: 2^-20 (|a| + |b|) mscale."""
    R = 2 * inv_freq.numel()
    axis = torch.cat([torch.full((n,), i, dtype=torch.long) for i, n in enumerate(pairs)]).to(x.device)
    # the angle modulo a turn in exact integer arithmetic over Python ints would be slow; fp64 is exact to
    # 2^-53 |angle|, below 2^-23 for |angle| < 2^30
    ang = pos.double()[..., axis] * inv_freq.to(x.device)
    c, s = torch.cos(ang)[:, :, None] * mscale, torch.sin(ang)[:, :, None] * mscale
    s = -s if inverse else s
    y = x.double().clone()
    ia = torch.arange(R // 2, device=x.device) if half else torch.arange(0, R, 2, device=x.device)
    ib = ia + (R // 2 if half else 1)
    a, b = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    bound = torch.zeros_like(y)
    bound[..., ia] = bound[..., ib] = 2.0 ** -20 * (a.abs() + b.abs()) * abs(mscale)
    return y, bound


def check(got, ref, bound, what=""):
    """Every element within its bound; NaN never passes."""
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = tuple(int(t) for t in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {float(got[i]):.9g}, "
                             f"want {float(ref[i]):.9g} +- {float(bound[i]):.3g}")
