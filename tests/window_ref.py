"""64-bit references of windowed attention and the paged cache, and the error bounds
their kernels' arithmetic allows (torch, any device; roundings as in train_ref)."""
import math

import torch

import train_ref as ref
from train_ref import BF16, EPS32


def sees(positions, n_keys, left, right, sinks, frame, key_valid_len):
    """[queries, keys] by the frames' numbers, from the definition."""
    j = torch.arange(n_keys, device=positions.device)
    fp = torch.div(positions, frame, rounding_mode="floor")[:, None]
    fj = torch.div(j, frame, rounding_mode="floor")[None, :]
    ok = (j < key_valid_len)[None, :].expand(len(positions), n_keys).clone()
    if left is not None:
        ok &= (fj >= fp - left) | (j < sinks)[None, :]
    if right is not None:
        ok &= fj <= fp + right
    return ok


def shared(t, H):
    """K or V [B, N, Hkv, D] as every query head sees it."""
    return t.repeat_interleave(H // t.shape[2], 2)


def forward(q, k, v, scale, allow, out_bf16):
    """fp64 (O [B, N, H, D], its bound), (LSE [B, H, N], its bound); rows without a key
    0 and -inf.  allow [B or 1, 1, N, Nkv]; k and v with q's heads.

    P = 2^(s scale log2 e - m) of the fp32 score: D additions, the products' and the
    exponent's roundings, each carried into it, and the exponential's own (2^-22);
    P enters the product rounded to bf16 (half a step), its sum does not.  Sums of n
    terms in fp32 add n steps of sum |terms|; joining pieces a few more."""
    D, n = q.shape[-1], k.shape[1]
    q, k, v = (t.double().transpose(1, 2) for t in (q, k, v))
    s = ((q @ k.transpose(-1, -2)) * scale).masked_fill(~allow, -math.inf)
    lse = torch.logsumexp(s, -1)
    some = ~torch.isinf(lse)
    p = torch.exp(s - lse.masked_fill(~some, 0.0)[..., None])
    o = p @ v
    size = ((q.abs() @ k.abs().transpose(-1, -2)) * scale).masked_fill(~allow, 0.0)
    top = torch.cat((size, size.new_zeros((*size.shape[:-1], 1))), -1).amax(-1, keepdim=True)   # (no keys: 0)
    e = EPS32 * (size * (D + 2) + 3 * top + 16)
    el = (p * e).sum(-1) + EPS32 * (n + 16)
    bo = (p * (BF16 + e)) @ v.abs() + el[..., None] * (p @ v.abs()) + EPS32 * n * (p @ v.abs()) + (BF16 if out_bf16 else EPS32) * o.abs()
    bl = (el + 4 * EPS32 * (lse.abs() + top[..., 0])).masked_fill(~some, 0.0)
    return (o.transpose(1, 2), 1.01 * bo.transpose(1, 2) + 2.0 ** -120), (lse, 1.01 * bl)


def check_forward(out, lse, want, rows=None):
    """rows [B, N]: the rows to look at (all of them when None)."""
    (o, bo), (l, bl) = want
    B, N = o.shape[:2]
    rows = torch.ones((B, N), dtype=torch.bool, device=o.device) if rows is None else rows
    ref.check(out[rows], o[rows], bo[rows], "out")
    got, l, bl = lse.transpose(1, 2)[rows], l.transpose(1, 2)[rows], bl.transpose(1, 2)[rows]
    none = torch.isinf(l)
    assert torch.equal(got == -math.inf, none), "rows without a key"
    ref.check(got[~none], l[~none], bl[~none], "lse")


def backward(q, k, v, out, lse, dout, scale, allow, dlse=None, grad_bf16=True):
    """(dq, dk, dv) with their bounds, dk and dv summed over the heads that share them:
    the bounds of the heads' parts, and the longer sum's roundings."""
    B, Nq, H, D = q.shape
    Nkv, Hkv = k.shape[1:3]
    (dq, bq), (dk, bk), (dv, bv) = ref.attn_bwd(q, shared(k, H), shared(v, H), out, lse, dout, scale, allow, dlse, grad_bf16)
    group = H // Hkv

    def summed(t):
        return t.reshape(B, Nkv, Hkv, group, D).sum(3)
    long = EPS32 * Nq * (group - 1)
    s = ((q.double().transpose(1, 2) @ shared(k, H).double().permute(0, 2, 3, 1)) * scale)
    p = torch.exp((s - lse.double()[..., None]).masked_fill(~allow | torch.isinf(lse)[..., None], -math.inf))
    dp = (dout.double().transpose(1, 2) @ shared(v, H).double().permute(0, 2, 3, 1)).abs() + 2 * (dout.double() * out.double()).abs().sum(-1).transpose(1, 2)[..., None]
    if dlse is not None:
        dp = dp + dlse.double().abs()[..., None]
    extra_k = summed(((p * dp).transpose(-1, -2) @ q.double().abs().transpose(1, 2)).transpose(1, 2)) * (scale * long)
    extra_v = summed((p.transpose(-1, -2) @ dout.double().abs().transpose(1, 2)).transpose(1, 2)) * long
    return (dq, bq), (summed(dk), summed(bk) + extra_k), (summed(dv), summed(bv) + extra_v)


def gathered(cache, table, n):
    """Keys [n, Hkv, D] of one sequence and which of them its table has a page for."""
    pages, page = cache.shape[:2]
    j = torch.arange(n, device=cache.device)
    index = table.long()[j // page] if n else j
    there = (index >= 0) & (index < pages)
    return cache[index.clamp(0, max(pages - 1, 0)), j % page] if n else cache[:0, 0], there
