"""Attention of streaming (autoregressive) video models, trained and served: cases, plain forms and exact values.

  window, forward    O and LSE of queries that see a sliding window of frames (or tokens) and a few first tokens
                     that stay visible (sinks); heads may share K and V
  window, backward   dq, dk, dv of the same, the probabilities recomputed from lse; dk and dv are sums over the
                     query heads that share them
  paged append       K and V of new tokens written into the pages of a cache
  paged attention    a chunk of new tokens, from one to a whole frame or prompt, over the paged cache

A query at position p, in frame f = floor(p / frame), sees the keys j < kv_len with
    j < (f + 1 + right) * frame  and  (j >= (f - left) * frame or j < sinks);
left or right None: no bound on that side.

`run` computes the plain form with elementary torch operations in 32 bits, or, with `own` set, makes the calls
a user makes of the library.
"""
import math

import torch

own = False
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the `tiny` workload with a window of 256 tokens and four sinks: launches and latency count
        _window("window_fwd_tiny", B=1, N=1024, H=2, Hkv=2, D=64, left=255, sinks=4),
        # the LTX-2-shaped padded sequence made causal by frames: 16 frames of 32 x 48 tokens, each seeing three
        # frames back, the first frame always visible, views of the fused projection
        _window("window_fwd_frames", B=1, N=24576, H=32, Hkv=32, D=128, left=3, sinks=1536, frame=1536, valid=24200, fused=True),
        # the Cosmos-shaped sequence with a token window, four query heads to a K/V head
        _window("window_fwd_tokens", B=1, N=44160, H=16, Hkv=4, D=128, left=2047, sinks=16),
        # backward of the first: what a small step pays
        _window("window_bwd_tiny", B=1, N=1024, H=2, Hkv=2, D=64, left=255, sinks=4, backward=True),
        # a quarter of the LTX-2-shaped sequence and of its heads, frames of 384, backward
        _window("window_bwd_frames", B=1, N=6144, H=8, Hkv=8, D=128, left=3, sinks=384, frame=384, valid=6050, fused=True,
                backward=True),
        # causal over a quarter of the Cosmos-shaped sequence, gradients of K and V summed over four heads
        _window("window_bwd_causal", B=1, N=11040, H=16, Hkv=4, D=128, left=None, backward=True),
        # one new token for each of 48 sequences
        _append("append_token", B=48, T=1, Hkv=8, D=128, page=64, pages=64, ragged=False),
        # a frame of new tokens for four streams
        _append("append_frame", B=4, T=1536, Hkv=32, D=128, page=128, pages=48, ragged=True),
        # one new token for one short sequence: the smallest call
        _paged("paged_token_one", B=1, T=1, H=16, Hkv=16, D=64, page=16, longest=1000),
        # one new token for each of 48 sequences of all lengths, four query heads to a K/V head: bound by the cache
        _paged("paged_token_batch", B=48, T=1, H=32, Hkv=8, D=128, page=64, longest=16384),
        # the next frame of two streams over their windows and their first frames
        _paged("paged_frame", B=2, T=1536, H=32, Hkv=32, D=128, page=128, longest=24576, left=6, sinks=1536, frame=1536,
               whole_frames=True),
        # ragged prompt chunks, causal, with pages that end inside a tile and five query heads to a K/V head
        _paged("paged_chunk", B=6, T=500, H=40, Hkv=8, D=128, page=48, longest=9000, ragged=True),
    ]


def _window(name, *, B, N, H, Hkv, D, left, sinks=0, frame=1, right=0, valid=-1, offset=0, Nkv=-1, fused=False, backward=False):
    Nkv = N if Nkv < 0 else Nkv
    return {"name": name, "op": "bwd" if backward else "fwd", "B": B, "N": N, "Nkv": Nkv, "H": H, "Hkv": Hkv, "D": D,
            "left": left, "right": right, "sinks": sinks, "frame": frame, "valid": Nkv if valid < 0 else valid,
            "offset": offset, "fused": fused}


def _append(name, *, B, T, Hkv, D, page, pages, ragged):
    return {"name": name, "op": "append", "B": B, "T": T, "Hkv": Hkv, "D": D, "page": page, "pages": pages, "ragged": ragged}


def _paged(name, *, B, T, H, Hkv, D, page, longest, left=None, right=0, sinks=0, frame=1, ragged=False, whole_frames=False):
    return {"name": name, "op": "paged", "B": B, "T": T, "H": H, "Hkv": Hkv, "D": D, "page": page, "longest": longest,
            "left": left, "right": right, "sinks": sinks, "frame": frame, "ragged": ragged, "whole_frames": whole_frames}


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("fwd", "fwd", "bwd", "bwd", "append", "paged", "paged", "paged"))
    D = rng.choice((64, 128))
    Hkv = _spread(rng, 1, 16)
    H = Hkv * rng.choice((1, 1, 2, 3, 4, 5, 8))
    frame = rng.choice((1, 1, _spread(rng, 2, 2000)))
    if op == "bwd" and frame > 1:
        frame = max(frame, 16)
    # (a few keys' gradients are differences of like values)
    left = rng.choice((None, _spread(rng, 16 if op == "bwd" else 1, 6000) if frame == 1 else rng.randint(0, 6)))
    sinks = rng.choice((0, _spread(rng, 1, 1600)))
    if op in ("fwd", "bwd"):
        N = _spread(rng, 16 if op == "bwd" else 1, 16384)
        budget = (1 << 32) if op == "fwd" else (1 << 31)  # (query, key) pairs of all heads
        H, Hkv = (H, Hkv) if N * N * H <= budget else (max(1, budget // (N * N)),) * 2
        B = rng.randint(1, max(1, min(3, budget // (N * N * H))))
        cross = rng.random() < 0.3  # the last rows of a longer sequence
        Nkv = N + _spread(rng, 1, 2000) if cross else N
        padded = left is None or sinks > 0  # (a row past the valid keys still sees some)
        c = _window("", B=B, N=N, H=H, Hkv=Hkv, D=D, left=left, sinks=sinks, frame=frame, right=rng.choice((0, 0, 0, 1, None)),
                    valid=rng.randint(Nkv - Nkv // 8, Nkv) if padded else Nkv, offset=Nkv - N, Nkv=Nkv,
                    fused=not cross and H == Hkv and rng.random() < 0.5, backward=op == "bwd")
    else:
        page = rng.choice((16, 32, 48, 64, 80, 128, 256))
        B = _spread(rng, 1, 48)
        T = rng.choice((1, 1, rng.randint(2, 8), _spread(rng, 8, 1600)))
        B = max(1, min(B, 6144 // T)) if T > 1 else B
        if op == "append":
            c = _append("", B=B, T=T, Hkv=Hkv, D=D, page=page, pages=(T + _spread(rng, 1, 2000)) // page + 2, ragged=rng.random() < 0.6)
        else:
            longest = T + _spread(rng, 1, 20_000)
            longest = min(longest, max(T, (1 << 33) // (B * T * H)))
            c = _paged("", B=B, T=T, H=H, Hkv=Hkv, D=D, page=page, longest=longest, left=left, sinks=sinks, frame=frame,
                       right=rng.choice((0, 0, 0, 1, None)), ragged=rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _normal(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    return {"fwd": _prepare_window, "bwd": _prepare_window, "append": _prepare_paged, "paged": _prepare_paged}[case["op"]](dict(case), gen)


def _prepare_window(c, gen):
    B, N, Nkv, H, Hkv, D = c["B"], c["N"], c["Nkv"], c["H"], c["Hkv"], c["D"]
    if c["fused"]:
        qkv = _normal((B, N, 3, H, D), gen)
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    else:
        q, k, v = _normal((B, N, H, D), gen, 1.5), _normal((B, Nkv, Hkv, D), gen), _normal((B, Nkv, Hkv, D), gen)
    s = {"c": c, "q": q, "k": k, "v": v, "scale": D ** -0.5}
    if c["op"] == "bwd":  # with the forward pass' results, as the program has them
        s["dout"] = _normal((B, N, H, D), gen, 0.25)
        s["out"], s["lse"] = _plain_window_fwd(s)
    return s


def _lengths(c, gen):
    """New tokens and keys (the new ones among them) of each sequence."""
    B, T = c["B"], c["T"]
    new = torch.full((B,), T, dtype=torch.int64, device=DEV)
    if c["ragged"]:
        new = torch.randint(T // 2, T + 1, (B,), generator=gen, device=DEV).clamp_(min=1)
    longest = c["longest"] if c["op"] == "paged" else c["page"] * c["pages"]
    if c.get("whole_frames"):
        lens = torch.randint(2, longest // T + 1, (B,), generator=gen, device=DEV) * T
        return new, lens
    old = torch.rand((B,), generator=gen, device=DEV) * (longest - new).clamp_(min=0)
    old[0] = longest - new[0]  # one of them fills the range
    return new, new + old.long()


def _prepare_paged(c, gen):
    B, T, Hkv, D, page = c["B"], c["T"], c["Hkv"], c["D"], c["page"]
    new, lens = _lengths(c, gen)
    width = -(-int(lens.max()) // page)
    total = B * width + 3
    table = torch.randperm(total, generator=gen, device=DEV)[:B * width].view(B, width)
    cache = _normal((total, 2, page, Hkv, D), gen)  # one allocation, K and V of a page beside each other
    s = {"c": c, "k_cache": cache[:, 0], "v_cache": cache[:, 1], "table": table.to(torch.int32), "kv_lens": lens.to(torch.int32),
         "new": new.to(torch.int32), "new_list": new.tolist(), "lens_list": lens.tolist(), "scale": D ** -0.5}
    if c["op"] == "append":
        qkv = _normal((B, T, 3, Hkv, D), gen)
        s["k"], s["v"] = qkv[:, :, 1], qkv[:, :, 2]
        return s
    s["q"] = _normal((B, T, c["H"], D), gen, 1.5)
    # rows behind a sequence's new tokens stay as they are
    s["out"] = torch.zeros((B, T, c["H"], D), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((B, c["H"], T), device=DEV)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["c"]["op"]
    if own:
        return _own(state, op)
    return {"fwd": _plain_window_fwd, "bwd": _plain_window_bwd, "append": _plain_append, "paged": _plain_paged}[op](state)


def _own(s, op):
    import dit_long_sequence_gb300 as dl
    c = s["c"]
    if op == "append":
        dl.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], new_lens=s["new"] if c["ragged"] else None)
        return s["k_cache"], s["v_cache"]
    window = {n: c[n] for n in ("left", "right", "sinks", "frame")}
    if op == "paged":
        return dl.attn_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], q_lens=s["new"] if c["ragged"] else None,
                                 scale=s["scale"], out=s["out"], lse=s["lse"], **window)
    window.update(offset=c["offset"], key_valid_len=c["valid"], scale=s["scale"])
    if op == "fwd":
        return dl.attn_fwd_window(s["q"], s["k"], s["v"], out_dtype=torch.bfloat16, **window)
    return dl.attn_bwd_window(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], **window)


def _bounds(c, pos, valid):
    """First key past the sinks and end of the keys of queries at `pos`."""
    start = torch.div(pos, c["frame"], rounding_mode="floor") * c["frame"]
    hi = torch.full_like(pos, valid) if c["right"] is None else (start + (c["right"] + 1) * c["frame"]).clamp(0, valid)
    lo = torch.zeros_like(pos) if c["left"] is None else (start - c["left"] * c["frame"]).clamp(min=0)
    return lo, hi


def _blocks(c, first, n, valid, rows=2048):
    """Blocks of rows, the keys that some row of a block sees, and which row sees which."""
    for r in range(0, n, rows):
        m = min(rows, n - r)
        pos = first + r + torch.arange(m, device=DEV)
        lo, hi = _bounds(c, pos, valid)
        ends = torch.stack((lo[0], hi[-1])).tolist()
        top = min(c["sinks"], ends[1], ends[0])
        keys = torch.cat((torch.arange(0, top, device=DEV), torch.arange(ends[0], max(ends[0], ends[1]), device=DEV)))
        hidden = (keys >= hi[:, None]) | ((keys < lo[:, None]) & (keys >= c["sinks"]))
        yield slice(r, r + m), keys, hidden


def _scores(q, k, hidden, scale):
    """[Hkv, group, rows, keys] scores of q [rows, H, D] and k [keys, Hkv, D], -inf where hidden."""
    rows, H, D = q.shape
    g = q.float().view(rows, k.shape[1], -1, D).permute(1, 2, 0, 3)
    x = (g.reshape(k.shape[1], -1, D) @ k.float().permute(1, 2, 0)).view(k.shape[1], -1, rows, k.shape[0])
    return x.mul_(scale).masked_fill_(hidden, -math.inf)


def _attend(x, v):
    """Softmax of scores and the sum of v [keys, Hkv, D]: [rows, H, D] and the LSE [H, rows]."""
    top = x.amax(-1, keepdim=True).clamp_(min=-3e38) if x.shape[-1] else x.new_full((*x.shape[:-1], 1), -3e38)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(1, 2) @ v.float().transpose(0, 1)).view(*p.shape[:-1], -1) / total.clamp(min=1e-37)
    lse = torch.where(total > 0, top + total.log(), -math.inf)
    return o.permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16), lse.flatten(0, 1)[..., 0]


def _plain_window_fwd(s):
    c = s["c"]
    out = torch.empty((c["B"], c["N"], c["H"], c["D"]), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((c["B"], c["H"], c["N"]), device=DEV)
    for rows, keys, hidden in _blocks(c, c["offset"], c["N"], c["valid"]):
        for b in range(c["B"]):
            out[b, rows], lse[b, :, rows] = _attend(_scores(s["q"][b, rows], s["k"][b, keys], hidden, s["scale"]), s["v"][b, keys])
    return out, lse


def _plain_window_bwd(s):
    c, scale = s["c"], s["scale"]
    Hkv, D = c["Hkv"], c["D"]
    dq = torch.empty((c["B"], c["N"], c["H"], D), dtype=torch.bfloat16, device=DEV)
    dk, dv = (torch.zeros((c["B"], c["Nkv"], Hkv, D), device=DEV) for _ in range(2))

    def by_group(t):  # [rows, H, D] -> [Hkv, group * rows, D]
        return t.float().view(t.shape[0], Hkv, -1, D).permute(1, 2, 0, 3).flatten(1, 2)
    for rows, keys, hidden in _blocks(c, c["offset"], c["N"], c["valid"]):
        for b in range(c["B"]):
            lse = s["lse"][b, :, rows]
            x = _scores(s["q"][b, rows], s["k"][b, keys], hidden, scale)
            p = x.sub_(torch.where(lse.isinf(), 0.0, lse).view(Hkv, -1, lse.shape[1], 1)).exp_().flatten(1, 2)
            q, k, v, do, o = by_group(s["q"][b, rows]), s["k"][b, keys].float(), s["v"][b, keys].float(), \
                by_group(s["dout"][b, rows]), by_group(s["out"][b, rows])
            dv[b, keys] += (p.transpose(1, 2) @ do).transpose(0, 1)
            ds = (do @ v.permute(1, 2, 0)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
            g = (ds @ k.transpose(0, 1)) * scale
            dq[b, rows] = g.view(Hkv, -1, lse.shape[1], D).permute(2, 0, 1, 3).flatten(1, 2).to(torch.bfloat16)
            dk[b, keys] += (ds.transpose(1, 2) @ q).transpose(0, 1) * scale
    return dq, dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def _plain_append(s):
    c = s["c"]
    t = torch.arange(c["T"], device=DEV)
    pos = (s["kv_lens"] - s["new"])[:, None].long() + t
    b, i = (t < s["new"][:, None]).nonzero(as_tuple=True)
    at = pos[b, i]
    where = s["table"][b, at // c["page"]].long(), at % c["page"]
    s["k_cache"][where] = s["k"][b, i]
    s["v_cache"][where] = s["v"][b, i]
    return s["k_cache"], s["v_cache"]


def _plain_paged(s):
    c = s["c"]
    for b in range(c["B"]):
        n, length = s["new_list"][b], s["lens_list"][b]
        for rows, keys, hidden in _blocks(c, length - n, n, length):
            where = s["table"][b][keys // c["page"]].long(), keys % c["page"]
            x = _scores(s["q"][b, rows], s["k_cache"][where], hidden, s["scale"])
            s["out"][b, rows], s["lse"][b, :, rows] = _attend(x, s["v_cache"][where])
    return s["out"], s["lse"]


# ---------------------------------------------------------------- what a pass cannot do without

def _pairs(c, first, n, valid):
    """(query, key) pairs of n rows from position `first`, and the keys that some row sees."""
    total, F = 0, c["frame"]
    f, last, seen = first // F, (first + n - 1) // F, 0
    while f <= last:
        count = min(first + n, (f + 1) * F) - max(first, f * F)
        hi = valid if c["right"] is None else min(max((f + 1 + c["right"]) * F, 0), valid)
        lo = 0 if c["left"] is None else max(0, (f - c["left"]) * F)
        total += count * (max(0, hi - lo) + min(c["sinks"], lo, hi))
        if f == first // F:
            low = lo
        seen = max(0, hi - low) + min(c["sinks"], low, hi)
        f += 1
    return total, seen


def work(case):
    c = case
    if c["op"] == "append":
        tokens = c["B"] * c["T"] * (0.75 if c["ragged"] else 1.0)
        return {"bytes": int(4 * 2 * tokens * c["Hkv"] * c["D"]) + 12 * c["B"], "flops": 0}
    row = 2 * c["D"]
    if c["op"] == "paged":  # lengths are drawn in prepare: spread evenly, the first at its longest
        mean_new = c["T"] * 0.75 if c["ragged"] else c["T"]
        n_bytes = flops = 0
        for i in range(c["B"]):
            n = max(1, round(mean_new))
            length = c["longest"] if i == 0 else n + (c["longest"] - n) // 2
            if c["whole_frames"]:
                length = (2 + c["longest"] // c["T"]) // 2 * c["T"]
            pairs, seen = _pairs(c, length - n, n, length)
            n_bytes += 2 * row * seen * c["Hkv"] + (2 * row + 4) * n * c["H"]
            flops += 4 * c["D"] * c["H"] * pairs
        return {"bytes": int(n_bytes), "flops": int(flops)}
    pairs, _ = _pairs(c, c["offset"], c["N"], c["valid"])
    rows_q, rows_k = c["B"] * c["H"] * c["N"], c["B"] * c["Hkv"] * c["valid"]
    if c["op"] == "fwd":
        return {"bytes": (2 * row + 4) * rows_q + 2 * row * rows_k, "flops": 4 * c["D"] * c["B"] * c["H"] * pairs}
    return {"bytes": (4 * row + 4) * rows_q + 2 * row * rows_k + 2 * row * c["B"] * c["Hkv"] * c["Nkv"],
            "flops": 10 * c["D"] * c["B"] * c["H"] * pairs}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    return {"fwd": _exact_fwd, "bwd": _exact_bwd, "paged": _exact_paged}[case["op"]](s)


def _sees(c, p, j):
    """Truth table of queries at positions p and keys j, by the frames' numbers."""
    fp, fj = torch.floor(p.double() / c["frame"])[:, None], torch.floor(j.double() / c["frame"])[None, :]
    ok = torch.ones((len(p), len(j)), dtype=torch.bool, device=DEV)
    if c["left"] is not None:
        ok &= (fj >= fp - c["left"]) | (j < c["sinks"])[None, :]
    if c["right"] is not None:
        ok &= fj <= fp + c["right"]
    return ok


def _exact_head(c, q, k, v, first, scale):
    """One head in pieces of rows: (rows, columns some row sees, truth table, scores, their LSE)."""
    j = torch.arange(k.shape[0], device=DEV)
    for r in range(0, q.shape[0], 1024):
        p = first + torch.arange(r, min(r + 1024, q.shape[0]), device=DEV)
        ok = _sees(c, p, j)
        cols = ok.any(0).nonzero()[:, 0]
        ok = ok[:, cols]
        x = torch.where(ok, torch.mm(q[r:r + 1024], k[cols].t()) * scale, -math.inf)
        yield slice(r, r + len(p)), cols, ok, x, torch.logsumexp(x, 1)


def _exact_fwd(s):
    c = s["c"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros((c["B"], c["H"], c["N"]), dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        for h in range(c["H"]):
            k, v = (s[n][b, :c["valid"], h * c["Hkv"] // c["H"]].double() for n in ("k", "v"))
            for rows, cols, ok, x, l in _exact_head(c, s["q"][b, :, h].double(), k, v, c["offset"], s["scale"]):
                lse[b, h, rows] = l
                out[b, rows, h] = torch.mm(torch.exp(x - l[:, None]).nan_to_num(0.0), v[cols])
    return out, lse


def _exact_bwd(s):
    c, scale = s["c"], s["scale"]
    dq, dk, dv = (torch.zeros(s[n].shape, dtype=torch.float64, device=DEV) for n in ("q", "k", "v"))
    for b in range(c["B"]):
        for h in range(c["H"]):
            hk = h * c["Hkv"] // c["H"]
            q, do, o = (s[n][b, :, h].double() for n in ("q", "dout", "out"))
            k, v = (s[n][b, :c["valid"], hk].double() for n in ("k", "v"))
            for rows, cols, ok, x, _ in _exact_head(c, q, k, v, c["offset"], scale):
                prob = torch.where(ok, torch.exp(x - s["lse"][b, h, rows].double()[:, None]), 0.0)
                dv[b, cols, hk] += torch.mm(prob.t(), do[rows])
                gs = scale * prob * (torch.mm(do[rows], v[cols].t()) - torch.einsum("id,id->i", do[rows], o[rows])[:, None])
                dq[b, rows, h] = torch.mm(gs, k[cols])
                dk[b, cols, hk] += torch.mm(gs.t(), q[rows])
    return dq, dk, dv


def _exact_append(s):
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    table = s["table"].tolist()
    page = s["c"]["page"]
    for b, (n, length) in enumerate(zip(s["new_list"], s["lens_list"])):
        at = length - n
        while at < length:  # a page at a time
            slot, room = at % page, min(page - at % page, length - at)
            i = at - (length - n)
            kc[table[b][at // page], slot:slot + room] = s["k"][b, i:i + room].double()
            vc[table[b][at // page], slot:slot + room] = s["v"][b, i:i + room].double()
            at += room
    return kc, vc


def _exact_paged(s):
    c = s["c"]
    out, lse = s["out"].double(), s["lse"].double()
    for b, (n, length) in enumerate(zip(s["new_list"], s["lens_list"])):
        pages = s["table"][b, :-(-length // c["page"])].long()
        for hk in range(c["Hkv"]):
            k, v = (s[t][pages, :, hk].flatten(0, 1)[:length].double() for t in ("k_cache", "v_cache"))
            for h in range(hk * c["H"] // c["Hkv"], (hk + 1) * c["H"] // c["Hkv"]):
                for rows, cols, ok, x, l in _exact_head(c, s["q"][b, :n, h].double(), k, v, length - n, s["scale"]):
                    lse[b, h, rows] = l
                    out[b, rows, h] = torch.mm(torch.exp(x - l[:, None]).nan_to_num(0.0), v[cols])
    return out, lse
