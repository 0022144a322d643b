"""The training operators in a row, as an attention block's step uses them:
modulated layer norm, a fused projection, head-wise RMS norms and rotary
positions on views of it, attention, and the way back into one fused gradient.
Every step is held to its 64-bit formula on the data that reached it, the whole
to the 64-bit gradient; then captured, replayed and run on two streams."""
import math
import types

import pytest
import torch

import train_ref as ref
from dit_long_sequence_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dl():
    import dit_long_sequence_gb300 as m
    return m


@pytest.fixture(autouse=True)
def no_wait_ran_out(dl):
    yield
    rc, info = dl.check_watchdog()
    assert rc == 0, info


class Block:
    """B sequences of N tokens, H heads of D; positions on two axes, the tokens
    from `valid` on are padding, `frame` tokens attend one another (0: all)."""

    def __init__(self, dl, B, N, H, D, valid, frame, half, seed):
        self.dl, self.B, self.N, self.H, self.D, self.valid, self.half = dl, B, N, H, D, valid, half
        g = wl.generator(DEV, seed)
        C = H * D

        def t(*shape, scale=1.0, dtype=BF):
            return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)
        self.x, self.dout = t(B, N, C), t(B, N, H, D, scale=0.5)
        self.w1, self.b1 = 1 + t(B, C, scale=0.2, dtype=torch.float32), t(B, C, scale=0.2, dtype=torch.float32)
        self.proj = t(C, 3 * C, scale=C ** -0.5)
        self.wq, self.wk = (1 + t(D, scale=0.2, dtype=torch.float32) for _ in range(2))
        self.freq = torch.cat([dl.rope_inv_freq(D // 2)[0], dl.rope_inv_freq(D // 2, base=100.0)[0]])
        self.pairs = (D // 4, D // 4)
        i = torch.arange(N, dtype=torch.int32, device=DEV)
        self.pos = torch.stack([i // 16, i % 16], -1)[None]
        self.bits = None
        self.allow = torch.zeros((B, 1, N, N), dtype=torch.bool, device=DEV)
        self.allow[..., :valid] = True
        if frame:
            same = (i[:valid, None] // frame) == (i[None, :valid] // frame)
            self.allow[:, 0, :valid, :valid] &= same
            self.bits = wl.pack_mask_bits(same[None].cpu()).to(DEV)

    def rope_args(self):
        return dict(layout="half" if self.half else "interleaved", axis_pairs=self.pairs)

    def forward(self):
        dl, B, N, H, D = self.dl, self.B, self.N, self.H, self.D
        s = types.SimpleNamespace()
        s.h, s.mean, s.rstd = dl.layer_norm_fwd(self.x, self.w1, self.b1)
        s.qkv = (s.h.view(B * N, H * D) @ self.proj).view(B, N, 3, H, D)
        s.qk = torch.empty((B, N, 2, H, D), dtype=BF, device=DEV)
        _, _, s.rq = dl.layer_norm_fwd(s.qkv[:, :, 0], self.wq, center=False, out=s.qk[:, :, 0])
        _, _, s.rk = dl.layer_norm_fwd(s.qkv[:, :, 1], self.wk, center=False, out=s.qk[:, :, 1])
        s.normed = s.qk.clone()
        both = s.qk.flatten(2, 3)
        dl.rope(both, self.freq, self.pos, out=both, **self.rope_args())
        q, k, v = s.qk[:, :, 0], s.qk[:, :, 1], s.qkv[:, :, 2]
        kw = dict(key_valid_len=self.valid, out_dtype=BF)
        s.o, s.lse = dl.attn_fwd(q, k, v, **kw) if self.bits is None else dl.attn_fwd_masked(q, k, v, self.bits, **kw)
        return s

    def backward(self, s):
        dl, B, N, H, D = self.dl, self.B, self.N, self.H, self.D
        r = types.SimpleNamespace()
        r.dqkv = torch.empty_like(s.qkv)
        dq, dk, dv = (r.dqkv[:, :, i] for i in range(3))
        args = (s.qk[:, :, 0], s.qk[:, :, 1], s.qkv[:, :, 2], s.o, s.lse, self.dout)
        kw = dict(key_valid_len=self.valid, dq=dq, dk=dk, dv=dv)
        if self.bits is None:
            dl.attn_bwd(*args, **kw)
        else:
            dl.attn_bwd_masked(*args, self.bits, **kw)
        r.of_attn = r.dqkv.clone()
        both = r.dqkv[:, :, :2].flatten(2, 3)
        assert both.data_ptr() == r.dqkv.data_ptr()
        dl.rope(both, self.freq, self.pos, inverse=True, out=both, **self.rope_args())
        r.of_rope = r.dqkv.clone()
        _, r.dwq, _ = dl.layer_norm_bwd(dq, s.qkv[:, :, 0], None, s.rq, self.wq, has_bias=False, dx=dq)
        _, r.dwk, _ = dl.layer_norm_bwd(dk, s.qkv[:, :, 1], None, s.rk, self.wk, has_bias=False, dx=dk)
        r.dh = (r.dqkv.view(B * N, 3 * H * D) @ self.proj.t()).view(B, N, H * D)
        r.dx, r.dw1, r.db1 = dl.layer_norm_bwd(r.dh, self.x, s.mean, s.rstd, self.w1)
        return r

    def exact(self):
        """The gradients of sum(O dout) by 64-bit autograd."""
        B, N, H, D = self.B, self.N, self.H, self.D
        leaves = [t.double().requires_grad_() for t in (self.x, self.w1, self.b1, self.wq, self.wk)]
        x, w1, b1, wq, wk = leaves
        h = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + 1e-6).sqrt() * w1[:, None] + b1[:, None]
        q, k, v = (h @ self.proj.double()).view(B, N, 3, H, D).unbind(2)

        def turn(t, w):
            t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
            f = self.freq.to(DEV)
            axis = torch.tensor([0] * self.pairs[0] + [1] * self.pairs[1], device=DEV)
            ang = self.pos[0].double()[:, axis] * f
            c, s = ang.cos()[None, :, None], ang.sin()[None, :, None]
            a, b = (t[..., :D // 2], t[..., D // 2:]) if self.half else (t[..., ::2], t[..., 1::2])
            y = torch.stack([a * c - b * s, a * s + b * c], -1)
            return y.transpose(-1, -2).flatten(-2) if self.half else y.flatten(-2)
        q, k = turn(q, wq), turn(k, wk)
        s = (q.transpose(1, 2) @ k.transpose(1, 2).transpose(-1, -2)) * D ** -0.5
        p = torch.softmax(s.masked_fill(~self.allow, -math.inf), -1)
        o = (p @ v.transpose(1, 2)).transpose(1, 2)
        return torch.autograd.grad((o * self.dout.double()).sum(), leaves)


CASES = [(2, 300, 4, 64, 290, 0, False), (1, 400, 3, 128, 400, 0, True), (2, 333, 2, 128, 320, 100, False), (1, 1100, 2, 64, 1000, 250, True)]


@pytest.mark.parametrize("B,N,H,D,valid,frame,half", CASES)
def test_every_step_on_what_reached_it(dl, B, N, H, D, valid, frame, half):
    m = Block(dl, B, N, H, D, valid, frame, half, 5)
    s = m.forward()
    r = m.backward(s)
    torch.cuda.synchronize()

    def near(got, want, bound, what):
        ref.check(got, want, 1.01 * bound + ref.BF16 * want.abs(), what)
    y, _, _, b = ref.layer_norm(m.x[:, :, None], m.w1, m.b1, 1e-6, True)
    near(s.h[:, :, None], y, b, "h")
    for i, w in ((0, m.wq), (1, m.wk)):
        y, _, _, b = ref.layer_norm(s.qkv[:, :, i], w, None, 1e-6, False)
        near(s.normed[:, :, i], y, b, "q, k norm")
        near(s.qk[:, :, i], *ref.rope(s.normed[:, :, i], m.freq, m.pos, m.pairs, half, 1.0, False), "rope")
    want = ref.attn_bwd(s.qk[:, :, 0], s.qk[:, :, 1], s.qkv[:, :, 2], s.o, s.lse, m.dout, D ** -0.5, m.allow)
    for i, (g, b) in enumerate(want):
        ref.check(r.of_attn[:, :, i], g, b, "attention")
    chain = B * N * H // 100 + 300      # as in the layer norm's own test
    for i, w, rstd, dw in ((0, m.wq, s.rq, r.dwq), (1, m.wk, s.rk, r.dwk)):
        near(r.of_rope[:, :, i], *ref.rope(r.of_attn[:, :, i], m.freq, m.pos, m.pairs, half, 1.0, True), "rope back")
        (g, b), (gw, bw), _ = ref.layer_norm_bwd(r.of_rope[:, :, i], s.qkv[:, :, i], None, rstd, w, chain)
        near(r.dqkv[:, :, i], g, b, "q, k norm back")
        ref.check(dw, gw, bw + 1e-30, "q, k weight")
    assert torch.equal(r.dqkv[:, :, 2], r.of_attn[:, :, 2]) and torch.equal(r.of_rope[:, :, 2], r.of_attn[:, :, 2])
    (g, b), (gw, bw), (gb, bb) = ref.layer_norm_bwd(r.dh[:, :, None], m.x[:, :, None], s.mean[:, :, None], s.rstd[:, :, None], m.w1, chain)
    near(r.dx[:, :, None], g, b, "dx")
    ref.check(r.dw1, gw, bw + 1e-30, "dw")
    ref.check(r.db1, gb, bb + 1e-30, "db")


@pytest.mark.parametrize("B,N,H,D,valid,frame,half", CASES)
def test_the_whole_gradient(dl, B, N, H, D, valid, frame, half):
    """Against 64-bit autograd, in norm: 14 tensors on the way are rounded to bf16
    (h, qkv, the norms of q and k, their turns, P, O, dS, the gradients of q, k
    and v, of the turns, of the norms, of h, of x), each by at most 2^-8 of its
    norm; with a condition of 4 on each that is 0.22.  A missing or reversed
    step is off by the gradient's own size."""
    m = Block(dl, B, N, H, D, valid, frame, half, 6)
    r = m.backward(m.forward())
    for name, got, want in zip(("x", "w1", "b1", "wq", "wk"), (r.dx, r.dw1, r.db1, r.dwq, r.dwk), m.exact()):
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 14 * 4 * ref.BF16, (name, off)


def _results(r):
    return [r.dx, r.dw1, r.db1, r.dwq, r.dwk, r.dqkv]


def test_captured_replayed_and_on_two_streams(dl):
    """Two blocks' steps as graphs, replayed at once on two streams, each with its
    own memory; new inputs through the same graphs; the same bits as alone."""
    blocks = [Block(dl, 2, 333, 2, 128, 320, 100, False, 7), Block(dl, 1, 700, 3, 64, 700, 0, True, 8)]
    alone = [_results(m.backward(m.forward())) for m in blocks]
    graphs, outs = [], []
    for m in blocks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = m.backward(m.forward())
        graphs.append(g)
        outs.append(_results(r))
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()

    def replay(times):
        for _ in range(times):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
    replay(6)
    for a, b in zip(alone, outs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    for m in blocks:
        m.x.mul_(-0.5)
        m.dout.add_(1.0)
    replay(1)
    for m, b in zip(blocks, outs):
        assert all(torch.equal(x, y) for x, y in zip(_results(m.backward(m.forward())), b))


def test_own_workspaces_on_a_given_stream_are_that_streams(dl, monkeypatch):
    """A workspace that a call allocates for itself is freed when the call
    returns, while its kernels may still run: it must come from the memory of
    the stream that the call was given."""
    from dit_long_sequence_gb300 import binding
    real, seen = binding._calls, []

    def spy(name, at):
        def f(*a):
            seen.append((name, a[at]))
            return getattr(real, name)(*a)
        return f
    monkeypatch.setattr(binding, "_calls", types.SimpleNamespace(attn_bwd=spy("attn_bwd", 15), norm_bwd=spy("norm_bwd", 9),
                                                               norm_fwd=real.norm_fwd))
    m = Block(dl, 1, 500, 2, 64, 490, 100, False, 9)
    q, k, v, do = (wl.randn_bf16((1, 500, 2, 64), 20 + i, DEV) for i in range(4))
    o, lse = dl.attn_fwd(q, k, v, out_dtype=BF)
    om, lm = dl.attn_fwd_masked(q, k, v, m.bits, key_valid_len=490, out_dtype=BF)
    y, mean, rstd = dl.layer_norm_fwd(m.x, m.w1)
    here = [*dl.attn_bwd(q, k, v, o, lse, do), *dl.attn_bwd_masked(q, k, v, om, lm, do, m.bits, key_valid_len=490),
            *dl.layer_norm_bwd(y, m.x, mean, rstd, m.w1)]
    assert [a[1] for a in seen] == [None] * 3
    seen.clear()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = [*dl.attn_bwd(q, k, v, o, lse, do, stream=side),
             *dl.attn_bwd_masked(q, k, v, om, lm, do, m.bits, key_valid_len=490, stream=side),
             *dl.layer_norm_bwd(y, m.x, mean, rstd, m.w1, stream=side)]
    assert all(a[1] is not None and a[1].dtype == torch.uint8 for a in seen) and len(seen) == 3
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(here, there))
    held = {t.data_ptr() for _, t in seen}
    side_blocks = {b["address"] for seg in torch.cuda.memory_snapshot() if seg["stream"] == side.cuda_stream for b in seg["blocks"]}
    assert held <= side_blocks


def test_offsets_past_32_bits(dl):
    """Batch entries more than 2^31 elements apart, and rows so; the same bits as packed."""
    far = 2 ** 31 + 4096
    buf = torch.empty(far + (1 << 20), dtype=BF, device=DEV)
    B, N, H, D = 2, 150, 2, 64
    at = iter(range(0, 1 << 20, N * H * D))

    def spread(t):
        view = buf.as_strided((B, N, H, D), (far, H * D, D, 1), next(at))
        if t is not None:
            view.copy_(t)
        return view
    q, k, v, do = (wl.randn_bf16((B, N, H, D), 40 + i, DEV) for i in range(4))
    o, lse = dl.attn_fwd(q, k, v, out_dtype=BF)
    want = dl.attn_bwd(q, k, v, o, lse, do)
    g = [spread(None) for _ in range(3)]
    dl.attn_bwd(*(spread(t) for t in (q, k, v, o)), lse, spread(do), dq=g[0], dk=g[1], dv=g[2])
    assert all(torch.equal(a, b) for a, b in zip(g, want))
    freq, _ = dl.rope_inv_freq(D)
    assert torch.equal(dl.rope(spread(q), freq, out=spread(None)), dl.rope(q, freq))
    w = torch.rand(D, device=DEV)
    y, mean, rstd = dl.layer_norm_fwd(q, w)
    z, m2, r2 = dl.layer_norm_fwd(spread(q), w, out=spread(None))
    assert torch.equal(z, y) and torch.equal(m2, mean) and torch.equal(r2, rstd)
    want = dl.layer_norm_bwd(do, q, mean, rstd, w)
    got = dl.layer_norm_bwd(spread(do), spread(q), mean, rstd, w, dx=spread(None))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # two rows that far apart
    x = wl.randn_bf16((1, 2, 1000), 50, DEV)
    rows = buf.as_strided((1, 2, 1000), (far, far, 1), 8)
    rows.copy_(x)
    y, mean, rstd = dl.layer_norm_fwd(x)
    assert torch.equal(dl.layer_norm_fwd(rows, out=rows)[0], y)
