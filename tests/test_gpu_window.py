"""GPU parity of dit_attn_fwd_window and dit_attn_bwd_window with the 64-bit formulas,
element by element within the bounds window_ref derives from the kernels'
roundings."""
import math

import pytest
import torch

import train_ref as ref
import window_ref as win
from dit_long_sequence_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def dl():
    import dit_long_sequence_gb300 as m
    return m


@pytest.fixture(autouse=True)
def no_wait_ran_out(dl):
    yield
    rc, info = dl.check_watchdog()
    assert rc == 0, info


def inputs(B, Nq, Nkv, H, Hkv, D, seed, scale_q=1.5):
    g = wl.generator(DEV, seed)

    def t(n, h, s=1.0):
        return (torch.randn((B, n, h, D), generator=g, device=DEV) * s).to(torch.bfloat16)
    return t(Nq, H, scale_q), t(Nkv, Hkv), t(Nkv, Hkv), t(Nq, H, 0.25)


def table_of(Nq, Nkv, w, offset, kvl):
    return win.sees(torch.arange(Nq, device=DEV) + offset, Nkv, *w, kvl)[None, None]


# left, right, sinks, frame
WINDOWS = [(None, 0, 0, 1), (100, 0, 4, 1), (0, 0, 0, 1), (0, 0, 1, 1), (300, 7, 130, 1), (None, None, 0, 1), (2, 0, 50, 50), (0, 1, 0, 37),
           (None, 0, 0, 200), (1, 0, 300, 96), (5, None, 0, 1), (0, 0, 2000, 64)]
# B, Nq, Nkv, H, Hkv, D, offset, kvl
SIZES = [(1, 1, 1, 1, 1, 64, 0, 1), (1, 300, 300, 2, 2, 128, 0, 300), (2, 257, 700, 3, 1, 64, 443, 690), (1, 640, 640, 4, 2, 128, 0, 611),
         (1, 129, 1000, 5, 1, 128, 871, 1000), (2, 513, 513, 2, 2, 64, 0, 513)]


@pytest.mark.parametrize("w", WINDOWS)
@pytest.mark.parametrize("B,Nq,Nkv,H,Hkv,D,offset,kvl", SIZES)
def test_forward_matches_the_formulas(dl, w, B, Nq, Nkv, H, Hkv, D, offset, kvl):
    q, k, v, _ = inputs(B, Nq, Nkv, H, Hkv, D, 11 + Nq + Nkv)
    left, right, sinks, frame = w
    allow = table_of(Nq, Nkv, w, offset, kvl)
    scale = D ** -0.5
    kk, vv = k.clone(), v.clone()
    kk[:, kvl:] = float("nan")       # pad keys are never read
    vv[:, kvl:] = float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = dl.attn_fwd_window(q, kk, vv, left=left, right=right, sinks=sinks, frame=frame, offset=offset, key_valid_len=kvl,
                                      out_dtype=dtype)
        torch.cuda.synchronize()
        assert out.dtype == dtype
        win.check_forward(out, lse, win.forward(q, win.shared(k, H), win.shared(v, H), scale, allow, dtype == torch.bfloat16))


@pytest.mark.parametrize("w", WINDOWS)
@pytest.mark.parametrize("B,Nq,Nkv,H,Hkv,D,offset,kvl", SIZES)
def test_backward_matches_the_formulas(dl, w, B, Nq, Nkv, H, Hkv, D, offset, kvl):
    q, k, v, dout = inputs(B, Nq, Nkv, H, Hkv, D, 12 + Nq + Nkv)
    left, right, sinks, frame = w
    allow = table_of(Nq, Nkv, w, offset, kvl)
    scale = 0.11
    o, l = ref.attn_forward(q, win.shared(k, H), win.shared(v, H), scale, allow)
    kk, vv = k.clone(), v.clone()
    kk[:, kvl:] = float("nan")
    vv[:, kvl:] = float("inf")
    for dtype, dlse in ((torch.bfloat16, None), (torch.float32, torch.randn((B, H, Nq), device=DEV))):
        out, lse = o.nan_to_num(0.0).to(dtype).contiguous(), l.float().contiguous()
        grads = dl.attn_bwd_window(q, kk, vv, out, lse, dout, left=left, right=right, sinks=sinks, frame=frame, offset=offset,
                                   key_valid_len=kvl, scale=scale, grad_dtype=dtype, dlse=dlse)
        torch.cuda.synchronize()
        want = win.backward(q, k, v, out, lse, dout, scale, allow, dlse, dtype == torch.bfloat16)
        for name, g, (r, b) in zip(("dq", "dk", "dv"), grads, want):
            assert g.dtype == dtype
            ref.check(g, r, b, name)
        assert (grads[1][:, kvl:] == 0).all() and (grads[2][:, kvl:] == 0).all()


def test_many_items(dl):
    """More items than SMs, so that CTAs go on to further ones; uneven ones (causal)."""
    B, N, H, Hkv, D = 2, 2500, 24, 12, 64
    q, k, v, dout = inputs(B, N, N, H, Hkv, D, 3)
    for w in ((None, 0, 0, 1), (300, 0, 10, 1)):
        out, lse = dl.attn_fwd_window(q, k, v, left=w[0], right=w[1], sinks=w[2], frame=w[3], out_dtype=torch.bfloat16)
        grads = dl.attn_bwd_window(q, k, v, out, lse, dout, left=w[0], right=w[1], sinks=w[2], frame=w[3])
        torch.cuda.synchronize()
        allow = table_of(N, N, w, 0, N)
        for b in range(B):
            for hk in (0, 5, Hkv - 1):
                hs = slice(2 * hk, 2 * hk + 2)
                one = [t[b:b + 1, :, hs].contiguous() for t in (q, out, dout)]
                kv = [t[b:b + 1, :, hk:hk + 1].contiguous() for t in (k, v)]
                l1 = lse[b:b + 1, hs].contiguous()
                win.check_forward(one[1], l1, win.forward(one[0], win.shared(kv[0], 2), win.shared(kv[1], 2), D ** -0.5, allow, True))
                want = win.backward(one[0], *kv, one[1], l1, one[2], D ** -0.5, allow)
                got = grads[0][b:b + 1, :, hs], grads[1][b:b + 1, :, hk:hk + 1], grads[2][b:b + 1, :, hk:hk + 1]
                for name, g, (r, bd) in zip(("dq", "dk", "dv"), got, want):
                    ref.check(g, r, bd, name)
