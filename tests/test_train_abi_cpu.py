"""Host-side refusals of the training operators (no GPU needed): every argument
check returns its status before anything touches a device.  Made-up device
addresses are passed, so these run only where no device is visible."""
import ctypes
import math

import pytest
import torch

deviceless = pytest.mark.skipif(torch.cuda.is_available(), reason="passes made-up device addresses")
FAKE = 0x1000_0000


@pytest.fixture(scope="module")
def lib():
    from dit_long_sequence_gb300 import build
    build.build()
    from dit_long_sequence_gb300 import binding
    return binding


def _bwd(lib, masked=False, **kw):
    good = lib.Strides4(8 * 4 * 128, 4 * 128, 128, 1)
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, odt=lib.DIT_F32, lse=FAKE, do=FAKE, dlse=None, B=1, Nq=8, Nkv=8, H=4, D=128,
             kvl=8, scale=0.088, dq=FAKE, dk=FAKE, dv=FAKE, gdt=lib.DIT_BF16, ws=FAKE, wsb=1 << 30, mask=FAKE, sb=0, si=4,
             rows=8, st={})
    a.update(kw)
    st = lib.AttnBwdStrides(*(a["st"].get(n, good) for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")))
    head = (a["q"], a["k"], a["v"], a["o"], a["odt"], a["lse"], a["do"], a["dlse"], ctypes.byref(st), a["B"], a["Nq"],
            a["Nkv"], a["H"], a["D"], a["kvl"])
    tail = (a["scale"], a["dq"], a["dk"], a["dv"], a["gdt"], a["ws"], a["wsb"], None)
    if masked:
        return lib.raw().dit_attn_bwd_masked(*head, a["mask"], a["sb"], a["si"], a["rows"], *tail)
    return lib.raw().dit_attn_bwd(*head, *tail)


@deviceless
def test_attn_bwd_refusals(lib):
    I, U, A = lib.DIT_ERR_INVALID_ARG, lib.DIT_ERR_UNSUPPORTED, lib.DIT_ERR_ALIGNMENT
    assert _bwd(lib, D=96) == U and _bwd(lib, B=70000) == U
    for kw in (dict(kvl=9), dict(kvl=-1), dict(scale=0.0), dict(scale=math.nan), dict(B=-1), dict(Nkv=-1, kvl=-1),
               dict(q=None), dict(do=None), dict(lse=None), dict(o=None), dict(dq=None), dict(dk=None), dict(dv=None),
               dict(odt=7), dict(gdt=7)):
        assert _bwd(lib, **kw) == I, kw
    for kw in (dict(q=FAKE + 8), dict(do=FAKE + 2), dict(dq=FAKE + 8), dict(dv=FAKE + 4), dict(o=FAKE + 8),
               dict(lse=FAKE + 2)):
        assert _bwd(lib, **kw) == A, kw
    S = lib.Strides4
    bad_align, not_dense, zero = S(4096, 516, 128, 1), S(4096, 512, 128, 2), S(4096, 0, 128, 1)
    for n in ("q", "k", "v", "dout"):
        assert _bwd(lib, st={n: bad_align}) == A and _bwd(lib, st={n: not_dense}) == U and _bwd(lib, st={n: zero}) == I
    for n in ("dq", "dk", "dv"):
        assert _bwd(lib, st={n: bad_align}) == A and _bwd(lib, st={n: not_dense}) == U and _bwd(lib, st={n: zero}) == I
    assert _bwd(lib, st={"o": S(4096, -512, 128, 1)}) == I and _bwd(lib, st={"o": S(4096, 514, 128, 1)}) == A
    assert _bwd(lib, B=0, q=None, dq=None) == lib.DIT_OK
    assert _bwd(lib, Nq=0, Nkv=0, kvl=0, dq=None) == lib.DIT_OK


@deviceless
def test_attn_bwd_masked_refusals(lib):
    I, A = lib.DIT_ERR_INVALID_ARG, lib.DIT_ERR_ALIGNMENT
    for kw in (dict(rows=9), dict(rows=-1), dict(mask=None), dict(si=2), dict(sb=-4)):
        assert _bwd(lib, masked=True, **kw) == I, kw
    for kw in (dict(si=6), dict(sb=2), dict(mask=FAKE + 4)):
        assert _bwd(lib, masked=True, **kw) == A, kw


@deviceless
def test_layer_norm_refusals(lib):
    I, U, A = lib.DIT_ERR_INVALID_ARG, lib.DIT_ERR_UNSUPPORTED, lib.DIT_ERR_ALIGNMENT
    st = lib.Strides4(8 * 64, 64, 64, 1)
    F = lib.DIT_F32

    def fwd(x=FAKE, xd=F, sx=st, B=2, N=8, H=1, C=64, w=FAKE, b=None, pb=1, eps=1e-6, center=1, y=FAKE, yd=F, sy=st,
            mean=FAKE, rstd=FAKE):
        return lib.raw().dit_layer_norm_fwd(x, xd, ctypes.byref(sx), B, N, H, C, w, b, pb, eps, center, y, yd,
                                            ctypes.byref(sy), mean, rstd, None)

    def bwd(dy=FAKE, dd=F, sd=st, x=FAKE, xd=F, sx=st, mean=FAKE, rstd=FAKE, w=FAKE, B=2, N=8, H=1, C=64, pb=1, center=1,
            dx=FAKE, so=st, dw=FAKE, db=FAKE, ws=FAKE, wsb=1 << 30):
        return lib.raw().dit_layer_norm_bwd(dy, dd, ctypes.byref(sd), x, xd, ctypes.byref(sx), mean, rstd, w, B, N, H, C,
                                            pb, center, dx, ctypes.byref(so), dw, db, ws, wsb, None)
    for f in (fwd, bwd):
        for kw in (dict(B=-1), dict(N=-1), dict(C=-1), dict(pb=3), dict(pb=0), dict(x=None), dict(rstd=None),
                   dict(mean=None), dict(xd=9)):
            assert f(**kw) == I, kw
        assert f(C=8200) == U and f(B=65536, pb=1, N=1 << 16) == U
        assert f(sx=lib.Strides4(512, 64, 64, 2)) == U and f(sx=lib.Strides4(512, -64, 64, 1)) == I
        assert f(x=FAKE + 2) == A and f(rstd=FAKE + 1) == A
        assert f(C=0) == lib.DIT_OK and f(B=0, pb=1) == lib.DIT_OK
    assert fwd(eps=-1.0) == I and fwd(eps=math.inf) == I and fwd(y=None) == I and fwd(xd=lib.DIT_BF16) == U
    assert fwd(sy=lib.Strides4(512, 0, 64, 1)) == I                    # rows of y at one place
    assert bwd(dy=None) == I and bwd(dx=None) == I and bwd(so=lib.Strides4(0, 64, 64, 1)) == I
    assert bwd(dw=FAKE + 2) == A


@deviceless
def test_rope_refusals(lib):
    I, U, A = lib.DIT_ERR_INVALID_ARG, lib.DIT_ERR_UNSUPPORTED, lib.DIT_ERR_ALIGNMENT
    st = lib.Strides4(8 * 256, 256, 64, 1)

    def call(x=FAKE, dt=lib.DIT_BF16, sx=st, B=1, N=8, H=4, D=64, R=64, lay=0, freq=None, pairs=(32,), axes=None, pos=None,
             psb=0, off=0, ms=1.0, y=FAKE, sy=st, nofreq=False):
        f = torch.ones(512, dtype=torch.float64) if freq is None else freq
        return lib.raw().dit_rope(x, dt, ctypes.byref(sx), B, N, H, D, R, lay, None if nofreq else f.data_ptr(),
                                  (ctypes.c_int * len(pairs))(*pairs), len(pairs) if axes is None else axes, pos, psb, off,
                                  ms, 0, y, ctypes.byref(sy), None)
    for kw in (dict(R=63), dict(R=66), dict(R=0), dict(lay=2), dict(ms=math.nan), dict(nofreq=True), dict(pairs=(31,)),
               dict(pairs=(33,)), dict(pairs=(33, -1), pos=FAKE), dict(pairs=(16, 16)), dict(pos=FAKE, psb=4), dict(B=-1),
               dict(freq=torch.full((32,), math.inf, dtype=torch.float64)), dict(x=None), dict(y=None), dict(dt=5),
               dict(sx=lib.Strides4(2048, -256, 64, 1)), dict(sy=lib.Strides4(2048, 0, 64, 1)), dict(axes=0)):
        assert call(**kw) == I, kw
    assert call(D=2048, sx=lib.Strides4(1 << 20, 1 << 16, 2048, 1)) == U
    assert call(D=512, R=512, pairs=(256,)) == U                       # more than 128 pairs
    assert call(pairs=(8, 8, 8, 4, 4), pos=FAKE) == U                  # five axes
    assert call(H=70000) == U and call(sx=lib.Strides4(2048, 256, 64, 2)) == U
    assert call(x=FAKE + 1) == A and call(pos=FAKE + 2) == A
    assert call(N=0) == lib.DIT_OK


def test_rope_schedules(lib):
    import dit_long_sequence_gb300 as dl
    for dim, base in ((2, 10000.0), (64, 10000.0), (128, 500000.0)):
        P = dim // 2
        plain, m = dl.rope_inv_freq(dim, base=base)
        want = torch.tensor([base ** (-i / P) for i in range(P)], dtype=torch.float64)
        assert m == 1.0 and torch.allclose(plain, want, rtol=1e-14, atol=0)
        lin, _ = dl.rope_inv_freq(dim, base=base, scaling="linear", factor=8.0)
        assert torch.allclose(lin, want / 8.0, rtol=1e-14, atol=0)
        big, _ = dl.rope_inv_freq(dim, base=base, scaling="base", factor=8.0)
        assert float(big[0]) == 1.0
        if P > 1:
            assert math.isclose(float(big[-1]), float(want[-1]) / 8.0, rel_tol=1e-12)   # the slowest pair: by factor
        parts, m = dl.rope_inv_freq(dim, base=base, scaling="by_parts", factor=8.0, original_len=4096)
        assert math.isclose(m, 0.1 * math.log(8.0) + 1.0, rel_tol=1e-6)
        turns = 4096 * want / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0, 1)
        assert torch.allclose(parts, keep * want + (1 - keep) * want / 8.0, rtol=1e-13, atol=0)
    for kw in (dict(base=0.0), dict(scaling="linear", factor=0.5), dict(scaling="by_parts", factor=2.0, original_len=0.0),
               dict(scaling="by_parts", factor=2.0, beta_fast=1.0, beta_slow=1.0)):
        with pytest.raises(dl.DitError):
            dl.rope_inv_freq(64, **kw)
    with pytest.raises(ValueError):
        dl.rope_inv_freq(63)
    with pytest.raises(ValueError):
        dl.rope_inv_freq(64, scaling="other")


def test_workspaces_of_nothing_are_empty(lib):
    import dit_long_sequence_gb300 as dl
    assert dl.attn_bwd_workspace_bytes(0, 8, 8, 4, 128, 8) == 0 and dl.attn_bwd_workspace_bytes(1, 8, 8, 4, 128, 0) == 0
    assert dl.attn_bwd_workspace_bytes(1, 8, 8, 4, 96, 8) == 0 and dl.attn_bwd_workspace_bytes(1, 8, 8, 4, 128, 9) == 0
    assert dl.layer_norm_bwd_workspace_bytes(0, 8, 1, 64) == 0 and dl.layer_norm_bwd_workspace_bytes(1, 8, 1, 9000) == 0
