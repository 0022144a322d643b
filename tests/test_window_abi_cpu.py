"""Host-side refusals of windowed attention and the paged cache (no GPU needed): every
argument check returns its status before anything touches a device.  Made-up device
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


def _window(lib, kw):
    w = dict(left=3, right=0, sinks=4, frame=2)
    w.update(kw.pop("w", {}))
    return None if kw.pop("no_window", False) else ctypes.byref(lib.Window(w["left"], w["right"], w["sinks"], w["frame"]))


def _fwd(lib, **kw):
    good = lib.Strides4(8 * 4 * 128, 4 * 128, 128, 1)
    win = _window(lib, kw)
    a = dict(q=FAKE, k=FAKE + 4096, v=FAKE + 8192, out=FAKE + 16384, odt=lib.DIT_F32, lse=FAKE + 32768, B=1, Nq=8, Nkv=8, H=4, Hkv=4, D=128,
             kvl=8, off=0, scale=0.088, ws=FAKE, wsb=1 << 40, st={})
    a.update(kw)
    st = lib.AttnStrides(*(a["st"].get(n, good) for n in "qkvo"))
    return lib.raw().dit_attn_fwd_window(a["q"], a["k"], a["v"], ctypes.byref(st), a["B"], a["Nq"], a["Nkv"], a["H"], a["Hkv"], a["D"], a["kvl"],
                                         win, a["off"], a["scale"], a["out"], a["odt"], a["lse"], a["ws"], a["wsb"], None)


def _bwd(lib, **kw):
    good = lib.Strides4(8 * 4 * 128, 4 * 128, 128, 1)
    win = _window(lib, kw)
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, do=FAKE, B=1, Nq=8, Nkv=8, H=4, Hkv=4, D=128, kvl=8, off=0, scale=0.088, dq=FAKE + 64,
             dk=FAKE + 128, dv=FAKE + 256, ws=FAKE, wsb=1 << 40, st={})
    a.update(kw)
    st = lib.AttnBwdStrides(*(a["st"].get(n, good) for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv")))
    return lib.raw().dit_attn_bwd_window(a["q"], a["k"], a["v"], a["o"], lib.DIT_F32, a["lse"], a["do"], None, ctypes.byref(st), a["B"], a["Nq"],
                                         a["Nkv"], a["H"], a["Hkv"], a["D"], a["kvl"], win, a["off"], a["scale"], a["dq"], a["dk"], a["dv"],
                                         lib.DIT_BF16, a["ws"], a["wsb"], None)


def _cache(lib, kw):
    s = lib.Strides4(16 * 4 * 128, 4 * 128, 128, 1)
    c = dict(k=FAKE, v=FAKE + 65536, ks=s, vs=s, pages=10, page=16, table=FAKE, stride=4, width=4, lens=FAKE)
    c.update(kw.pop("c", {}))
    return None if kw.pop("no_cache", False) else ctypes.byref(
        lib.PagedCache(c["k"], c["v"], c["ks"], c["vs"], c["pages"], c["page"], c["table"], c["stride"], c["width"], c["lens"]))


def _paged(lib, **kw):
    win, cache = _window(lib, kw), _cache(lib, kw)
    good = lib.Strides4(8 * 4 * 128, 4 * 128, 128, 1)
    a = dict(q=FAKE, sq=good, ql=None, B=2, T=1, H=4, Hkv=4, D=128, scale=0.1, out=FAKE + 1024, odt=lib.DIT_BF16, so=good, lse=FAKE + 2048, ws=FAKE,
             wsb=1 << 40)
    a.update(kw)
    return lib.raw().dit_attn_fwd_paged(a["q"], ctypes.byref(a["sq"]), cache, a["ql"], a["B"], a["T"], a["H"], a["Hkv"], a["D"], win, a["scale"],
                                        a["out"], a["odt"], ctypes.byref(a["so"]), a["lse"], a["ws"], a["wsb"], None)


def _append(lib, **kw):
    cache = _cache(lib, kw)
    good = lib.Strides4(8 * 4 * 128, 4 * 128, 128, 1)
    a = dict(k=FAKE + 32, sk=good, v=FAKE + 64, sv=good, nl=None, B=2, T=1, Hkv=4, D=128)
    a.update(kw)
    return lib.raw().dit_paged_append(a["k"], ctypes.byref(a["sk"]), a["v"], ctypes.byref(a["sv"]), cache, a["nl"], a["B"], a["T"], a["Hkv"],
                                      a["D"], None)


BAD_WINDOWS = [dict(frame=0), dict(frame=-1), dict(frame=(1 << 30) + 1), dict(sinks=-1)]


@deviceless
def test_window_forward_refusals(lib):
    I, U, A = lib.DIT_ERR_INVALID_ARG, lib.DIT_ERR_UNSUPPORTED, lib.DIT_ERR_ALIGNMENT
    S = lib.Strides4
    for w in BAD_WINDOWS:
        assert _fwd(lib, w=w) == I, w
    for kw in (dict(no_window=True), dict(kvl=9), dict(kvl=-1), dict(scale=0.0), dict(scale=math.inf), dict(B=-1), dict(Hkv=3), dict(Hkv=0),
               dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(lse=None), dict(odt=5), dict(out=FAKE)):
        assert _fwd(lib, **kw) == I, kw
    for kw in (dict(D=96), dict(B=70000), dict(H=258, Hkv=2), dict(off=1 << 29), dict(off=-(1 << 29)), dict(Nkv=(1 << 29) + 1)):
        assert _fwd(lib, **kw) == U, kw
    for kw in (dict(q=FAKE + 8), dict(out=FAKE + 16384 + 8), dict(lse=FAKE + 2), dict(st={"o": S(4096, 514, 128, 1)}),
               dict(st={"k": S(4096, 516, 128, 1)})):
        assert _fwd(lib, **kw) == A, kw
    assert _fwd(lib, st={"v": S(4096, 512, 128, 2)}) == U and _fwd(lib, st={"q": S(4096, 0, 128, 1)}) == I
    assert _fwd(lib, st={"o": S(4096, 0, 128, 1)}) == I         # rows of out at one place
    assert _fwd(lib, B=0, q=None, out=None) == lib.DIT_OK and _fwd(lib, Nq=0) == lib.DIT_OK and _fwd(lib, H=0, Hkv=0) == lib.DIT_OK


@deviceless
def test_window_backward_refusals(lib):
    I, U = lib.DIT_ERR_INVALID_ARG, lib.DIT_ERR_UNSUPPORTED
    for w in BAD_WINDOWS:
        assert _bwd(lib, w=w) == I, w
    for kw in (dict(no_window=True), dict(Hkv=3), dict(Hkv=0), dict(Hkv=-1), dict(kvl=9), dict(dq=None), dict(dk=None), dict(do=None), dict(dq=FAKE)):
        assert _bwd(lib, **kw) == I, kw
    for kw in (dict(D=80), dict(H=258, Hkv=2), dict(off=1 << 29), dict(Nkv=(1 << 29) + 1)):
        assert _bwd(lib, **kw) == U, kw
    assert _bwd(lib, st={"dk": lib.Strides4(4096, 512, 0, 1)}) == I
    assert _bwd(lib, B=0) == lib.DIT_OK


@deviceless
def test_paged_refusals(lib):
    I, U, A = lib.DIT_ERR_INVALID_ARG, lib.DIT_ERR_UNSUPPORTED, lib.DIT_ERR_ALIGNMENT
    S = lib.Strides4
    for call in (_paged, _append):
        for kw in (dict(no_cache=True), dict(c=dict(k=None)), dict(c=dict(table=None)), dict(c=dict(lens=None)), dict(c=dict(pages=-1)),
                   dict(c=dict(page=0)), dict(c=dict(width=-1)), dict(c=dict(stride=-1)), dict(c=dict(ks=S(0, 512, 128, 1))), dict(B=-1)):
            assert call(lib, **kw) == I, (call, kw)
        for kw in (dict(c=dict(page=20)), dict(c=dict(page=1 << 20, width=1 << 12)), dict(c=dict(vs=S(8192, 512, 128, 2))), dict(B=70000)):
            assert call(lib, **kw) == U, (call, kw)
        for kw in (dict(c=dict(k=FAKE + 8)), dict(c=dict(vs=S(8192, 516, 128, 1))), dict(c=dict(lens=FAKE + 2)), dict(c=dict(table=FAKE + 1))):
            assert call(lib, **kw) == A, (call, kw)
    for w in BAD_WINDOWS:
        assert _paged(lib, w=w) == I, w
    for kw in (dict(no_window=True), dict(q=None), dict(out=None), dict(lse=None), dict(Hkv=3), dict(scale=-1.0), dict(odt=9), dict(out=FAKE)):
        assert _paged(lib, **kw) == I, kw
    assert _paged(lib, D=256) == U and _paged(lib, ql=FAKE + 2) == A and _paged(lib, q=FAKE + 8) == A
    for kw in (dict(k=None), dict(v=None), dict(k=FAKE), dict(v=FAKE + 65536), dict(c=dict(k=FAKE, v=FAKE))):
        assert _append(lib, **kw) == I, kw
    assert _append(lib, D=12) == U and _append(lib, D=2048) == U and _append(lib, nl=FAKE + 1) == A
    assert _paged(lib, T=0) == lib.DIT_OK and _append(lib, T=0) == lib.DIT_OK


def test_no_workspace_for_what_is_refused(lib):
    with_window = lib.Window(1, 0, 0, 0)
    assert lib.raw().dit_attn_fwd_window_workspace_bytes(1, 8, 4, 4, 128, 8, ctypes.byref(with_window), 0) == 0
    assert lib.attn_fwd_window_workspace_bytes(1, 8, 4, 3, 128, 8) == 0 and lib.attn_bwd_window_workspace_bytes(1, 8, 8, 4, 3, 128, 8) == 0
    assert lib.attn_fwd_paged_workspace_bytes(1, 1, 4, 4, 96, 16, 10) == 0
