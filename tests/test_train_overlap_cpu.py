"""The training operators refuse results that begin where an input or another
result begins, except in the in-place forms that the header names.  Host checks
(made-up device addresses, so only where no device is visible): a call that
passes them goes on to ask the driver and fails there with another status."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="passes made-up device addresses")
P = [0x1000_0000 + (i << 24) for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    from dit_long_sequence_gb300 import build
    build.build()
    from dit_long_sequence_gb300 import binding
    return binding


def test_attn_bwd(lib):
    s = lib.Strides4(8 * 4 * 128, 4 * 128, 128, 1)
    st = lib.AttnBwdStrides(*[s] * 8)

    def call(**kw):
        a = dict(q=P[0], k=P[1], v=P[2], o=P[3], lse=P[4], do=P[5], dlse=P[6], dq=P[7], dk=P[8], dv=P[9], ws=P[10])
        a.update(kw)
        return lib.raw().dit_attn_bwd(a["q"], a["k"], a["v"], a["o"], lib.DIT_BF16, a["lse"], a["do"], a["dlse"], ctypes.byref(st),
                                      1, 8, 8, 4, 128, 8, 0.1, a["dq"], a["dk"], a["dv"], lib.DIT_BF16, a["ws"], 1 << 30, None)
    assert call() not in (lib.DIT_OK, lib.DIT_ERR_INVALID_ARG)
    grads = {"dq": P[7], "dk": P[8], "dv": P[9]}
    for g, at in grads.items():
        for other in ("q", "k", "v", "o", "lse", "do", "dlse", "ws", *(n for n in grads if n != g)):
            assert call(**{other: at}) == lib.DIT_ERR_INVALID_ARG, (g, other)
    assert call(k=P[0], v=P[0]) != lib.DIT_ERR_INVALID_ARG          # inputs may be one


def test_layer_norm(lib):
    s, other = lib.Strides4(8 * 64, 64, 64, 1), lib.Strides4(8 * 128, 128, 64, 1)
    F, H = lib.DIT_F32, lib.DIT_BF16

    def fwd(sy=s, yd=F, y=P[0], B=2):
        return lib.raw().dit_layer_norm_fwd(P[0], F, ctypes.byref(s), B, 8, 1, 64, None, None, 1, 1e-6, 1, y, yd,
                                            ctypes.byref(sy), P[1], P[2], None)

    def bwd(dx, so=s, dd=F, dw=P[5], db=P[6]):
        return lib.raw().dit_layer_norm_bwd(P[0], dd, ctypes.byref(s), P[1], F, ctypes.byref(s), P[2], P[3], P[4], 2, 8, 1, 64,
                                            1, 1, dx, ctypes.byref(so), dw, db, P[8], 1 << 30, None)
    I = lib.DIT_ERR_INVALID_ARG
    assert fwd() != I and fwd(y=P[9], sy=other) != I and fwd(sy=other) == I and fwd(yd=H) == I
    assert fwd(sy=lib.Strides4(1 << 20, 64, 64, 1), B=1) != I        # the batch stride of one batch entry says nothing
    assert bwd(P[0]) != I and bwd(P[1]) != I and bwd(P[9], other) != I
    assert bwd(P[0], other) == I and bwd(P[1], other) == I and bwd(P[0], dd=H) == I
    assert bwd(P[9], db=P[5]) == I and bwd(P[9], dw=None, db=None) != I


def test_rope(lib):
    s, other = lib.Strides4(8 * 256, 256, 64, 1), lib.Strides4(8 * 512, 512, 64, 1)
    freq = torch.ones(32, dtype=torch.float64)

    def call(y, sy):
        return lib.raw().dit_rope(P[0], lib.DIT_BF16, ctypes.byref(s), 1, 8, 4, 64, 64, 0, freq.data_ptr(),
                                  (ctypes.c_int * 1)(32), 1, None, 0, 0, 1.0, 0, y, ctypes.byref(sy), None)
    I = lib.DIT_ERR_INVALID_ARG
    assert call(P[0], s) != I and call(P[1], other) != I and call(P[0], other) == I
