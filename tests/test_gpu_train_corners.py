"""The training operators in corners of what their documentation allows that the
other tests do not reach."""
import math

import pytest
import torch

from dit_long_sequence_gb300 import workloads as wl
from test_gpu_attn_bwd import _allow, _check, _forward, _inputs, _mask

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dl():
    import dit_long_sequence_gb300 as m
    return m


@pytest.fixture(autouse=True)
def no_wait_ran_out(dl):
    yield
    rc, info = dl.check_watchdog()
    assert rc == 0, info


# ---------------------------------------------------------------- layer norm

@pytest.mark.parametrize("shape", [(0, 5, 64), (0, 5, 2, 64), (2, 0, 2, 64), (2, 5, 0, 64), (0, 0, 64)])
@pytest.mark.parametrize("given", [False, True])
def test_parameter_gradients_over_no_rows_are_zeros(dl, shape, given):
    x = torch.empty(shape, dtype=BF, device=DEV)
    w = torch.ones(64, device=DEV)
    rows = torch.empty(shape[:-1], device=DEV)
    dw, db = torch.full_like(w, 3.0), torch.full_like(w, 3.0)
    if given:
        _, a, b = dl.layer_norm_bwd(x, x, rows, rows, w, dweight=dw, dbias=db)
        assert a is dw and b is db
    else:
        del dw, db      # (fresh results would take this memory)
        _, a, b = dl.layer_norm_bwd(x, x, rows, rows, w)
    torch.cuda.synchronize()
    assert bool((a == 0).all() and (b == 0).all())


def test_a_set_of_parameters_for_each_of_no_batch_entries(dl):
    x, w = torch.empty((0, 5, 64), device=DEV), torch.empty((0, 64), device=DEV)
    dx, dw, db = dl.layer_norm_bwd(x, x, x[..., 0], x[..., 0], w)
    assert dx.shape == x.shape and dw.shape == w.shape and db.shape == w.shape


# ---------------------------------------------------------------- attention backward

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("junk", [math.nan, math.inf])
def test_rows_without_a_key_contribute_nothing_whatever_they_hold(dl, D, junk):
    """A merge of two LSE of -inf has NaN gradients, and O of such a row may be
    anything: the same bits as with zeros there."""
    B, N, H = 2, 300, 2
    q, k, v, dout, g = _inputs(B, N, N, H, D, 15)
    m = _mask("holes", B, N, N, g)
    allow = _allow(B, N, N, N, m)
    out, lse = _forward(q, k, v, D ** -0.5, allow, F)
    bits = wl.pack_mask_bits(m).to(DEV)
    dlse = torch.randn((B, H, N), generator=g, device=DEV)
    none = torch.isinf(lse)
    assert bool(none.any())
    got = []
    for fill in (0.0, junk):
        o = out.masked_fill(none.transpose(1, 2)[..., None], fill)
        d = dlse.masked_fill(none, fill)
        got.append(dl.attn_bwd_masked(q, k, v, o, lse, dout, bits, dlse=d))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    empty = ~allow[:, 0].any(-1)
    assert bool((got[1][0][empty] == 0).all())


@pytest.mark.parametrize("Nq,Nkv,kvl", [(1, 1, 1), (33, 65, 64), (127, 129, 97), (161, 255, 250), (1000, 31, 31)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("grad_dtype", [BF, F])
def test_tiles_that_end_inside_a_warps_rows(dl, Nq, Nkv, kvl, D, grad_dtype):
    """The rows of one warp that are there and those that are not: gradients in
    the middle of a larger buffer, whose other rows stay."""
    q, k, v, dout, _ = _inputs(2, Nq, Nkv, 2, D, 23 + Nq)
    allow = _allow(2, Nq, Nkv, kvl)
    out, lse = _forward(q, k, v, D ** -0.5, allow, BF)
    bufs = [torch.full((2, n + 256, 2, D), 5.0, dtype=grad_dtype, device=DEV) for n in (Nq, Nkv, Nkv)]
    views = [b[:, :b.shape[1] - 256] for b in bufs]
    dl.attn_bwd(q, k, v, out, lse, dout, key_valid_len=kvl, dq=views[0], dk=views[1], dv=views[2])
    torch.cuda.synchronize()
    _check(views, q, k, v, out, lse, dout, D ** -0.5, allow)
    assert all(bool((b[:, b.shape[1] - 256:] == 5.0).all()) for b in bufs)
