"""GPU parity of dit_layer_norm_fwd / _bwd with the 64-bit formulas within
train_ref's derived bounds."""
import pytest
import torch

import train_ref as ref
from dit_long_sequence_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def dl():
    import dit_long_sequence_gb300 as m
    return m


def _rnd(t):
    return ref.BF16 if t == BF else 2.0 ** -24


# (B, N, H, C): one row to many, C of one channel, odd, past each vector and thread count, the widest
SHAPES = [(1, 1, 1, 1), (2, 3, 1, 7), (1, 5, 1, 8), (3, 37, 1, 130), (2, 19, 1, 1000), (1, 33, 1, 2048), (2, 70, 1, 4096),
          (1, 9, 1, 4100), (1, 4, 1, 8192), (1, 3, 1, 8191), (2, 50, 6, 128), (1, 700, 3, 64), (2, 5000, 1, 24)]


def _data(B, N, H, C, tx, seed, strided):
    g = wl.generator(DEV, seed)
    x = (torch.randn((B, N, 3 if strided else 1, H, C), generator=g, device=DEV) * 2 +
         torch.randn((C,), generator=g, device=DEV) * 3).to(tx)[:, :, -1]
    return x, g


@pytest.mark.parametrize("B,N,H,C", SHAPES)
@pytest.mark.parametrize("tx,ty", [(BF, BF), (F, F), (F, BF)])
@pytest.mark.parametrize("center,per_batch,strided", [(True, False, False), (False, False, True), (True, True, True)])
def test_forward_and_backward(dl, B, N, H, C, tx, ty, center, per_batch, strided):
    x, g = _data(B, N, H, C, tx, 3 + C, strided)
    shape = (B, C) if per_batch else (C,)
    w = 1 + 0.3 * torch.randn(shape, generator=g, device=DEV)
    b = torch.randn(shape, generator=g, device=DEV)
    eps = 1e-5
    y, mean, rstd = dl.layer_norm_fwd(x, w, b, eps=eps, center=center, out_dtype=ty)
    want, m, r, bound = ref.layer_norm(x, w, b, eps, center)
    ref.check(y, want, 1.01 * bound + _rnd(ty) * want.abs(), "y")
    xa = x.double().abs().mean(-1)
    if center:
        ref.check(mean, m, 64 * 2.0 ** -24 * xa + 1e-30, "mean")
    else:
        assert mean is None
    # rstd' = -rstd^3 / 2 of the variance, whose error is a chain of 64 on deviations that carry the mean's error
    dev = (x.double() - (m[..., None] if center else 0)).abs().mean(-1)
    ref.check(rstd, r, 64 * ref.EPS32 * r * (1 + r * r * dev * xa), "rstd")

    dy = torch.randn((B, N, H, C), generator=g, device=DEV).to(ty)
    dx, dw, db = dl.layer_norm_bwd(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    assert dx.dtype == tx and dw.shape == w.shape and db.shape == w.shape
    # rows in one chain of sums: a thread's own (blocks of 256 threads on at least 100 SMs, or one block), its
    # block's row slots (at most 256), the partials
    chain = B * N * H // 100 + 300
    (rx, bx), (rw, bw), (rb, bb) = ref.layer_norm_bwd(dy, x, mean, rstd, w, chain)
    ref.check(dx, rx, 1.01 * bx + _rnd(tx) * rx.abs(), "dx")
    ref.check(dw, rw, bw + 1e-30, "dweight")
    ref.check(db, rb, bb + 1e-30, "dbias")
    again = dl.layer_norm_bwd(dy, x, mean, rstd, w)
    assert all(torch.equal(s, t) for s, t in zip((dx, dw, db), again))


@pytest.mark.parametrize("tx,ty", [(BF, BF), (F, BF)])
@pytest.mark.parametrize("N,C", [(2500, 1152), (1300, 1501), (1200, 2560), (900, 1538), (300, 5120), (400, 6150), (170, 7001), (1, 5120),
                                 (301, 6144), (2, 4104), (1201, 4616)])
def test_rows_of_three_to_fifteen_warps(dl, N, C, tx, ty):
    """Numbers of warps that are no power of two, in blocks of one to five rows."""
    test_forward_and_backward(dl, 1, N, 1, C, tx, ty, True, False, False)


def test_three_dimensions_and_no_parameters(dl):
    x, g = _data(2, 11, 1, 96, BF, 5, False)
    x = x[:, :, 0]
    y, mean, rstd = dl.layer_norm_fwd(x)
    want, _, _, bound = ref.layer_norm(x.unsqueeze(2), None, None, 1e-6, True)
    assert y.shape == x.shape and mean.shape == (2, 11)
    ref.check(y, want[:, :, 0], 1.01 * bound[:, :, 0] + ref.BF16 * want[:, :, 0].abs())
    dx, dw, db = dl.layer_norm_bwd(y, x, mean, rstd)
    assert dw is None and db is None
    (rx, bx), _, _ = ref.layer_norm_bwd(y.unsqueeze(2), x.unsqueeze(2), mean.unsqueeze(2), rstd.unsqueeze(2), None, 400)
    ref.check(dx, rx[:, :, 0], 1.01 * bx[:, :, 0] + ref.BF16 * rx[:, :, 0].abs())
    # one parameter gradient without the other
    w = torch.ones(96, device=DEV)
    _, dw, db = dl.layer_norm_bwd(y, x, mean, rstd, w, has_bias=False)
    _, dw2, db2 = dl.layer_norm_bwd(y, x, mean, rstd, w)
    assert db is None and torch.equal(dw, dw2)
    only = torch.empty(96, device=DEV)
    _, none, got = dl.layer_norm_bwd(y, x, mean, rstd, None, dbias=only)
    assert none is None and got is only and torch.equal(only, db2)


def test_against_differences(dl):
    """dx, dweight, dbias along random directions against central differences of
    the fp64 loss sum(y dy): fp32 results, so the elementwise bounds apply, and
    1e-6 of the loss' size for the difference (step 1e-4)."""
    B, N, C = 2, 13, 200
    x, g = _data(B, N, 1, C, F, 8, False)
    w, b = (torch.randn((B, C), generator=g, device=DEV) for _ in range(2))
    dy = torch.randn((B, N, 1, C), generator=g, device=DEV)
    y, mean, rstd = dl.layer_norm_fwd(x, w, b, eps=1e-5)
    grads = dl.layer_norm_bwd(dy, x, mean, rstd, w)
    bounds = ref.layer_norm_bwd(dy, x, mean, rstd, w, 400)

    def loss(x_, w_, b_):
        return float((ref.layer_norm(x_, w_, b_, 1e-5, True)[0] * dy.double()).sum())
    args = [t.double() for t in (x, w, b)]
    size = float((ref.layer_norm(x, w, b, 1e-5, True)[0] * dy.double()).abs().sum())
    for i in range(3):
        d = torch.randn(args[i].shape, generator=g, device=DEV, dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-4 * d, args[i] - 1e-4 * d
        diff = (loss(*up) - loss(*down)) / 2e-4
        got = float((grads[i].double().reshape(d.shape) * d).sum())
        assert abs(got - diff) <= float((bounds[i][1] * d.abs()).sum()) + 3e-6 * size


def test_in_place_and_neighbours(dl):
    x, g = _data(2, 40, 2, 64, BF, 12, False)
    y, mean, rstd = dl.layer_norm_fwd(x)
    buf = torch.full((2, 45, 3, 64), 5.0, dtype=BF, device=DEV)
    view = buf[:, :40, :2]
    view.copy_(x)
    z, m2, r2 = dl.layer_norm_fwd(view, out=view)
    assert torch.equal(z, y) and torch.equal(m2, mean) and torch.equal(r2, rstd)
    assert (buf[:, 40:] == 5).all() and (buf[:, :, 2] == 5).all()
    dy = torch.randn(x.shape, generator=g, device=DEV).to(BF)
    w = torch.rand(64, generator=g, device=DEV)
    dx, dw, _ = dl.layer_norm_bwd(dy, x, mean, rstd, w)
    x2, d2 = x.clone(), dy.clone()
    a, dwa, _ = dl.layer_norm_bwd(dy, x2, mean, rstd, w, dx=x2)
    b, dwb, _ = dl.layer_norm_bwd(d2, x, mean, rstd, w, dx=d2)
    assert torch.equal(a, dx) and torch.equal(b, dx) and torch.equal(dw, dwa) and torch.equal(dw, dwb)


def test_rows_of_one_value_and_far_from_zero(dl):
    x = torch.full((1, 3, 1, 512), 1000.0, device=DEV)
    x[0, 1] += torch.randn(512, generator=wl.generator(DEV, 1), device=DEV)[None]
    y, mean, rstd = dl.layer_norm_fwd(x, eps=1e-6)
    want, m, r, bound = ref.layer_norm(x, None, None, 1e-6, True)
    ref.check(y[:, 1], want[:, 1], 1.01 * bound[:, 1] + 2.0 ** -24 * want[:, 1].abs())
    assert (y[:, 0] == 0).all() and (y[:, 2] == 0).all()      # sums of one value are exact here
    assert torch.allclose(rstd[0, 0], torch.full((1,), 1e3, device=DEV), rtol=1e-6)


def test_no_rows(dl):
    x = torch.empty((2, 0, 1, 64), device=DEV)
    y, mean, rstd = dl.layer_norm_fwd(x)
    assert y.numel() == 0
    w = torch.ones((2, 64), device=DEV)
    dw, db = torch.full_like(w, 3.0), torch.full_like(w, 3.0)
    dl.layer_norm_bwd(x, x, mean, rstd, w, dweight=dw, dbias=db)
    torch.cuda.synchronize()
    assert (dw == 0).all() and (db == 0).all()


def test_captured(dl):
    x, g = _data(1, 900, 1, 256, BF, 15, False)
    w = torch.rand(256, generator=g, device=DEV)
    y, mean, rstd = dl.layer_norm_fwd(x, w)
    first = dl.layer_norm_bwd(y, x, mean, rstd, w)
    dx, dw, db = (torch.empty_like(t) for t in first)
    ws = torch.empty(dl.layer_norm_bwd_workspace_bytes(1, 900, 1, 256), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dl.layer_norm_bwd(y, x, mean, rstd, w, dx=dx, dweight=dw, dbias=db, workspace=ws)
    for _ in range(2):
        ws.fill_(0xFF)
        dw.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(first, (dx, dw, db)))


def test_refusals(dl):
    from dit_long_sequence_gb300 import binding as E
    x, _ = _data(2, 4, 1, 64, BF, 17, False)
    with pytest.raises(dl.DitError) as e:
        dl.layer_norm_fwd(x, out_dtype=F)
    assert e.value.status == E.DIT_ERR_UNSUPPORTED
    with pytest.raises(dl.DitError) as e:
        dl.layer_norm_fwd(x, out=torch.empty(x.shape, dtype=BF, pin_memory=True))
    assert e.value.status == E.DIT_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        dl.layer_norm_fwd(x, torch.ones(63, device=DEV))
    with pytest.raises(ValueError):
        dl.layer_norm_fwd(x, torch.ones(64, device=DEV), torch.ones((2, 64), device=DEV))
    with pytest.raises(TypeError):
        dl.layer_norm_fwd(x.half())
    y, mean, rstd = dl.layer_norm_fwd(x)
    with pytest.raises(ValueError):
        dl.layer_norm_bwd(y[:1], x, mean, rstd)
    with pytest.raises(ValueError):
        dl.layer_norm_bwd(y, x, mean[:1], rstd)
