"""GPU parity of dit_rope with the 64-bit rotation within train_ref's bound (and
half a step of y's type)."""
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


def _check(y, x, freq, pos, pairs, half, mscale=1.0, inverse=False):
    want, bound = ref.rope(x, freq, pos, pairs, half, mscale, inverse)
    rnd = ref.BF16 if y.dtype == BF else 2.0 ** -24
    ref.check(y, want, 1.01 * bound + rnd * want.abs())
    R = 2 * freq.numel()
    assert torch.equal(y[..., R:], x[..., R:])


def _x(shape, dtype, seed, pad=0):
    B, N, H, D = shape
    g = wl.generator(DEV, seed)
    return torch.randn((B, N, H + pad, D), generator=g, device=DEV).to(dtype)[:, :, :H], g


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("B,N,H,D,R,pad", [(1, 1, 1, 64, 64, 0), (2, 37, 3, 128, 96, 2), (1, 300, 20, 128, 128, 0),
                                           (3, 5, 2, 80, 20, 0), (2, 9, 1, 72, 34, 1), (1, 50, 5, 256, 256, 0),
                                           (1, 7, 2, 65, 30, 0), (2, 11, 3, 6, 2, 1), (48, 1, 32, 64, 64, 0)])
def test_matches_the_rotation(dl, half, dtype, B, N, H, D, R, pad):
    x, g = _x((B, N, H, D), dtype, D + R, pad)
    freq, ms = dl.rope_inv_freq(R, scaling="by_parts", factor=4.0, original_len=512)
    pos = torch.randint(-1000, 200_000, (B, N, 1), generator=g, device=DEV, dtype=torch.int32)
    for inverse in (False, True):
        y = dl.rope(x, freq, pos, layout="half" if half else "interleaved", mscale=ms, inverse=inverse)
        torch.cuda.synchronize()
        _check(y, x, freq, pos, (R // 2,), half, ms, inverse)


def test_default_and_one_dimensional_positions_and_offset(dl):
    x, _ = _x((2, 130, 2, 64), BF, 4)
    freq, _ = dl.rope_inv_freq(64)
    pos = torch.arange(130, dtype=torch.int32, device=DEV)
    a = dl.rope(x, freq)
    _check(a, x, freq, pos[None, :, None], (32,), False)
    assert torch.equal(a, dl.rope(x, freq, pos)) and torch.equal(a, dl.rope(x, freq, pos - 77, offset=77))
    whole = dl.rope(x, freq, offset=5)
    one = torch.cat([dl.rope(x[:, i:i + 1], freq, offset=5 + i) for i in range(0, 130, 43)], 1)
    assert torch.equal(one, whole[:, ::43])          # a token by itself, as in the whole sequence


def test_video_axes_match_the_table_form(dl):
    """Three axes over the latent grid: the same rotation as
    qkv_norm_rope_to_head_major's fp32 tables (rope_tables_3d), q and k of the
    stacked buffer in one call."""
    grid, H, D = (4, 6, 10), 3, 128
    N = 240
    qkv = wl.randn_bf16((1, N, 3, H, D), 6, DEV)
    pairs = (16, 24, 24)
    freq = torch.cat([dl.rope_inv_freq(2 * p)[0] for p in pairs])
    t, h, w = torch.meshgrid(*(torch.arange(n) for n in grid), indexing="ij")
    pos = torch.stack((t, h, w), -1).reshape(1, N, 3).to(torch.int32).to(DEV)
    x = qkv[:, :, :2].flatten(2, 3)
    y = dl.rope(x, freq, pos, axis_pairs=pairs)
    _check(y, x, freq, pos, pairs, False)
    cos, sin = wl.rope_tables_3d(grid, D, device=DEV)
    q, k, _ = dl.qkv_norm_rope_to_head_major(qkv, rope_cos=cos, rope_sin=sin)
    both = torch.cat((q, k), 1).transpose(1, 2)
    # the two round the same values, whose fp32 errors may put a few on either side of a rounding boundary
    assert float((both == y).float().mean()) > 0.99


def test_far_positions_lose_nothing(dl):
    """Positions up to 2^31 - 1 against Python's exact integer reduction."""
    import math
    from fractions import Fraction
    R = 8
    freq, _ = dl.rope_inv_freq(R)
    pos = [2 ** 31 - 1, -2 ** 31, 1_000_003, 123_456_789]
    x = torch.zeros((1, len(pos), 1, R), device=DEV)
    x[..., 0::2] = 1.0
    y = dl.rope(x, freq, torch.tensor(pos, dtype=torch.int32, device=DEV)).cpu().double()
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    for n, p in enumerate(pos):
        for i in range(R // 2):
            ang = float((Fraction(float(freq[i])) * p) % two_pi)
            # the frequency over 2 pi in fp64 is off by 2^-52 of itself: |pos| * freq * 2^-52 rad; and 2^-20 as above
            tol = 2.0 ** -20 + abs(p) * float(freq[i]) * 2.0 ** -52
            assert abs(float(y[0, n, 0, 2 * i]) - math.cos(ang)) <= tol
            assert abs(float(y[0, n, 0, 2 * i + 1]) - math.sin(ang)) <= tol


def test_inverse_is_the_transpose_and_undoes(dl):
    x, g = _x((2, 33, 4, 96), F, 21)
    z = torch.randn(x.shape, generator=g, device=DEV)
    freq, ms = dl.rope_inv_freq(64, scaling="by_parts", factor=16.0)
    for layout in ("interleaved", "half"):
        kw = dict(layout=layout, offset=99_991)
        fx, bz = dl.rope(x, freq, mscale=ms, **kw).double(), dl.rope(z, freq, mscale=ms, inverse=True, **kw).double()
        # <R x, z> = <x, R^T z>, each side within 2^-19 of sum |x| |z| over the pairs
        size = float((x.double().abs().sum(-1) * z.double().abs().sum(-1)).sum()) * ms
        assert abs(float((fx * z.double()).sum() - (x.double() * bz).sum())) <= 2.0 ** -18 * size
        back = dl.rope(dl.rope(x, freq, **kw), freq, inverse=True, **kw)
        pair = x.abs().amax(-1, keepdim=True).double()
        assert bool(((back - x).double().abs() <= 2.0 ** -17 * pair).all())


def test_in_place_neighbours_streams_and_capture(dl):
    buf = torch.full((2, 60, 3, 4, 64), 9.0, dtype=BF, device=DEV)
    buf[:, :50, :2] = wl.randn_bf16((2, 50, 2, 4, 64), 31, DEV)
    freq, _ = dl.rope_inv_freq(48)
    x = buf[:, :50, :2].flatten(2, 3)
    assert x.data_ptr() == buf.data_ptr()
    want = dl.rope(x, freq, layout="half")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = dl.rope(x, freq, layout="half", stream=side)
    torch.cuda.synchronize()
    assert torch.equal(on_side, want)
    keep = x.clone()
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dl.rope(x, freq, layout="half", out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(x, keep)
    dl.rope(x, freq, layout="half", out=x)
    torch.cuda.synchronize()
    assert torch.equal(x, want) and (buf[:, 50:] == 9).all() and (buf[:, :, 2] == 9).all()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D,R", [(128, 26), (192, 166), (128, 20), (40, 36), (64, 62), (48, 2), (256, 250), (8, 6), (184, 184)])
def test_half_layout_of_any_pairs_in_and_out_of_place(dl, dtype, D, R):
    """Halves that begin inside 16 bytes, chunks that hold both halves or the end
    of the turned channels; the same bits in place, and in a view that leaves
    its neighbours alone."""
    x, g = _x((2, 333, 5, D), dtype, D + R, 1)
    freq, _ = dl.rope_inv_freq(R)
    y = dl.rope(x, freq, layout="half", offset=17)
    pos = torch.arange(17, 350, dtype=torch.int32, device=DEV)[None, :, None]
    _check(y, x, freq, pos, (R // 2,), True)
    buf = torch.full((2, 340, 7, D), 4.0, dtype=dtype, device=DEV)
    dl.rope(x, freq, layout="half", offset=17, out=buf[:, 3:336, 1:6])
    assert torch.equal(buf[:, 3:336, 1:6], y)
    rest = buf.clone()
    rest[:, 3:336, 1:6] = 4.0
    assert (rest == 4.0).all()
    z = x.clone()
    dl.rope(z, freq, layout="half", offset=17, out=z)
    assert torch.equal(z, y)


def test_refusals(dl):
    from dit_long_sequence_gb300 import binding as E
    x, _ = _x((1, 4, 2, 64), BF, 41)
    freq, _ = dl.rope_inv_freq(64)
    with pytest.raises(dl.DitError) as e:
        dl.rope(x, freq, out=torch.empty(x.shape, dtype=BF, pin_memory=True))
    assert e.value.status == E.DIT_ERR_INVALID_ARG
    with pytest.raises(dl.DitError):
        dl.rope(x[..., :32], freq)                          # more rotated channels than the head has
    with pytest.raises(dl.DitError):
        dl.rope(x, freq, axis_pairs=(16, 16))               # two axes need positions
    with pytest.raises(ValueError):
        dl.rope(x, freq, torch.zeros((1, 4, 2), dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        dl.rope(x, freq.to(DEV))
    with pytest.raises(TypeError):
        dl.rope(x, freq, torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        dl.rope(x, freq, layout="other")
