"""The training operators in corners of what their documentation allows that the
other tests do not reach."""
import ctypes
import math
import subprocess
import threading
import time
import types
from fractions import Fraction

import pytest
import torch

import train_ref as ref
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


@pytest.mark.parametrize("tx,ty,spread", [(F, F, 0.01), (F, BF, 0.01), (BF, BF, 8.0)])
@pytest.mark.parametrize("B,N,H,C", [(1, 64, 1, 500), (2, 40, 1, 4096), (1, 50, 3, 128), (1, 30, 1, 5120), (1, 20, 1, 4097)])
def test_backward_of_rows_far_from_zero(dl, B, N, H, C, tx, ty, spread):
    """Rows around 1,000.  x - mean is one rounding of the difference and its
    product with rstd another, so xh is good to 2^-23 of itself, however far the
    mean is: train_ref's bounds with |xh| in the place of (|x| + |mean|) rstd."""
    g = wl.generator(DEV, 7 + C)
    x = (1000.0 + spread * torch.randn((B, N, H, C), generator=g, device=DEV)).to(tx)
    w = 1 + 0.3 * torch.randn(C, generator=g, device=DEV)
    _, mean, rstd = dl.layer_norm_fwd(x, w, out_dtype=ty)
    dy = torch.randn(x.shape, generator=g, device=DEV).to(ty)
    dx, dw, db = dl.layer_norm_bwd(dy, x, mean, rstd, w)
    x64, d, r, w64 = x.double(), dy.double(), rstd.double()[..., None], w.double()
    xh = (x64 - mean.double()[..., None]) * r
    gr = d * w64
    c1, c2 = gr.mean(-1, keepdim=True), (gr * xh).mean(-1, keepdim=True)
    want = r * (gr - c1 - xh * c2)
    bound = 64 * ref.EPS32 * r * (gr.abs() + gr.abs().mean(-1, keepdim=True) + 2 * xh.abs() * (gr * xh).abs().mean(-1, keepdim=True))
    ref.check(dx, want, 1.01 * bound + (ref.BF16 if tx == BF else 2.0 ** -24) * want.abs(), "dx")
    chain = B * N * H // 100 + 300      # as in the layer norm's own test
    ref.check(dw, (d * xh).sum((0, 1, 2)), ref.EPS32 * (chain + 4) * (d * xh).abs().sum((0, 1, 2)) + 1e-30, "dweight")
    ref.check(db, d.sum((0, 1, 2)), ref.EPS32 * chain * d.abs().sum((0, 1, 2)) + 1e-30, "dbias")


# ---------------------------------------------------------------- rotary positions

def test_far_offsets(dl):
    """Offsets far past 32 bits, frequencies above one and below zero: each is
    held to 2^-65 of a turn a step, so an angle is off by 2 pi |position| 2^-65,
    and the rotation by 2^-20 besides (train_ref)."""
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    freq = torch.tensor([1.0, 3.75, -0.3, 1e-4, 100.1, 0.7071067811865476], dtype=torch.float64)
    x = torch.zeros((1, 3, 1, 12), device=DEV)
    x[..., 0::2] = 1.0
    pos = torch.tensor([0, 1, -5], dtype=torch.int32, device=DEV)
    for offset in (2 ** 31 + 9, 2 ** 36 + 12_345, -(2 ** 40) - 77, 2 ** 44 + 3):
        for inverse in (False, True):
            y = dl.rope(x, freq, pos, offset=offset, inverse=inverse).cpu().double()
            for n in range(3):
                p = offset + int(pos[n])
                for i in range(6):
                    ang = float((Fraction(float(freq[i])) * p) % two_pi)
                    tol = 2.0 ** -20 + 2 * math.pi * abs(p) * 2.0 ** -65
                    assert abs(float(y[0, n, 0, 2 * i]) - math.cos(ang)) <= tol, (offset, i)
                    sign = -1 if inverse else 1
                    assert abs(float(y[0, n, 0, 2 * i + 1]) - sign * math.sin(ang)) <= tol, (offset, i)


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


@pytest.mark.parametrize("kind", ["frames", "holes"])
@pytest.mark.parametrize("B,Nq,Nkv,H,D,rows,kvl", [(2, 300, 300, 2, 64, 300, 300), (1, 513, 1000, 1, 128, 513, 999), (2, 200, 77, 3, 64, 150, 70)])
def test_a_mask_with_a_gradient_of_the_lse_and_fp32_results(dl, kind, B, Nq, Nkv, H, D, rows, kvl):
    q, k, v, dout, g = _inputs(B, Nq, Nkv, H, D, 17 + Nq)
    m = _mask(kind, B, rows, kvl, g)
    allow = _allow(B, Nq, Nkv, kvl, m)
    out, lse = _forward(q, k, v, 0.11, allow, F)
    dlse = torch.randn((B, H, Nq), generator=g, device=DEV)
    grads = dl.attn_bwd_masked(q, k, v, out, lse, dout, wl.pack_mask_bits(m).to(DEV), dlse=dlse, key_valid_len=kvl, scale=0.11,
                               grad_dtype=F)
    torch.cuda.synchronize()
    _check(grads, q, k, v, out, lse, dout, 0.11, allow, dlse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("grad_dtype", [BF, F])
@pytest.mark.parametrize("N,H", [(333, 3), (1700, 40)])      # items in pieces, whole items
def test_gradients_on_16_byte_boundaries(dl, D, grad_dtype, N, H):
    """Rows a 16-byte multiple apart that is none of 32 bytes: the same bits as
    packed, and nothing beside the rows is touched."""
    B = 1
    q, k, v, dout, _ = _inputs(B, N, N, H, D, 19)
    out, lse = dl.attn_fwd(q, k, v, key_valid_len=N - 3)
    want = dl.attn_bwd(q, k, v, out, lse, dout, key_valid_len=N - 3, grad_dtype=grad_dtype)
    step = D + (8 if grad_dtype == BF else 4)
    bufs = [torch.full((B, N, H, step), -7.0, dtype=grad_dtype, device=DEV) for _ in range(3)]
    views = [b[..., step - D:] for b in bufs]
    assert all(t.data_ptr() % 32 == 16 for t in views)
    dl.attn_bwd(q, k, v, out, lse, dout, key_valid_len=N - 3, dq=views[0], dk=views[1], dv=views[2])
    torch.cuda.synchronize()
    for b, t, w in zip(bufs, views, want):
        assert torch.equal(t, w) and bool((b[..., :step - D] == -7.0).all())


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


# ---------------------------------------------------------------- calls

def _stream_of_memory(t):
    """The stream whose pool a tensor's memory belongs to."""
    at = t.data_ptr()
    found = [s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"]]
    assert len(found) == 1
    return found[0]


@pytest.fixture
def step(dl):
    x, do = wl.randn_bf16((2, 200, 2, 64), 61, DEV), wl.randn_bf16((2, 200, 2, 64), 62, DEV)
    w, freq = torch.ones(64, device=DEV), dl.rope_inv_freq(64)[0]
    o, lse = dl.attn_fwd(x, x, x, out_dtype=BF)
    m = torch.ones((1, 200, 200), dtype=torch.bool)
    bits = wl.pack_mask_bits(m).to(DEV)
    _, mean, rstd = dl.layer_norm_fwd(x, w)
    torch.cuda.synchronize()

    def calls(**kw):
        return [*dl.layer_norm_fwd(x, w, **kw), *dl.layer_norm_bwd(do, x, mean, rstd, w, **kw), dl.rope(x, freq, **kw),
                *dl.attn_bwd(x, x, x, o, lse, do, **kw), *dl.attn_bwd_masked(x, x, x, o, lse, do, bits, **kw)]
    return calls


def test_results_of_a_given_stream_are_that_streams_memory(dl, step):
    """A result that is dropped early must not be handed out to the current
    stream's work while the other stream still writes it, nor may a result reused
    by the other stream be one that the current stream still reads."""
    want = step()
    side = torch.cuda.Stream()
    got = step(stream=side)
    assert {_stream_of_memory(t) for t in got} == {side.cuda_stream}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # dropped while the current stream still has work with it: the given stream does not get it back
    torch.cuda._sleep(200_000_000)
    held = {t.data_ptr() for t in got}
    del got
    again = step(stream=side)
    torch.cuda.current_stream().synchronize()
    assert not held & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    # a stream that is the current one is like none
    with torch.cuda.stream(side):
        same = step(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(same, want))


def test_the_default_stream_given_from_beside_another(dl, step, monkeypatch):
    from dit_long_sequence_gb300 import binding
    want = step()
    real, spaces = binding._calls, []

    def spy(name, at):
        def f(*a):
            spaces.append(a[at])
            return getattr(real, name)(*a)
        return f
    monkeypatch.setattr(binding, "_calls", types.SimpleNamespace(attn_bwd=spy("attn_bwd", 15), norm_bwd=spy("norm_bwd", 9),
                                                               norm_fwd=real.norm_fwd, rope=real.rope))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plain = types.SimpleNamespace(cuda_stream=0)        # any object with a handle
    for given in (torch.cuda.default_stream(), plain):
        spaces.clear()
        with torch.cuda.stream(side):
            got = step(stream=given)
        torch.cuda.synchronize()
        assert len(spaces) == 3 and {_stream_of_memory(t) for t in spaces} == {0}
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_given_results_on_a_given_stream_stay_the_callers(dl):
    x = wl.randn_bf16((1, 50, 2, 64), 63, DEV)
    freq = dl.rope_inv_freq(64)[0]
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert dl.rope(x, freq, out=out, stream=side) is out
    torch.cuda.synchronize()
    assert torch.equal(out, dl.rope(x, freq))


def test_no_memory_left_has_its_own_type(dl):
    x = torch.empty((1, 1, 1, 64), dtype=BF, device=DEV).expand(64, 4096, 64, 64)      # a result of 2 GB
    freq = dl.rope_inv_freq(64)[0]
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 28)) / torch.cuda.get_device_properties(0).total_memory)
    try:
        for call in (lambda: dl.rope(x, freq), lambda: dl.layer_norm_fwd(x)):
            with pytest.raises(torch.OutOfMemoryError):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert dl.rope(x[:1, :4], freq).shape == (1, 4, 64, 64)


_WAITER = """
#include <unistd.h>
volatile int flag = 0;
int wait_for_flag() { for (int i = 0; i < 3000; ++i) { if (flag) return 0; usleep(1000); } return 4; }
"""


def test_other_threads_run_while_a_call_waits(dl, tmp_path):
    """The library's function is replaced by one that waits (3 s at most) for
    another Python thread: a call that kept the interpreter's lock would wait in
    vain, as it would for a full launch queue."""
    from dit_long_sequence_gb300 import binding
    src, lib = tmp_path / "waiter.c", tmp_path / "waiter.so"
    src.write_text(_WAITER)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", str(src), "-o", str(lib)], check=True)
    waiter = ctypes.CDLL(str(lib))
    names = ("dit_attn_bwd", "dit_attn_bwd_masked", "dit_attn_bwd_workspace_bytes", "dit_layer_norm_fwd",
             "dit_layer_norm_bwd", "dit_layer_norm_bwd_workspace_bytes", "dit_rope")
    real = [ctypes.cast(getattr(binding.raw(), n), ctypes.c_void_p).value for n in names]
    wait = ctypes.cast(waiter.wait_for_flag, ctypes.c_void_p).value
    flag = ctypes.c_int.in_dll(waiter, "flag")
    x, w = wl.randn_bf16((1, 8, 2, 64), 64, DEV), torch.ones(64, device=DEV)
    freq = dl.rope_inv_freq(64)[0]
    o, lse = dl.attn_fwd(x, x, x, out_dtype=BF)
    _, mean, rstd = dl.layer_norm_fwd(x, w)
    bits = torch.full((1, 8, 4), -1, dtype=torch.int32, device=DEV)
    dl.rope(x, freq)

    def raise_flag():
        time.sleep(0.05)
        flag.value = 1
    calls = {"dit_rope": lambda: dl.rope(x, freq), "dit_layer_norm_fwd": lambda: dl.layer_norm_fwd(x, w),
             "dit_layer_norm_bwd": lambda: dl.layer_norm_bwd(x, x, mean, rstd, w),
             "dit_attn_bwd": lambda: dl.attn_bwd(x, x, x, o, lse, x),
             "dit_attn_bwd_masked": lambda: dl.attn_bwd_masked(x, x, x, o, lse, x, bits)}
    for name, call in calls.items():
        flag.value = 0
        binding._calls.bind(*(wait if n == name else a for n, a in zip(names, real)))
        t = threading.Thread(target=raise_flag)
        try:
            t.start()
            call()      # (a wait that ran out is a DitError)
        finally:
            binding._calls.bind(*real)
            t.join()


def test_a_given_stream_inside_a_capture(dl, step):
    """A side stream that the captured one forks and joins: its results are of the
    graph's memory, dropped ones among them, and replays give the same bits."""
    want = step()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        step(stream=side)
        got = step(stream=side)
        main.wait_stream(side)
        copies = [t.clone() for t in got]
    for _ in range(3):
        for t in got + copies:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(got, want, copies))


def test_threads_with_streams_of_their_own(dl, step):
    want = step()
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = step()
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    wrong.append(1)
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
