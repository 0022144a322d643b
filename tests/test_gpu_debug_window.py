"""The windowed attention kernel in the debug library: a key tile that its bounds check
refuses ends the CTA's work (copies and a claim in flight are waited for, tensor memory is
released), an O element that it refuses is skipped; the report names the check, and the
next calls are right.  Nothing outside a buffer is touched either way."""
import ctypes
import time

import pytest
import torch

from dit_long_sequence_gb300 import binding as bd
from dit_long_sequence_gb300 import workloads as wl
from test_gpu_paged import ints, make_cache

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
ROLE_LOAD, ROLE_SOFTMAX, BND_KEY, BND_OUT = 3, 1, 102, 105


@pytest.fixture(scope="module")
def dbg():
    lib = bd.load_debug_library()
    lib.dit_check_watchdog(None, None)
    yield lib
    lib.dit_debug_configure(0, 0, 0, 0, 0)


def _status(lib):
    info = (ctypes.c_uint32 * 4)()
    return lib.dit_check_watchdog(torch.cuda.current_stream().cuda_stream, info), list(info)


def _window(left, right, sinks, frame):
    return ctypes.byref(bd.Window(-1 if left is None else left, -1 if right is None else right, sinks, frame))


def make_call(lib, paged, B, T, n, H, Hkv, D, left, sinks, seed):
    """A call of the debug library, its results, and what the product library gives."""
    q = wl.randn_bf16((B, T, H, D), seed, DEV)
    out, lse = torch.zeros((B, T, H, D), dtype=torch.bfloat16, device=DEV), torch.zeros((B, H, T), device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    if paged:
        k, v, table = make_cache([n] * B, 64, Hkv, D, seed)
        lens = ints([n] * B)
        want = bd.attn_fwd_paged(q, k, v, table, lens, left=left, sinks=sinks)
        ws = torch.empty(bd.attn_fwd_paged_workspace_bytes(B, T, H, Hkv, D, 64, table.shape[1], left=left, sinks=sinks) + 16, dtype=torch.uint8, device=DEV)
        cache = bd.PagedCache(k.data_ptr(), v.data_ptr(), bd.Strides4(*k.stride()), bd.Strides4(*v.stride()), k.shape[0], 64, table.data_ptr(),
                              table.stride(0), table.shape[1], lens.data_ptr())
        keep = (q, k, v, table, lens, ws)

        def call():
            return lib.dit_attn_fwd_paged(q.data_ptr(), ctypes.byref(bd.Strides4(*q.stride())), ctypes.byref(cache), None, B, T, H, Hkv, D,
                                          _window(left, 0, sinks, 1), D ** -0.5, out.data_ptr(), bd.DIT_BF16, ctypes.byref(bd.Strides4(*out.stride())),
                                          lse.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    else:
        k, v = (wl.randn_bf16((B, n, Hkv, D), seed + i, DEV) for i in (1, 2))
        want = bd.attn_fwd_window(q, k, v, left=left, sinks=sinks, offset=n - T, out_dtype=torch.bfloat16)
        ws = torch.empty(bd.attn_fwd_window_workspace_bytes(B, T, H, Hkv, D, n, left=left, sinks=sinks, offset=n - T) + 16, dtype=torch.uint8, device=DEV)
        st = bd.AttnStrides(*(bd.Strides4(*t.stride()) for t in (q, k, v, out)))
        keep = (q, k, v, ws)

        def call():
            return lib.dit_attn_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(st), B, T, n, H, Hkv, D, n, _window(left, 0, sinks, 1),
                                           n - T, D ** -0.5, out.data_ptr(), bd.DIT_BF16, lse.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    call.keep = keep
    torch.cuda.synchronize()
    return call, (out, lse), want


def run_short(lib, call, short):
    assert lib.dit_debug_configure(0, 0, 0, 20_000, short) == bd.DIT_OK
    t0 = time.perf_counter()
    try:
        assert call() == bd.DIT_OK
        return *_status(lib), time.perf_counter() - t0
    finally:
        lib.dit_debug_configure(0, 0, 0, 0, 0)


# whole items and pieces (few items), one query tile and two, more items than SMs (claims)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,T,n,H,Hkv,left,sinks", [(1, 1, 3000, 4, 2, None, 0), (40, 1, 900, 16, 8, 500, 3), (1, 300, 300, 2, 2, None, 0),
                                                    (2, 700, 2000, 4, 2, 300, 5), (2, 2500, 2500, 32, 32, 1000, 4)])
@pytest.mark.parametrize("short", ["last tile", "a few tiles", "all"])
def test_a_refused_tile_ends_its_ctas_work(dbg, D, paged, B, T, n, H, Hkv, left, sinks, short):
    call, got, want = make_call(dbg, paged, B, T, n, H, Hkv, D, left, sinks, 7)
    rc, info, took = run_short(dbg, call, {"last tile": (n - 1) % 128 + 1, "a few tiles": min(n, 400), "all": n}[short])
    assert rc == bd.DIT_ERR_BOUNDS and info[2:] == [ROLE_LOAD, BND_KEY], (rc, info)
    assert took < 1.0
    assert call() == bd.DIT_OK and _status(dbg)[0] == bd.DIT_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("paged", [False, True])
def test_a_refused_element_is_skipped(dbg, paged):
    """The last of O's elements, four short: the stores that reach them are skipped, all others made."""
    B, T, n, H, D = 2, 2500, 2560, 32, 64
    call, (out, lse), want = make_call(dbg, paged, B, T, n, H, H, D, 700, 3, 17)
    rc, info, _ = run_short(dbg, call, 4)
    assert rc == bd.DIT_ERR_BOUNDS and info[2:] == [ROLE_SOFTMAX, BND_OUT], (rc, info)
    differs = (out != want[0]).any(-1).nonzero().tolist()
    assert differs == [[B - 1, T - 1, H - 1]] and (out[-1, -1, -1] == 0).all()
    assert call() == bd.DIT_OK and _status(dbg)[0] == bd.DIT_OK
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,N,Nkv,H,Hkv,left,sinks,short", [(1, 300, 300, 4, 2, None, 0, 100), (2, 1500, 1600, 6, 2, 300, 5, 129), (1, 2500, 2500, 16, 16, 500, 130, 2400),
                                                            (1, 260, 1500, 2, 1, 700, 0, 1500)])
def test_a_refused_tile_ends_the_backward_ctas_work(dbg, D, B, N, Nkv, H, Hkv, left, sinks, short):
    """The window's items, pieces and shared heads: key items, query items, or both."""
    q, k, v, do = (wl.randn_bf16((B, n, h, D), 40 + i, DEV) for i, (n, h) in enumerate(((N, H), (Nkv, Hkv), (Nkv, Hkv), (N, H))))
    kw = dict(left=left, sinks=sinks, offset=Nkv - N)
    o, lse = bd.attn_fwd_window(q, k, v, out_dtype=torch.bfloat16, **kw)
    want = bd.attn_bwd_window(q, k, v, o, lse, do, **kw)
    ws = torch.empty(bd.attn_bwd_window_workspace_bytes(B, N, Nkv, H, Hkv, D, Nkv, **kw), dtype=torch.uint8, device=DEV)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    st = bd.AttnBwdStrides(*(bd.Strides4(*t.stride()) for t in (q, k, v, o, do, *grads)))
    torch.cuda.synchronize()

    def call():
        return dbg.dit_attn_bwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), bd.DIT_BF16, lse.data_ptr(), do.data_ptr(), None,
                                       ctypes.byref(st), B, N, Nkv, H, Hkv, D, Nkv, _window(left, 0, sinks, 1), Nkv - N, D ** -0.5,
                                       *(g.data_ptr() for g in grads), bd.DIT_BF16, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    rc, info, took = run_short(dbg, call, short)
    assert rc == bd.DIT_ERR_BOUNDS and info[2:] == [ROLE_LOAD, BND_KEY], (rc, info)
    assert took < 1.0
    assert call() == bd.DIT_OK and _status(dbg)[0] == bd.DIT_OK
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
