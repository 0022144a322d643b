"""The attention backward kernel in the debug library: a tile that its bounds
check refuses ends the CTA's work (no copy, no further items), the report names
the check, and the next calls are right.  With the rows the check allows
shortened, the last tiles of an item fail it; nothing outside a buffer is
touched either way."""
import ctypes
import os
import re
import subprocess
import sys
import time

import pytest
import torch

from dit_long_sequence_gb300 import binding as bd
from dit_long_sequence_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = torch.device("cuda:0")
ROLE_LOAD, BND_KEY = 3, 102


@pytest.fixture(scope="module")
def dbg():
    lib = bd.load_debug_library()
    lib.dit_check_watchdog(None, None)
    yield lib
    lib.dit_debug_configure(0, 0, 0, 0, 0)


def _status(lib):
    info = (ctypes.c_uint32 * 4)()
    return lib.dit_check_watchdog(torch.cuda.current_stream().cuda_stream, info), list(info)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("Nq,Nkv,short", [(300, 255, 100), (255, 300, 100), (2500, 2500, 2400), (130, 1500, 129)])
def test_a_refused_tile_ends_its_ctas_work(dbg, D, masked, Nq, Nkv, short):
    """In key items, in query items, in both, and with nothing left to load."""
    B, H = 2, 3
    q, k, v, do = (wl.randn_bf16((B, n, H, D), 70 + i, DEV) for i, n in enumerate((Nq, Nkv, Nkv, Nq)))
    o, lse = bd.attn_fwd(q, k, v, out_dtype=torch.bfloat16)
    words = 4 * ((Nkv + 127) // 128)
    bits = torch.full((1, Nq, words), -1, dtype=torch.int32, device=DEV)
    want = bd.attn_bwd_masked(q, k, v, o, lse, do, bits) if masked else bd.attn_bwd(q, k, v, o, lse, do)
    ws = torch.empty(bd.attn_bwd_workspace_bytes(B, Nq, Nkv, H, D, Nkv, masked), dtype=torch.uint8, device=DEV)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    st = bd.AttnBwdStrides(*(bd.Strides4(*t.stride()) for t in (q, k, v, o, do, *grads)))

    def call():
        head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), bd.DIT_BF16, lse.data_ptr(), do.data_ptr(), None,
                ctypes.byref(st), B, Nq, Nkv, H, D, Nkv)
        tail = (D ** -0.5, *(g.data_ptr() for g in grads), bd.DIT_BF16, ws.data_ptr(), ws.numel(),
                torch.cuda.current_stream().cuda_stream)
        if masked:
            return dbg.dit_attn_bwd_masked(*head, bits.data_ptr(), 0, words, Nq, *tail)
        return dbg.dit_attn_bwd(*head, *tail)
    assert dbg.dit_debug_configure(0, 0, 0, 20_000, short) == bd.DIT_OK
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    try:
        assert call() == bd.DIT_OK
        rc, info = _status(dbg)
    finally:
        dbg.dit_debug_configure(0, 0, 0, 0, 0)
    assert rc == bd.DIT_ERR_BOUNDS and info[2:] == [ROLE_LOAD, BND_KEY], (rc, info)
    assert time.perf_counter() - t0 < 1.0
    assert call() == bd.DIT_OK and _status(dbg)[0] == bd.DIT_OK
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_the_parity_tests_through_the_debug_library():
    env = dict(os.environ, DIT_ATTN_DEBUG="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu",
                        "-k", "formulas or chunks or fused or no_keys", "tests/test_gpu_attn_bwd.py"], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) >= 30, r.stdout[-500:]
