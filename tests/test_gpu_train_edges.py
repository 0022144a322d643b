"""Calls of the training operators at the edges of what their documentation
allows: masks that leave nothing, more tiles than the occupancy bits of a warp
hold, nothing at all, a first call inside a capture, attention forward and
backward at once on two streams."""
import math
import os
import subprocess
import sys

import pytest
import torch

import train_ref as ref
from dit_long_sequence_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dl():
    import dit_long_sequence_gb300 as m
    return m


@pytest.fixture(autouse=True)
def no_wait_ran_out(dl):
    yield
    rc, info = dl.check_watchdog()
    assert rc == 0, info


def _qkv(B, Nq, Nkv, H, D, seed):
    return [wl.randn_bf16((B, n, H, D), seed + i, DEV) for i, n in enumerate((Nq, Nkv, Nkv, Nq))]


@pytest.mark.parametrize("D", [64, 128])
def test_a_mask_that_forbids_everything(dl, D):
    q, k, v, do = _qkv(2, 300, 200, 2, D, 3)
    bits = torch.zeros((1, 300, 8), dtype=torch.int32, device=DEV)
    out, lse = dl.attn_fwd_masked(q, k, v, bits, out_dtype=BF)
    assert bool((lse == -math.inf).all())
    grads = [torch.full_like(t, 3.0) for t in (q, k, v)]
    dl.attn_bwd_masked(q, k, v, out, lse, do, bits, dq=grads[0], dk=grads[1], dv=grads[2])
    assert all(bool((g == 0).all()) for g in grads)


@pytest.mark.parametrize("Nq,Nkv", [(130, 131_500), (262_400, 100)])
def test_more_tiles_than_a_warp_holds_bits_for(dl, Nq, Nkv):
    """Beyond 1,024 key tiles (query items) and 1,024 blocks of 256 rows (key
    items) nothing is skipped, and the mask holds all the same."""
    q, k, v, do = _qkv(1, Nq, Nkv, 1, 64, 11)
    g = wl.generator(DEV, 12)
    words = 4 * ((Nkv + 127) // 128)
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, Nq, words), generator=g, device=DEV, dtype=torch.int32)
    bits &= torch.randint(-2 ** 31, 2 ** 31 - 1, (1, Nq, words), generator=g, device=DEV, dtype=torch.int32)
    bits[:, ::9] = 0
    bits[:, :, : words // 2] = 0          # whole tiles of nothing
    allow = ((bits[0, :, :, None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1).bool().reshape(Nq, -1)[:, :Nkv]
    allow = allow[None, None]
    out, lse = ref.attn_forward(q, k, v, 0.125, allow)
    out, lse = out.to(BF).contiguous(), lse.float().contiguous()
    grads = dl.attn_bwd_masked(q, k, v, out, lse, do, bits)
    want = ref.attn_bwd(q, k, v, out, lse, do, 0.125, allow, None, True)
    for name, got, (w, b) in zip(("dq", "dk", "dv"), grads, want):
        ref.check(got, w, b, name)


def test_nothing_at_all(dl):
    e = torch.empty
    for B, N, H in ((0, 5, 2), (2, 5, 0), (2, 0, 2)):
        q = e((B, N, H, 64), dtype=BF, device=DEV)
        lse = e((B, H, N), device=DEV)
        assert all(g.shape == q.shape for g in dl.attn_bwd(q, q, q, q, lse, q))
        freq, _ = dl.rope_inv_freq(64)
        assert dl.rope(q, freq).shape == q.shape
        w = torch.ones(64, device=DEV)
        y, mean, rstd = dl.layer_norm_fwd(q, w)
        dx, dw, db = dl.layer_norm_bwd(y, q, mean, rstd, w)
        assert dx.shape == q.shape and (B == 0 or bool((dw == 0).all() and (db == 0).all()))


_FIRST = """
import sys, torch
import dit_long_sequence_gb300 as dl
from dit_long_sequence_gb300 import workloads as wl
dev = torch.device("cuda:0")
q, k, v, do, o = (wl.randn_bf16((1, 900, 2, 64), i, dev) for i in range(5))
lse = torch.zeros((1, 2, 900), device=dev) + 7.0
bits = torch.full((1, 900, 32), -1, dtype=torch.int32, device=dev)
w, freq = torch.ones(64, device=dev), dl.rope_inv_freq(64)[0]


def calls():
    y, mean, rstd = dl.layer_norm_fwd(q, w)
    return [*dl.attn_bwd(q, k, v, o, lse, do), *dl.attn_bwd_masked(q, k, v, o, lse, do, bits), y, rstd,
            *dl.layer_norm_bwd(do, q, mean, rstd, w), dl.rope(q, freq)]


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
want = calls()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert dl.check_watchdog()[0] == 0
print("same bits")
"""


def test_the_first_calls_of_a_process_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stderr[-2000:]


def test_forward_and_backward_calls_at_once(dl):
    """Both kernels take a whole SM's tensor memory and most of its shared memory;
    on two streams they share the GPU and neither waits for the other."""
    q, k, v, do = _qkv(1, 2500, 2500, 4, 128, 21)
    p = _qkv(1, 3000, 700, 3, 64, 25)
    o, lse = dl.attn_fwd(q, k, v, out_dtype=BF)
    po, pl = dl.attn_fwd(*p[:3], out_dtype=BF)
    want_b, want_p, want_f = dl.attn_bwd(q, k, v, o, lse, do), dl.attn_bwd(*p[:3], po, pl, p[3]), o
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        with torch.cuda.stream(a):
            got.append((dl.attn_bwd(q, k, v, o, lse, do), want_b))
            got.append((dl.attn_fwd(q, k, v, out_dtype=BF)[:1], (want_f,)))
        with torch.cuda.stream(b):
            got.append((dl.attn_fwd(*p[:3], out_dtype=BF)[:1], (po,)))
            got.append((dl.attn_bwd(*p[:3], po, pl, p[3]), want_p))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g, w in got for x, y in zip(g, w))
