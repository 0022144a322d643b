"""Windowed attention and the paged cache as they are used and at their edges: a
streaming block's step in a row, evicted and missing pages, captured replays, side
streams, strided views, differences, repeated bits, refusals from Python."""
import math
import subprocess
import sys
import os

import pytest
import torch

import train_ref as ref
import window_ref as win
from dit_long_sequence_gb300 import workloads as wl
from test_gpu_paged import ints, make_cache, run_and_check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CAUSAL = (None, 0, 0, 1)


@pytest.fixture(scope="module")
def dl():
    import dit_long_sequence_gb300 as m
    return m


@pytest.fixture(autouse=True)
def no_wait_ran_out(dl):
    yield
    rc, info = dl.check_watchdog()
    assert rc == 0, info


def rand(shape, seed, s=1.0):
    return (torch.randn(shape, generator=wl.generator(DEV, seed), device=DEV) * s).to(torch.bfloat16)


def test_a_stream_is_generated_frame_by_frame(dl):
    """Rotary positions, append, attention over the cache, frame by frame and then token
    by token, give what one windowed call over the whole sequence gives, and its
    gradients are those of the formulas."""
    B, F, frames, H, Hkv, D, page = 2, 96, 5, 4, 2, 64, 40
    N = F * frames
    w = dict(left=2, right=0, sinks=F, frame=F)
    x = rand((B, N, H + 2 * Hkv, D), 1)
    freq = dl.rope_inv_freq(D)[0]
    qk = dl.rope(x[:, :, :H + Hkv], freq)
    q, k, v = qk[:, :, :H], qk[:, :, H:], x[:, :, H + Hkv:]
    whole, lse = dl.attn_fwd_window(q, k, v, out_dtype=torch.bfloat16, **w)
    allow = win.sees(torch.arange(N, device=DEV), N, 2, 0, F, F, N)[None, None]
    want = win.forward(q, win.shared(k, H), win.shared(v, H), D ** -0.5, allow, True)
    win.check_forward(whole, lse, want)

    width = -(-N // page)
    pages = torch.full((B * width, 2, page, Hkv, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    kc, vc = pages[:, 0], pages[:, 1]
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(2)).view(B, width).to(torch.int32).to(DEV)
    got, got_lse = torch.empty_like(whole), torch.empty_like(lse)
    at = 0
    for n in [F] * (frames - 1) + [1] * 3 + [F - 3]:
        part = slice(at, at + n)
        turned = dl.rope(x[:, part, :H + Hkv], freq, offset=at)
        lens = ints([at + n] * B)
        dl.paged_append(turned[:, :, H:], x[:, part, H + Hkv:], kc, vc, table, lens)
        if n == F:      # a frame sees itself whole; single tokens see what is there of theirs
            o, l = dl.attn_fwd_paged(turned[:, :, :H], kc, vc, table, lens, **w)
        else:
            o, l = dl.attn_fwd_paged(turned[:, :, :H], kc, vc, table, lens, left=None, right=0)
        got[:, part], got_lse[:, :, part] = o, l
        at += n
    torch.cuda.synchronize()
    full = F * (frames - 1)
    win.check_forward(got[:, :full], got_lse[:, :, :full], ((want[0][0][:, :full], want[0][1][:, :full]), (want[1][0][:, :, :full], want[1][1][:, :, :full])))
    causal = win.sees(torch.arange(N, device=DEV), N, *CAUSAL, N)[None, None]
    (o, bo), (l, bl) = win.forward(q, win.shared(k, H), win.shared(v, H), D ** -0.5, causal, True)
    win.check_forward(got[:, full:], got_lse[:, :, full:], ((o[:, full:], bo[:, full:]), (l[:, :, full:], bl[:, :, full:])))

    dout = rand(whole.shape, 3, 0.25)
    grads = dl.attn_bwd_window(q, k, v, whole, lse, dout, **w)
    for name, g, (r, b) in zip(("dq", "dk", "dv"), grads, win.backward(q, k, v, whole, lse, dout, D ** -0.5, allow)):
        ref.check(g, r, b, name)


def test_the_window_call_is_the_plain_call_without_a_window(dl):
    q, k, v = rand((1, 700, 2, 128), 4), rand((1, 900, 2, 128), 5), rand((1, 900, 2, 128), 6)
    allow = torch.ones((1, 1, 700, 900), dtype=torch.bool, device=DEV)
    allow[..., 871:] = False
    want = win.forward(q, k, v, 128 ** -0.5, allow, False)
    for o, l in (dl.attn_fwd_window(q, k, v, right=None, key_valid_len=871), dl.attn_fwd(q, k, v, key_valid_len=871)):
        win.check_forward(o, l, want)


@pytest.mark.parametrize("T,H,Hkv,D", [(1, 4, 2, 128), (3, 16, 2, 64), (200, 4, 2, 128), (90, 6, 1, 64)])
def test_missing_pages_hold_no_keys(dl, T, H, Hkv, D):
    lens = [1100, 700, T, 1500]
    breaks = [(0, 1, -1), (0, 5, -7), (1, 0, 2 ** 31 - 1), (1, 2, 10 ** 6), (2, 0, -1), (3, 3, -2 ** 31), (3, 4, -1), (3, 9, -1)]
    for w in (CAUSAL, (200, 0, 64, 1)):
        run_and_check(dl, lens, [T] * 4, T, H, Hkv, D, 48, w, 21, break_pages=breaks, given_lens=False)


def test_a_table_narrower_than_its_sequences(dl):
    """Positions past the table hold no keys; the queries keep their positions."""
    run_and_check(dl, [500, 90, 4000], [1, 1, 1], 1, 4, 2, 64, 32, (300, 0, 5, 1), 31, width=4, given_lens=False)
    run_and_check(dl, [500, 90, 300], [140, 80, 150], 150, 4, 2, 64, 32, (None, None, 0, 1), 32, width=6)


def test_odd_lengths_on_the_device(dl):
    """Negative lengths, more queries than tokens (queries before position 0 see nothing)."""
    run_and_check(dl, [-5, 3, 10, 0], [2, 7, 9, 4], 8, 4, 2, 64, 16, CAUSAL, 41)
    run_and_check(dl, [-1, 30, 200, 0], [160, 100, 400, 50], 160, 2, 1, 128, 16, (40, 0, 3, 1), 42)


@pytest.mark.parametrize("T", [1, 150])
def test_evicted_tokens_may_be_anything(dl, T):
    """What no query sees any more, NaN in K and V, changes nothing: not its pages, not the
    rest of the pages and tiles that the window begins and the sinks end in."""
    n, page, H, Hkv, D, left, sinks = 1111, 64, 4, 2, 128, 300, 5
    k, v, table = make_cache([n], page, Hkv, D, 51)
    q = rand((1, T, H, D), 52, 1.5)
    call = dict(left=left, sinks=sinks)
    want = dl.attn_fwd_paged(q, k, v, table, ints([n]), **call)
    first = n - T - left
    for j in list(range(sinks, first)) + list(range(n, -(-n // page) * page)):
        p = int(table[0, j // page])
        k[p, j % page], v[p, j % page] = float("nan"), float("inf")
    got = dl.attn_fwd_paged(q, k, v, table, ints([n]), **call)
    torch.cuda.synchronize()
    if T * H // Hkv <= 128:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # (of several blocks, later ones begin later: a block's own unseen keys are what may be anything)
    assert torch.equal(got[0][:, :128 // (H // Hkv)], want[0][:, :128 // (H // Hkv)])


@pytest.mark.parametrize("T,longest", [(1, 3000), (300, 2000)])
def test_one_sequence_many_pieces_repeat_the_same_bits(dl, T, longest):
    k, v, table = make_cache([longest, 40], 16, 2, 64, 61)
    q = rand((2, T, 6, 64), 62, 1.5)
    assert dl.attn_fwd_paged_workspace_bytes(2, T, 6, 2, 64, 16, table.shape[1]) > 0
    lens, ql = ints([longest, 40]), ints([T, min(T, 33)])
    a = dl.attn_fwd_paged(q, k, v, table, lens, q_lens=ql, out=torch.zeros_like(q), lse=torch.zeros((2, 6, T), device=DEV))
    b = dl.attn_fwd_paged(q, k, v, table, lens, q_lens=ql, out=torch.zeros_like(q), lse=torch.zeros((2, 6, T), device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_and_replayed(dl):
    """The whole serving step in one graph, replayed with other lengths and tokens; and a
    training step beside it.  The first calls of this process' shapes are made inside."""
    B, T, H, Hkv, D, page, width = 3, 1, 6, 2, 128, 16, 60
    pages = rand((B * width, 2, page, Hkv, D), 71)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    lens, x = ints([1, 1, 1]), rand((B, T, H + 2 * Hkv, D), 72)
    tq, tk, tv, td = (rand((1, 333, h, 64), 73 + i) for i, h in enumerate((4, 2, 2, 4)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dl.paged_append(x[:, :, H:H + Hkv], x[:, :, H + Hkv:], pages[:, 0], pages[:, 1], table, lens)
        out, lse = dl.attn_fwd_paged(x[:, :, :H], pages[:, 0], pages[:, 1], table, lens, left=500, sinks=3)
        to, tl = dl.attn_fwd_window(tq, tk, tv, left=100, out_dtype=torch.bfloat16)
        tg = dl.attn_bwd_window(tq, tk, tv, to, tl, td, left=100)
    for step, (a, b, c) in enumerate([(1, 5, 17), (700, 2, 130), (960, 959, 128)]):
        lens.copy_(ints([a, b, c]))
        x.copy_(rand(x.shape, 80 + step))
        tq.copy_(rand(tq.shape, 90 + step))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone(), to.clone(), tl.clone(), [g.clone() for g in tg]
        w1 = dl.attn_fwd_paged(x[:, :, :H], pages[:, 0], pages[:, 1], table, lens, left=500, sinks=3)
        w2 = dl.attn_fwd_window(tq, tk, tv, left=100, out_dtype=torch.bfloat16)
        w3 = dl.attn_bwd_window(tq, tk, tv, *w2, td, left=100)
        torch.cuda.synchronize()
        assert all(torch.equal(p, r) for p, r in zip(got[:4], (*w1, *w2))) and all(torch.equal(p, r) for p, r in zip(got[4], w3))
        for i, n in enumerate((a, b, c)):
            at = n - 1
            assert torch.equal(pages[int(table[i, at // page]), 0, at % page], x[i, 0, H:H + Hkv])


def test_on_a_given_stream(dl):
    q, k, v, do = (rand((1, 500, h, 128), 100 + i) for i, h in enumerate((4, 2, 2, 4)))
    kc, vc, table = make_cache([700, 30], 32, 2, 128, 101)
    lens, pq = ints([700, 30]), rand((2, 1, 4, 128), 102)
    torch.cuda.synchronize()
    want = dl.attn_fwd_window(q, k, v, left=90)
    wg = dl.attn_bwd_window(q, k, v, want[0], want[1], do, left=90)
    wp = dl.attn_fwd_paged(pq, kc, vc, table, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dl.attn_fwd_window(q, k, v, left=90, stream=s)
    gg = dl.attn_bwd_window(q, k, v, got[0], got[1], do, left=90, stream=s)
    gp = dl.attn_fwd_paged(pq, kc, vc, table, lens, stream=s)
    dl.paged_append(k[:, :2].expand(2, -1, -1, -1)[:, :1], v[:, :1].expand(2, -1, -1, -1), kc, vc, table, lens, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*want, *wg, *wp), (*got, *gg, *gp)))
    assert torch.equal(kc[int(table[1, 0]), 29], k[0, 0]) and torch.equal(vc[int(table[0, 21]), 699 % 32], v[0, 0])


def test_strided_views_and_given_results(dl):
    B, N, H, Hkv, D = 2, 300, 4, 2, 64
    x = rand((B, N, H + 2 * Hkv + 1, D), 110)
    q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:H + 2 * Hkv]
    big = torch.full((B, N, H + 3, D), 9.0, dtype=torch.bfloat16, device=DEV)
    out = big[:, :, 1:1 + H]
    o, l = dl.attn_fwd_window(q, k, v, left=64, sinks=2, out=out)
    want = dl.attn_fwd_window(q.contiguous(), k.contiguous(), v.contiguous(), left=64, sinks=2, out_dtype=torch.bfloat16)
    assert o is out and torch.equal(out, want[0]) and torch.equal(l, want[1])
    assert (big[:, :, 0] == 9).all() and (big[:, :, 1 + H:] == 9).all()
    do = rand((B, N, H, D), 111)
    dx = torch.full_like(x, 9.0)
    g = dl.attn_bwd_window(q, k, v, out, l, do, left=64, sinks=2, dq=dx[:, :, :H], dk=dx[:, :, H:H + Hkv], dv=dx[:, :, H + Hkv:H + 2 * Hkv])
    wg = dl.attn_bwd_window(q.contiguous(), k.contiguous(), v.contiguous(), want[0], l, do, left=64, sinks=2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(g, wg)) and (dx[:, :, -1] == 9).all()
    # a head-major cache, and new tokens at odd addresses
    kc, vc = (rand((20, Hkv, 16, D), 112 + i).transpose(1, 2) for i in range(2))
    table = torch.arange(20, dtype=torch.int32, device=DEV).view(2, 10)
    odd = rand((2 * 5 * Hkv * D + 1,), 114)[1:].view(2, 5, Hkv, D)
    dl.paged_append(odd, odd, kc, vc, table, ints([37, 160]))
    torch.cuda.synchronize()
    assert all(torch.equal(c[int(table[b, (n - 5 + t) // 16]), (n - 5 + t) % 16], odd[b, t]) for c in (kc, vc) for b, n in enumerate((37, 160)) for t in range(5))


@pytest.mark.parametrize("T,D", [(1, 64), (4, 128), (300, 64), (300, 128)])
@pytest.mark.parametrize("rise", [3.0, -3.0])
def test_scores_that_grow_and_fall(dl, T, D, rise):
    """A row's offset moves tile after tile (or never): scores grow by a hundred log2 units
    a tile and more."""
    n, H, Hkv, page = 1500, 4, 2, 32
    k, v, table = make_cache([n], page, Hkv, D, 170)
    q = rand((1, T, H, D), 171, 0.25)
    q[..., 0] = 8.0
    j = torch.arange(n, device=DEV)
    at = table[0, j // page].long(), j % page
    k[at[0], at[1], :, 0] = (rise * (j if rise > 0 else j - n).float() / 16)[:, None].to(torch.bfloat16)
    kk, vv = k[at][None], v[at][None]
    for w in (CAUSAL, (700, 0, 4, 1)):
        allow = win.sees(torch.arange(n - T, n, device=DEV), n, *w, n)[None, None]
        want = win.forward(q, win.shared(kk, H), win.shared(vv, H), 1.0, allow, True)
        got = dl.attn_fwd_paged(q, k, v, table, ints([n]), left=w[0], sinks=w[2], scale=1.0)
        flat = dl.attn_fwd_window(q, kk, vv, left=w[0], sinks=w[2], offset=n - T, scale=1.0, out_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        win.check_forward(*got, want)
        win.check_forward(*flat, want)


def test_no_keys(dl):
    q = rand((1, 40, 2, 64), 120)
    kv = rand((1, 40, 1, 64), 121)
    out, lse = dl.attn_fwd_window(q, kv, kv, key_valid_len=0)
    assert (out == 0).all() and (lse == -math.inf).all()
    for g in dl.attn_bwd_window(q, kv, kv, out.to(torch.bfloat16), lse, q, key_valid_len=0):
        assert (g == 0).all()
    none = dl.attn_fwd_window(q, kv, kv, offset=-40)                       # queries before the first key
    assert (none[0] == 0).all() and (none[1] == -math.inf).all()
    empty = torch.empty((0, 16, 1, 64), dtype=torch.bfloat16, device=DEV)
    table = torch.zeros((1, 3), dtype=torch.int32, device=DEV)
    for T in (1, 40):
        o, l = dl.attn_fwd_paged(q[:, :T], empty, empty, table, ints([30]))
        assert (o == 0).all() and (l == -math.inf).all()
    dl.paged_append(kv, kv, empty, empty, table, ints([40]))
    assert dl.attn_fwd_window(q[:, :0], kv, kv)[0].shape == (1, 0, 2, 64)


@pytest.mark.parametrize("w", [(None, 0, 0, 1), (20, 0, 3, 1), (1, 0, 0, 16)])
def test_the_gradient_is_that_of_differences(dl, w):
    """Central differences of the fp64 formula, K and V shared by three heads."""
    B, N, H, Hkv, D = 1, 70, 3, 1, 64
    q, k, v, do = rand((B, N, H, D), 130), rand((B, N, Hkv, D), 131), rand((B, N, Hkv, D), 132), rand((B, N, H, D), 133)
    allow = win.sees(torch.arange(N, device=DEV), N, *w, N)[None, None]
    kw = dict(left=w[0], right=w[1], sinks=w[2], frame=w[3])
    out, lse = dl.attn_fwd_window(q, k, v, **kw)
    grads = dl.attn_bwd_window(q, k, v, out, lse, do, grad_dtype=torch.float32, **kw)

    def loss(q, k, v):
        o, _ = ref.attn_forward(q, win.shared(k, H), win.shared(v, H), D ** -0.5, allow)
        return float((o * do.double()).sum())
    want = win.backward(q, k, v, out, lse, do, D ** -0.5, allow, grad_bf16=False)
    for i, (g, (_, bound)) in enumerate(zip(grads, want)):
        d = torch.randn(g.shape, generator=wl.generator(DEV, 140 + i), device=DEV, dtype=torch.float64)
        eps, args = 1e-5, [q.double(), k.double(), v.double()]
        plus, minus = ([a + s * eps * d if j == i else a for j, a in enumerate(args)] for s in (1, -1))
        slope = (loss(*plus) - loss(*minus)) / (2 * eps)
        # (the differences' own error: eps^2 of the third derivative and fp64's rounding over eps)
        assert abs(float((g.double() * d).sum()) - slope) <= float((bound * d.abs()).sum()) + 1e-4 * abs(slope) + 1e-5


def test_python_refusals(dl):
    q, kv = rand((1, 8, 4, 64), 150), rand((1, 8, 2, 64), 151)
    for kw in (dict(left=-1), dict(right=-2), dict(sinks=-1), dict(frame=0)):
        with pytest.raises(ValueError):
            dl.attn_fwd_window(q, kv, kv, **kw)
    with pytest.raises(TypeError):
        dl.attn_fwd_window(q.float(), kv, kv)
    with pytest.raises(ValueError):
        dl.attn_fwd_window(q, kv, kv[:, :7])
    with pytest.raises(dl.DitError):
        dl.attn_fwd_window(q, torch.cat((kv, kv[:, :, :1]), 2), torch.cat((kv, kv[:, :, :1]), 2))      # 4 heads over 3
    with pytest.raises(dl.DitError):
        dl.attn_fwd_window(q, kv, kv, out=q)
    cache, table, lens = rand((4, 16, 2, 64), 152), torch.zeros((1, 4), dtype=torch.int32, device=DEV), ints([8])
    for bad in ((cache, cache[:2], table, lens), (cache, cache, table.long(), lens), (cache, cache, table, lens.long()),
                (cache, cache, table[:, ::2], lens), (cache, cache, table, ints([8, 8])), (cache.float(), cache.float(), table, lens)):
        with pytest.raises((TypeError, ValueError)):
            dl.attn_fwd_paged(q, *bad)
    with pytest.raises(ValueError):
        dl.attn_fwd_paged(q, cache, cache, table, lens, q_lens=ints([1, 2]))
    with pytest.raises(ValueError):
        dl.paged_append(q, q, cache, cache.clone(), table, lens)               # other heads
    with pytest.raises(dl.DitError):
        dl.paged_append(kv, kv, cache, cache, table, lens)                     # K and V at one place
    long = torch.zeros((1, 400), dtype=torch.int32, device=DEV)
    assert dl.attn_fwd_paged_workspace_bytes(1, 1, 4, 2, 64, 16, 400) > 16
    with pytest.raises(dl.DitError):
        dl.attn_fwd_paged(q[:, :1], cache, cache.clone(), long, lens, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_far_pages(dl):
    """A cache whose elements lie beyond 32-bit offsets, read and written at both ends."""
    Hkv, D, page = 8, 128, 256
    pages = 2 ** 32 // (page * Hkv * D) + 40                                # 2^32 elements and more in each tensor: 17 GB
    kc, vc = (torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = ints([[pages - 1, 0, pages - 2, 3]])
    new = rand((1, 900, 2, Hkv, D), 160)
    dl.paged_append(new[:, :, 0], new[:, :, 1], kc, vc, table, ints([900]))
    for T in (1, 200):
        q = rand((1, T, 16, D), 161, 1.5)
        out, lse = dl.attn_fwd_paged(q, kc, vc, table, ints([900]))
        allow = win.sees(torch.arange(900 - T, 900, device=DEV), 900, *CAUSAL, 900)[None, None]
        win.check_forward(out, lse, win.forward(q, win.shared(new[:, :, 0], 16), win.shared(new[:, :, 1], 16), D ** -0.5, allow, True))


def test_the_parity_tests_through_the_debug_library():
    env = dict(os.environ, DIT_ATTN_DEBUG="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_gpu_window.py",
                        "tests/test_gpu_paged.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-1000:]
