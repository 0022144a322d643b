"""Windowed attention and the paged cache at their corners on the GPU: no query heads,
many heads to a K/V head, queries before the first key, what nobody sees."""
import threading

import pytest
import torch

import train_ref as ref
import window_ref as win
from dit_long_sequence_gb300 import workloads as wl
from test_gpu_paged import ints, make_cache, run_and_check

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_without_query_heads_are_zeros(dl, dtype):
    B, N, Hkv, D = 2, 300, 3, 64
    q, kv = rand((B, N, 0, D), 1), rand((B, N, Hkv, D), 2)
    out, lse = dl.attn_fwd_window(q, kv, kv, left=5)
    assert out.shape == (B, N, 0, D) and lse.shape == (B, 0, N)
    dk, dv = (torch.full((B, N, Hkv, D), 9.0, dtype=dtype, device=DEV) for _ in range(2))
    for given in (dict(dk=dk, dv=dv), dict(grad_dtype=dtype)):
        grads = dl.attn_bwd_window(q, kv, kv, out, lse, q, left=5, sinks=2, **given)
        torch.cuda.synchronize()
        assert grads[0].shape == q.shape and all(g.dtype == dtype and (g == 0).all() for g in grads[1:])


def table_of(Nq, Nkv, w, offset, kvl):
    return win.sees(torch.arange(Nq, device=DEV) + offset, Nkv, *w, kvl)[None, None]


WINDOWS = [(None, 0, 0, 1), (100, 3, 4, 1), (1, 0, 70, 48), (None, None, 0, 1)]


# B, Nq, Nkv, H, Hkv, D, offset: 42 tokens a tile down to one; queries before the first key
@pytest.mark.parametrize("w", WINDOWS)
@pytest.mark.parametrize("B,Nq,Nkv,H,Hkv,D,offset", [(2, 70, 200, 96, 2, 64, 130), (1, 5, 300, 128, 1, 128, 295), (1, 33, 140, 65, 1, 64, 107),
                                                      (1, 1, 260, 128, 1, 64, 259), (2, 3, 130, 100, 2, 128, 127),
                                                      (1, 400, 300, 4, 2, 64, -150), (2, 300, 129, 3, 3, 128, -260), (1, 200, 64, 6, 2, 128, -137)])
def test_many_heads_and_negative_positions(dl, w, B, Nq, Nkv, H, Hkv, D, offset):
    left, right, sinks, frame = w
    q, k, v, dout = rand((B, Nq, H, D), 3 + Nq, 1.5), rand((B, Nkv, Hkv, D), 4), rand((B, Nkv, Hkv, D), 5), rand((B, Nq, H, D), 6, 0.25)
    kw = dict(left=left, right=right, sinks=sinks, frame=frame, offset=offset)
    allow, scale = table_of(Nq, Nkv, w, offset, Nkv), D ** -0.5
    out, lse = dl.attn_fwd_window(q, k, v, out_dtype=torch.bfloat16, **kw)
    grads = dl.attn_bwd_window(q, k, v, out, lse, dout, **kw)
    torch.cuda.synchronize()
    win.check_forward(out, lse, win.forward(q, win.shared(k, H), win.shared(v, H), scale, allow, True))
    for name, g, (r, b) in zip(("dq", "dk", "dv"), grads, win.backward(q, k, v, out, lse, dout, scale, allow)):
        ref.check(g, r, b, name)


@pytest.mark.parametrize("w", WINDOWS)
@pytest.mark.parametrize("T,H,Hkv,D,page", [(1, 128, 1, 128, 64), (1, 96, 2, 64, 48), (2, 100, 1, 64, 16), (9, 128, 1, 64, 24), (3, 65, 1, 128, 136),
                                            (50, 96, 2, 128, 1000)])
def test_many_heads_over_pages(dl, w, T, H, Hkv, D, page):
    run_and_check(dl, [T, 300, 1000, max(1, T // 2)], [T, T, max(1, T // 2), T], T, H, Hkv, D, page, w, 9 + T + page)


@pytest.mark.parametrize("T,H,Hkv", [(1, 4, 2), (150, 4, 2), (300, 4, 2), (300, 2, 2), (90, 10, 2)])
@pytest.mark.parametrize("left,sinks", [(300, 5), (300, 0), (40, 200)])
def test_evicted_tokens_change_no_row(dl, T, H, Hkv, left, sinks):
    """What no query of the call sees, NaN and infinite in K and V, changes no bit of any row,
    those of an item's second tile and of later blocks among them."""
    n, page, D = 1111, 64, 128
    k, v, table = make_cache([n], page, Hkv, D, 51)
    q = rand((1, T, H, D), 52, 1.5)
    call = dict(left=left, sinks=sinks)
    want = dl.attn_fwd_paged(q, k, v, table, ints([n]), **call)
    # (the first query, at n - T, sees the keys from n - T - left on)
    at = torch.tensor(list(range(sinks, n - T - left)) + list(range(n, -(-n // page) * page)), device=DEV)
    where = table[0][at // page].long(), at % page
    k[where], v[where] = float("nan"), float("inf")
    got = dl.attn_fwd_paged(q, k, v, table, ints([n]), **call)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("paged", [False, True])
def test_keys_that_a_later_block_no_longer_sees(dl, paged):
    """Each block by itself: keys that only earlier blocks see may hold anything for it."""
    n, page, H, Hkv, D, left, sinks = 1400, 64, 4, 2, 128, 200, 3
    T, rows = 900, 2 * (128 // (H // Hkv))
    k, v, table = make_cache([n], page, Hkv, D, 53)
    q = rand((1, T, H, D), 54, 1.5)
    j = torch.arange(n, device=DEV)
    where = table[0][j // page].long(), j % page

    def run():
        if paged:
            return dl.attn_fwd_paged(q, k, v, table, ints([n]), left=left, sinks=sinks)
        return dl.attn_fwd_window(q, k[where][None], v[where][None], left=left, sinks=sinks, offset=n - T, out_dtype=torch.bfloat16)
    want = run()
    for block in (1, 3, 7):
        first = n - T + block * rows - left             # of the block's keys, the sinks beside
        k0, v0 = k.clone(), v.clone()
        gone = tuple(t[sinks:first] for t in where)
        k[gone], v[gone] = float("inf"), float("nan")
        got = run()
        torch.cuda.synchronize()
        assert torch.equal(got[0][:, block * rows:], want[0][:, block * rows:]) and torch.equal(got[1][..., block * rows:], want[1][..., block * rows:])
        k.copy_(k0)
        v.copy_(v0)


def test_a_hidden_key_may_hold_anything(dl):
    """K at a key that a row does not see meets only a comparison: NaN and infinities at keys of
    the row's own block, V finite there."""
    N, H, Hkv, D = 250, 2, 1, 64
    q, k, v = rand((1, N, H, D), 55, 1.5), rand((1, N, Hkv, D), 56), rand((1, N, Hkv, D), 57)
    want = dl.attn_fwd_window(q, k, v, left=30)
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = k.clone()
        bad[:, 60] = value                              # seen by the queries 60 to 90
        got = dl.attn_fwd_window(q, bad, v, left=30)
        torch.cuda.synchronize()
        rows = [i for i in range(N) if not 60 <= i <= 90]
        assert torch.equal(got[0][:, rows], want[0][:, rows]) and torch.equal(got[1][:, :, rows], want[1][:, :, rows])


def test_two_streams_at_once(dl):
    """The same calls from two threads on two streams, many times over: the results of one alone."""
    B, N, H, Hkv, D, page = 2, 700, 6, 2, 64, 32
    sets = []
    for i in range(2):
        q, k, v, do = (rand((B, N, h, D), 60 + 4 * i + j) for j, h in enumerate((H, Hkv, Hkv, H)))
        kc, vc, table = make_cache([900, 333], page, Hkv, D, 70 + i)
        sets.append((q, k, v, do, kc, vc, table, ints([900, 333]), rand((B, 1, H, D), 80 + i)))

    def step(q, k, v, do, kc, vc, table, lens, one):
        o, l = dl.attn_fwd_window(q, k, v, left=150, sinks=3, out_dtype=torch.bfloat16)
        g = dl.attn_bwd_window(q, k, v, o, l, do, left=150, sinks=3)
        dl.paged_append(k[:, :3], v[:, :3], kc, vc, table, lens)
        return (o, l, *g, *dl.attn_fwd_paged(one, kc, vc, table, lens), *dl.attn_fwd_paged(q[:, :200], kc, vc, table, lens, left=77), kc, vc)
    want = [[t.clone() for t in step(*s)] for s in sets]
    torch.cuda.synchronize()
    got, streams = [None, None], [torch.cuda.Stream() for _ in range(2)]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                got[i] = step(*sets[i])
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert b is not None and all(torch.equal(x, y) for x, y in zip(a, b))


def test_rows_of_a_wider_table(dl):
    """A table that is a view of a wider one, and one row shared by all sequences."""
    k, v, table = make_cache([500, 500], 32, 2, 64, 90)
    wide = torch.full((2, 40), -1, dtype=torch.int32, device=DEV)
    wide[:, 5:5 + table.shape[1]] = table
    view = wide[:, 5:5 + table.shape[1]]
    for T in (1, 140):
        q = rand((2, T, 4, 64), 91 + T)
        a, b = dl.attn_fwd_paged(q, k, v, table, ints([500, 431])), dl.attn_fwd_paged(q, k, v, view, ints([500, 431]))
        c = dl.attn_fwd_paged(q, k, v, table[:1].expand(2, -1), ints([500, 431]))
        d = dl.attn_fwd_paged(q, k, v, table[:1].repeat(2, 1), ints([500, 431]))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for p, r in ((a, b), (c, d)) for x, y in zip(p, r))


def test_host_memory_is_refused(dl):
    """Buffers that are not the device's are refused before anything is enqueued (pinned: no
    regression could fault)."""
    q, kv = rand((1, 140, 4, 64), 95), rand((1, 140, 2, 64), 96)
    cache, table, lens = rand((8, 32, 2, 64), 97), torch.arange(8, dtype=torch.int32, device=DEV).view(1, 8), ints([200])
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, pin_memory=True)
    lse = torch.full((1, 4, 140), float("nan"), pin_memory=True)
    o, l = dl.attn_fwd_window(q, kv, kv, out_dtype=torch.bfloat16)
    calls = [lambda **r: dl.attn_fwd_window(q, kv, kv, **r), lambda **r: dl.attn_fwd_paged(q, cache, cache.clone(), table, lens, **r)]
    for call in calls:
        for r in (dict(out=out), dict(lse=lse)):
            with pytest.raises(dl.DitError):
                call(**r)
    for name, like in (("dq", q), ("dk", kv), ("dv", kv)):
        with pytest.raises(dl.DitError):
            dl.attn_bwd_window(q, kv, kv, o, l, q, **{name: torch.full(like.shape, float("nan"), dtype=torch.bfloat16, pin_memory=True)})
    for bad in ((table.cpu(), lens), (table, lens.cpu())):
        with pytest.raises((TypeError, ValueError)):
            dl.attn_fwd_paged(q, cache, cache.clone(), *bad)
        with pytest.raises((TypeError, ValueError)):
            dl.paged_append(kv, kv, cache, cache.clone(), *bad)
    torch.cuda.synchronize()
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 200])
def test_large_values_under_growing_scores(dl, T, D):
    """V of 2^64 and scores that grow by 32 log2 units a tile, nearly as far as a row's offset
    stands still: the sums before the division stay finite."""
    n, H = 1500, 2
    q, k, v = rand((1, T, H, D), 180, 0.25), rand((1, n, H, D), 181), rand((1, n, H, D), 182) * 2.0 ** 64
    q[..., 0] = 8.0
    k[..., 0] = (torch.arange(n, device=DEV).float() * (0.25 * 0.6931 / 8.0))[None, :, None].to(torch.bfloat16)
    for w in ((None, 0, 0, 1), (900, 0, 4, 1)):
        o, l = dl.attn_fwd_window(q, k, v, left=w[0], sinks=w[2], offset=n - T, scale=1.0)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(o).all())
        win.check_forward(o, l, win.forward(q, k, v, 1.0, table_of(T, n, w, n - T, n), False))


@pytest.mark.parametrize("page", [128, 8192])
@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("left,sinks,frame", [(300, 5, 1), (0, 200, 1000), (0, 3, 50000)])
def test_positions_next_to_2_31(dl, page, T, left, sinks, frame):
    """A table of nearly 2^31 tokens whose entries name a few pages over and over: its last
    tokens appended and attended, and queries past its end."""
    H, Hkv, D = 4, 2, 64
    width = (2 ** 31 - 256) // page
    capacity = width * page
    cache = rand((3, 2, page, Hkv, D), 190)
    table = (torch.arange(width, device=DEV) % 3).to(torch.int32).view(1, width).expand(2, -1)
    lens = ints([capacity, 2 ** 31 - 1])
    new = rand((2, 3, 2, Hkv, D), 191)
    dl.paged_append(new[:, :, 0], new[:, :, 1], cache[:, 0], cache[:, 1], table, lens)
    torch.cuda.synchronize()
    for t in range(3):
        at = capacity - 3 + t
        assert torch.equal(cache[(at // page) % 3, :, at % page], new[0, t])        # (the other sequence's are past the table)
    q = rand((2, T, H, D), 192, 1.5)
    out, lse = dl.attn_fwd_paged(q, cache[:, 0], cache[:, 1], table, lens, left=left, sinks=sinks, frame=frame)
    torch.cuda.synchronize()
    for b, n in enumerate((capacity, 2 ** 31 - 1)):
        p = torch.arange(n - T, n, device=DEV)
        lo = min(int((p[0] // frame - left) * frame), capacity)
        j = torch.cat((torch.arange(min(sinks, lo), device=DEV), torch.arange(lo, capacity, device=DEV)))
        k, v = (cache[(j // page) % 3, i, j % page][None] for i in range(2))
        fp, fj = (p // frame)[:, None], (j // frame)[None]
        allow = ((fj <= fp) & ((fj >= fp - left) | (j < sinks)[None]))[None, None]
        win.check_forward(out[b:b + 1], lse[b:b + 1], win.forward(q[b:b + 1], win.shared(k, H), win.shared(v, H), D ** -0.5, allow, True))
