"""GPU parity of dit_paged_append and dit_attn_fwd_paged: copies bit for bit, attention
with the 64-bit formulas within the bounds window_ref derives."""
import math

import pytest
import torch

import window_ref as win
from dit_long_sequence_gb300 import workloads as wl

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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make_cache(lens, page, Hkv, D, seed, width=None, fill=None):
    """(k_cache, v_cache, table): every sequence's pages shuffled, a few pages over."""
    g = wl.generator(DEV, seed)
    need = [-(-max(n, 0) // page) for n in lens]
    width = max(need + [1]) if width is None else width
    total = sum(need) + 3
    cache = torch.randn((total, 2, page, Hkv, D), generator=g, device=DEV).to(torch.bfloat16)
    order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), width), 2 ** 31 - 1, dtype=torch.int32)      # entries past the pages are never used
    for b, n in enumerate(need):
        for i in range(n):
            p = order.pop()
            if i < width:
                table[b, i] = p
    k, v = cache[:, 0], cache[:, 1]
    if fill is not None:        # stale rows behind a sequence's last token, and pages of nobody
        for b, n in enumerate(lens):
            if n > 0 and n % page and n // page < width:
                k[int(table[b, n // page]), n % page:] = fill
                v[int(table[b, n // page]), n % page:] = fill
        for i in order:
            k[i], v[i] = fill, fill
    return k, v, table.to(DEV)


def expect(q, k, v, table, lens, q_lens, w, scale, out_bf16):
    """Per sequence with queries: its number, how many, what they must give."""
    B, T, H, D = q.shape
    for b in range(B):
        n, m = max(lens[b], 0), min(max(q_lens[b], 0), T)
        if m == 0:
            continue
        cap = min(n, table.shape[1] * k.shape[1])
        kk, there = win.gathered(k, table[b], cap)
        vv, _ = win.gathered(v, table[b], cap)
        kk, vv = (torch.where(there[:, None, None], t, torch.zeros_like(t)) for t in (kk, vv))
        pos = torch.arange(m, device=DEV) + n - m
        allow = (win.sees(pos, cap, *w, cap) & there[None, :])[None, None]
        yield b, m, win.forward(q[b:b + 1, :m], win.shared(kk[None], H), win.shared(vv[None], H), scale, allow, out_bf16)


def run_and_check(dl, lens, q_lens, T, H, Hkv, D, page, w, seed, out_dtype=torch.bfloat16, fill=float("nan"), width=None, break_pages=(),
                  given_lens=True):
    B = len(lens)
    k, v, table = make_cache(lens, page, Hkv, D, seed, width, fill)
    for b, i, value in break_pages:
        table[b, i] = value
    q = (torch.randn((B, T, H, D), generator=wl.generator(DEV, seed + 1), device=DEV) * 1.5).to(torch.bfloat16)
    out = torch.full((B, T, H, D), 77.0, dtype=out_dtype, device=DEV)
    lse = torch.full((B, H, T), 55.0, device=DEV)
    left, right, sinks, frame = w
    got = dl.attn_fwd_paged(q, k, v, table, ints(lens), q_lens=ints(q_lens) if given_lens else None, left=left, right=right, sinks=sinks,
                            frame=frame, out=out, lse=lse)
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is lse
    for b in range(B):
        m = min(max(q_lens[b], 0), T)
        assert (out[b, m:] == 77.0).all() and (lse[b, :, m:] == 55.0).all()
    for b, m, want in expect(q, k, v, table, lens, q_lens, w, D ** -0.5, out_dtype == torch.bfloat16):
        win.check_forward(out[b:b + 1, :m], lse[b:b + 1, :, :m], want)


WINDOWS = [(None, 0, 0, 1), (100, 0, 4, 1), (0, 0, 0, 1), (2, 0, 50, 50), (None, None, 0, 1), (1, 1, 300, 96)]


@pytest.mark.parametrize("w", WINDOWS)
@pytest.mark.parametrize("H,Hkv,D,page", [(2, 2, 128, 64), (8, 1, 64, 16), (6, 2, 128, 48), (4, 4, 64, 256), (10, 2, 128, 8)])
def test_single_tokens(dl, w, H, Hkv, D, page):
    lens = [1, 2, 17, 128, 129, 700, 1500, 0, 333]
    run_and_check(dl, lens, [1] * len(lens), 1, H, Hkv, D, page, w, 5 + page)


@pytest.mark.parametrize("w", WINDOWS)
@pytest.mark.parametrize("T,H,Hkv,D,page", [(5, 8, 2, 128, 64), (16, 4, 1, 64, 24), (33, 3, 1, 128, 80), (128, 2, 2, 64, 32), (300, 2, 1, 128, 128),
                                            (611, 5, 1, 64, 48)])
def test_chunks(dl, w, T, H, Hkv, D, page):
    lens = [T, 3 * T + 5, 40, 1200, max(1, T // 2), 900]
    q_lens = [T, T, min(T, 40), T // 2 + 1, max(1, T // 2), 0]
    run_and_check(dl, lens, q_lens, T, H, Hkv, D, page, w, 7 + T, out_dtype=torch.float32 if page == 80 else torch.bfloat16)


@pytest.mark.parametrize("T,Hkv,D,page,given", [(1, 8, 128, 64, False), (7, 3, 64, 8, True), (300, 2, 128, 48, True), (1, 1, 8, 16, True)])
def test_append(dl, T, Hkv, D, page, given):
    lens = [T, T + 5, 2 * T + 100, 1000, 0, T // 2]
    new = [T, max(0, T - 1), T, T + 9, 1, T] if given else [T] * 6      # counts above T are T; tokens before position 0 are dropped
    k, v, table = make_cache(lens, page, Hkv, D, 3 + T)
    qkv = torch.randn((len(lens), T, 3, Hkv, D), device=DEV).to(torch.bfloat16)
    want_k, want_v = k.clone(), v.clone()
    for b, n in enumerate(lens):
        m = min(max(new[b], 0), T)
        for t in range(m):
            at = n - m + t
            if at >= 0:
                want_k[int(table[b, at // page]), at % page] = qkv[b, t, 1]
                want_v[int(table[b, at // page]), at % page] = qkv[b, t, 2]
    dl.paged_append(qkv[:, :, 1], qkv[:, :, 2], k, v, table, ints(lens), new_lens=ints(new) if given else None)
    torch.cuda.synchronize()
    assert torch.equal(k, want_k) and torch.equal(v, want_v)
