"""Host-side checks of what the windowed kernels' grids are made of (csrc/window_span.h,
window.h, window_plan.h, bwd_plan.h), compiled into a small program with g++: the queries
that a backward key item streams and the order of the forward items against their
definitions, the plans' means, pieces and workspaces."""
import os
import random
import shutil
import subprocess

import pytest

from test_window_plan_cpu import CSRC, ROOT, _cuda_include, _sees

HARNESS = r"""
#include <cstdio>
#include "bwd_plan.h"
int main() {
    char what;
    while (std::scanf(" %c", &what) == 1) {
        dit_window_t d;
        if (what == 'g') {                      // order of the items
            dit::WindowArgs a{};
            int late;
            if (std::scanf("%d %d %d %d", &a.B, &a.Hkv, &a.n_blk, &late) != 4) return 1;
            dit::order_items(a, late);
            for (int i = 0; i < a.B * a.Hkv * a.n_blk; ++i) {
                int b, h, blk;
                dit::place(a, static_cast<uint32_t>(i), b, h, blk);
                std::printf("%d %d %d ", b, h, blk);
            }
        } else if (what == 'l') {
            double first, mean;
            long long heads, blocks;
            int sms;
            if (std::scanf("%lf %lf %lld %lld %d", &first, &mean, &heads, &blocks, &sms) != 5) return 1;
            std::printf("%d", dit::late_blocks(first, mean, heads, blocks, sms));
        } else if (what == 'd') {               // division by a fixed number
            unsigned n, by, rem;
            if (std::scanf("%u %u", &n, &by) != 2) return 1;
            const unsigned q = dit::FastDiv(by).divmod(n, rem);
            std::printf("%u %u", q, rem);
        } else {
            if (std::scanf("%d %d %d %d", &d.left, &d.right, &d.sinks, &d.frame) != 4) return 1;
            const dit::Window w = dit::make_window(d);
            if (what == 'q') {                  // queries of a key tile
                long long k0, k1;
                int n, offset;
                if (std::scanf("%lld %lld %d %d", &k0, &k1, &n, &offset) != 4) return 1;
                const dit::QueryRange r = dit::query_range(w, k0, k1, w.sinks, n, offset);
                std::printf("%lld %lld %lld %lld", (long long)r.first, (long long)r.end, (long long)r.full, (long long)r.full_end);
            } else if (what == 't') {           // spans and the number of tiles alone
                int first, last, kv;
                if (std::scanf("%d %d %d", &first, &last, &kv) != 3) return 1;
                const dit::Span a = dit::span_of(w, first, kv), b = dit::span_of(w, last, kv);
                const dit::KeyTiles t = dit::key_tiles(w, first, last, kv);
                std::printf("%d %d %d %d %d %d %d %d", a.lo, a.hi, b.lo, b.hi, t.n, t.ns, t.w0, t.n > 0 ? t.at(t.n - 1) : -1);
            } else if (what == 'm') {           // mean key tiles, in 2^-20
                int T, rows, offset, kv;
                if (std::scanf("%d %d %d %d", &T, &rows, &offset, &kv) != 4) return 1;
                std::printf("%lld", (long long)(dit::mean_key_tiles(w, T, rows, offset, kv) * 1048576.0));
            } else if (what == 'b') {           // the backward plan
                int B, Nq, Nkv, H, Hkv, D, valid, offset, sms;
                if (std::scanf("%d %d %d %d %d %d %d %d %d", &B, &Nq, &Nkv, &H, &Hkv, &D, &valid, &offset, &sms) != 9) return 1;
                const dit::BwdPlan p = dit::plan_attn_bwd_window(B, Nq, Nkv, H, Hkv, D, valid, w, offset, sms);
                std::printf("%d %d %d %lld %lld %lld %d %d %d %lld %lld %lld", p.q_tiles, p.kv_tiles, p.kv_out_tiles, (long long)p.key_items,
                            (long long)p.query_items, (long long)p.q_whole, p.f_kv, p.f_q, p.kv_cut, (long long)p.stat_bytes,
                            (long long)p.part_kv_bytes, (long long)p.part_q_bytes);
            }
        }
        std::printf("\n");
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    inc = _cuda_include()
    if shutil.which("g++") is None or inc is None:
        pytest.skip("g++ and the CUDA headers are needed")
    d = tmp_path_factory.mktemp("ranges")
    (d / "main.cpp").write_text(HARNESS)
    exe = str(d / "main")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    "-I", inc, str(d / "main.cpp"), "-o", exe], check=True, capture_output=True)

    def run(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return [[int(x) for x in line.split()] for line in r.stdout.splitlines()]
    return run


def windows(rng):
    return (rng.choice((-1, 0, 1, 3, rng.randint(0, 500))), rng.choice((-1, 0, 0, 1, rng.randint(0, 200))),
            rng.choice((0, 1, 5, 128, 300, 5000)), rng.choice((1, 1, 2, 37, 128, 400)))


def line(what, *groups):
    return " ".join([what, *(str(x) for g in groups for x in (g if isinstance(g, tuple) else (g,)))])


def test_the_queries_of_a_key_tile_match_the_definition(ask):
    rng = random.Random(3)
    cases = []
    for _ in range(400):
        kv = rng.choice((1, 127, 128, 129, rng.randint(1, 600)))
        k0 = 128 * rng.randint(0, (kv - 1) // 128)
        cases.append((windows(rng), k0, min(k0 + 128, kv), rng.choice((1, 128, rng.randint(1, 500))), rng.choice((0, 0, -300, rng.randint(-500, 700))), kv))
    for (w, k0, k1, n, offset, kv), (first, end, full, full_end) in zip(cases, ask(line("q", w, k0, k1, n, offset) for w, k0, k1, n, offset, _ in cases)):
        left, right, sinks, frame = w
        tile = set(range(k0, k1))
        some, whole = [], []
        for i in range(n):
            seen = tile & set(_sees(offset + i, kv, left, right, sinks, frame))
            if seen:
                some.append(i)
            if seen == tile:
                whole.append(i)
        case = (w, k0, k1, n, offset, kv)
        assert 0 <= first <= n and 0 <= end <= n and 0 <= full <= n and 0 <= full_end <= n, case
        assert (list(range(first, end)) if first < end else []) == some, case       # no query more, none less
        assert set(range(full, full_end)) <= set(whole), case
        if not 0 < sinks - k0 < k1 - k0:        # (a tile that the sinks end in may be seen whole through both)
            assert set(range(full, full_end)) == set(whole), case


def test_spans_at_the_far_end_of_positions(ask):
    """Positions next to 2^31 over a cache, a window of 2^30 tokens."""
    far = 2 ** 31 - 256
    got = ask([line("t", (2 ** 30, 0, 3, 1), far - 44, far - 1, far), line("t", (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 30), far - 44, far - 1, far),
               line("t", (1, 0, 0, 2 ** 30), far - 44, far - 1, far), line("t", (-1, 0, 0, 1), 2 ** 31 - 301, 2 ** 31 - 2, far)])
    lo = far - 44 - 2 ** 30
    assert got[0] == [lo, far - 43, lo + 43, far, 1 + far // 128 - lo // 128, 1, lo // 128, far // 128 - 1]
    assert got[1][:5] == [0, far, 0, far, far // 128]
    assert got[2] == [0, far, 0, far, far // 128, 0, 0, far // 128 - 1]      # the frame before that of the position begins at 0
    assert got[3] == [0, 2 ** 31 - 300, 0, far, far // 128, 0, 0, far // 128 - 1]        # queries past the last key


def test_division_by_a_fixed_number(ask):
    rng = random.Random(4)
    top = 2 ** 31 - 1
    cases = [(n, d) for d in (1, 2, 3, 5, 7, 48, 128, 1536, 2 ** 30 - 1, 2 ** 30, top) for n in (0, 1, d - 1, d, min(d + 1, top), top - 1, top)]
    cases += [(rng.randint(0, top), rng.randint(1, top)) for _ in range(500)] + [(rng.randint(0, top), rng.randint(1, 5000)) for _ in range(500)]
    for (n, d), (q, r) in zip(cases, ask(line("d", n, d) for n, d in cases)):
        assert (q, r) == divmod(n, d), (n, d)


def test_every_block_is_one_item(ask):
    """(batch entry, K/V head, block) each exactly once; the last blocks first within a head, the
    late ones behind all others, the earliest last."""
    cases = [(B, Hkv, n, late) for B in (1, 3) for Hkv in (1, 2, 5) for n in (1, 2, 7, 40) for late in (0, 1, n // 2) if late <= n // 2]
    for (B, Hkv, n, late), got in zip(cases, ask(line("g", *c) for c in cases)):
        items = list(zip(got[::3], got[1::3], got[2::3]))
        assert sorted(items) == [(b, h, k) for b in range(B) for h in range(Hkv) for k in range(n)], (B, Hkv, n, late)
        main = B * Hkv * (n - late)
        assert all(k >= late for _, _, k in items[:main]) and all(k < late for _, _, k in items[main:])
        assert items[:main] == [(b, h, k) for b in range(B) for h in range(Hkv) for k in range(n - 1, late - 1, -1)]
        assert [k for _, _, k in items[main:]] == sorted((k for _, _, k in items[main:]), reverse=True)


def test_late_blocks(ask):
    rng = random.Random(5)
    cases = [(rng.choice((0.0, 1.0, 5.0, 12.0)), rng.choice((1.0, 2.0, 9.9, 10.0, 30.0)), rng.choice((0, 1, 4, 64, 152, 400, 100000)),
              rng.choice((1, 2, 3, 16, 96, 5000)), 152) for _ in range(300)]
    for (first, mean, heads, blocks, sms), (late,) in zip(cases, ask(line("l", *c) for c in cases)):
        assert 0 <= late <= blocks // 2
        if 2 * first > mean or heads == 0:
            assert late == 0
        elif blocks // 2 * heads >= 2 * sms:        # about two turns of the SMs
            assert 2 * sms <= late * heads < 2 * sms + heads
        else:
            assert late == blocks // 2


def blocks_tiles(w, T, rows, offset, kv):
    """Key tiles of every block of `rows` queries, from the definition."""
    out = []
    for first in range(0, T, rows):
        seen = set()
        for i in range(first, min(first + rows, T)):
            seen |= {j // 128 for j in _sees(offset + i, kv, *w)}
        out.append(len(seen))
    return out


def test_mean_key_tiles(ask):
    """Up to 32 blocks the mean of all (a window's tiles, and those between two queries' windows)."""
    rng = random.Random(6)
    cases = [(windows(rng), rng.randint(1, 700), rng.choice((2, 84, 128, 256)), rng.randint(-200, 300), rng.randint(1, 900)) for _ in range(60)]
    cases = [c for c in cases if -(-c[1] // c[2]) <= 32]
    assert len(cases) > 30
    for (w, T, rows, offset, kv), (mean,) in zip(cases, ask(line("m", *c) for c in cases)):
        want = blocks_tiles(w, T, rows, offset, kv)
        assert abs(mean / 2 ** 20 - sum(want) / len(want)) < 1e-5, (w, T, rows, offset, kv)


def test_the_backward_plan(ask):
    """Pieces within their limits, workspaces that hold them, the sinks' tiles first; a piece of
    a common key item or of a query item no longer than about the even share."""
    rng = random.Random(7)
    cases = [((1023, 0, 16, 1), 1, 4096, 4096, 1, 1, 64, 4096, 0, 152), ((3, 0, 384, 384), 1, 6144, 6144, 8, 8, 128, 6050, 0, 152),
             ((-1, 0, 0, 1), 1, 11040, 11040, 16, 4, 128, 11040, 0, 152), ((5, 0, 3, 1), 2, 0, 300, 4, 2, 64, 0, 0, 152)]
    for _ in range(60):
        n = rng.choice((1, 100, 700, 2500))
        past = rng.choice((0, 0, 500))
        hkv = rng.choice((1, 2, 5))
        cases.append((windows(rng), rng.randint(1, 3), n, n + past, hkv * rng.choice((1, 3, 8)), hkv, rng.choice((64, 128)),
                      rng.randint((n + past) // 2, n + past), past, 152))
    for case, got in zip(cases, ask(line("b", *c) for c in cases)):
        w, B, Nq, Nkv, H, Hkv, D, valid, offset, sms = case
        q_tiles, kv_tiles, out_tiles, key_items, query_items, q_whole, f_kv, f_q, kv_cut, stat, part_kv, part_q = got
        assert (q_tiles, kv_tiles, out_tiles) == (-(-Nq // 128), -(-valid // 128), -(-Nkv // 128)), case
        assert (key_items, query_items) == (B * Hkv * out_tiles, B * H * q_tiles)
        assert 1 <= f_kv <= 64 and 1 <= f_q <= 64 and q_whole == (query_items if f_q == 1 else 0)
        assert stat >= 2 * 4 * 128 * B * H * q_tiles + 4 and stat % 256 == 0
        assert part_kv >= (B * Hkv * kv_cut * f_kv * 2 * 128 * D * 4 if f_kv > 1 else 0) and part_kv % 256 == 0
        assert part_q >= (query_items * f_q * 128 * D * 4 if f_q > 1 else 0) and part_q % 256 == 0
        sink_tiles = min(-(-w[2] // 128), kv_tiles)
        assert kv_cut in ((0, out_tiles, sink_tiles) if Nq else (0,)), case
        if f_kv > 1:
            assert kv_cut > 0
        if not Nq or not kv_tiles:
            assert f_kv == f_q == 1 and kv_cut == 0
            continue
        per_query = blocks_tiles(w, Nq, 128, offset, valid) if valid * Nq <= 2 ** 21 else None
        if per_query is None:
            continue
        share = 7 * B * H * sum(per_query) / sms
        # (or pieces of two to three tiles; the plan samples nine tiles, whose neighbours may see some more)
        assert 3 * max(per_query) / f_q <= max(1.02 * share, 9) + 3 * (1 + len(per_query) // 8) or f_q == 64, case
