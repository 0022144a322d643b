"""Host-side checks of the window's arithmetic and the forward grid's plan
(csrc/window_span.h, csrc/window_plan.h), compiled into a small program with g++:
what a query sees and the tiles of a block against the definition, key by key."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dit_long_sequence_gb300", "csrc")
HARNESS = r"""
#include <cstdio>
#include "window_plan.h"
int main() {
    dit_window_t d; int first, last, kv, T, H, group; long long items; int sms;
    char what;
    while (std::scanf(" %c", &what) == 1) {
        if (what == 's') {
            if (std::scanf("%d %d %d %d %d %d %d", &d.left, &d.right, &d.sinks, &d.frame, &first, &last, &kv) != 7) return 1;
            const dit::Window w = dit::make_window(d);
            const dit::Span a = dit::span_of(w, first, kv), b = dit::span_of(w, last, kv);
            const dit::KeyTiles t = dit::key_tiles(w, first, last, kv);
            std::printf("%d %d %d %d %d", a.lo, a.hi, b.lo, b.hi, t.n);
            for (int i = 0; i < t.n; ++i) std::printf(" %d", t.at(i));
            std::printf("\n");
        } else {
            double tiles;
            if (std::scanf("%lld %lf %d %d %d", &items, &tiles, &sms, &T, &group) != 5) return 1;
            std::printf("%d %d %d\n", dit::plan_pieces(items, tiles, sms), dit::plan_pieces_few(items, tiles, sms), dit::part_rows_of(T, group));
        }
    }
    return 0;
}
"""


def _cuda_include():
    for d in (os.environ.get("CUDA_HOME", ""), "/usr/local/cuda"):
        if d and os.path.exists(os.path.join(d, "include", "cuda.h")):
            return os.path.join(d, "include")
    return None


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    inc = _cuda_include()
    if shutil.which("g++") is None or inc is None:
        pytest.skip("g++ and the CUDA headers are needed")
    d = tmp_path_factory.mktemp("window")
    (d / "main.cpp").write_text(HARNESS)
    exe = str(d / "main")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    "-I", inc, str(d / "main.cpp"), "-o", exe], check=True, capture_output=True)

    def run(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return [[int(x) for x in line.split()] for line in r.stdout.splitlines()]
    return run


def _sees(p, kv, left, right, sinks, frame):
    f = p // frame
    return [j for j in range(kv) if (right < 0 or j < (f + 1 + right) * frame) and (left < 0 or j >= (f - left) * frame or j < sinks)]


def test_spans_and_tiles_match_the_definition(ask):
    rng = random.Random(1)
    cases = []
    for _ in range(1500):
        left, right = rng.choice((-1, 0, 1, 3, rng.randint(0, 900))), rng.choice((-1, 0, 0, 1, rng.randint(0, 300)))
        frame, sinks = rng.choice((1, 1, 2, 37, 128, 500)), rng.choice((0, 1, 5, 128, 300, 5000))
        first = rng.randint(-400, 1500)
        cases.append((left, right, sinks, frame, first, first + rng.randint(0, 255), rng.choice((0, 1, 127, 128, 129, rng.randint(1, 1400)))))
    for (left, right, sinks, frame, first, last, kv), got in zip(cases, ask("s " + " ".join(map(str, c)) for c in cases)):
        for p, (lo, hi) in ((first, got[:2]), (last, got[2:4])):
            assert 0 <= lo <= hi <= kv
            want = _sees(p, kv, left, right, sinks, frame)
            assert want == sorted(set(range(min(sinks, hi))) | set(range(lo, hi))), (left, right, sinks, frame, p, kv)
        n, tiles = got[4], got[5:]
        need = set()
        for p in range(first, last + 1, max(1, (last - first) // 40)):
            need |= {j // 128 for j in _sees(p, kv, left, right, sinks, frame)}
        need |= {j // 128 for j in _sees(last, kv, left, right, sinks, frame)}
        assert len(tiles) == n and sorted(set(tiles)) == tiles and need <= set(tiles)
        assert not tiles or tiles[-1] * 128 < kv


def test_extreme_arguments_stay_in_range(ask):
    big = 2 ** 30
    cases = [(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, big, -2 ** 29, -2 ** 29 + 5, 2 ** 29), (0, 0, 0, big, 2 ** 29 - 1, 2 ** 29 - 1, 2 ** 29),
             (big, 0, 3, 1, 2 ** 31 - 300, 2 ** 31 - 257, 2 ** 31 - 256)]
    got = ask("s " + " ".join(map(str, c)) for c in cases[:2])
    assert got[0][:4] == [0, 2 ** 29, 0, 2 ** 29] and got[1][:4] == [0, 2 ** 29, 0, 2 ** 29]
    assert ask(["s 0 0 3 1 2147483347 2147483390 2147483391"])[0][:5] == [2147483347, 2147483348, 2147483390, 2147483391, 2]


def test_pieces(ask):
    rng = random.Random(2)
    cases = [(rng.choice((1, 2, 8, 16, 151, 152, 153, 300, 600, 608, 5000)), rng.choice((0.0, 1.0, 2.5, 9.0, 64.0, 1000.0)), 152,
              rng.choice((1, 5, 16, 32, 64, 128, 129, 4000)), rng.choice((1, 2, 3, 5, 8, 128))) for _ in range(400)]
    for (items, tiles, sms, T, group), (f, few, rows) in zip(cases, ask("p " + " ".join(map(str, c)) for c in cases)):
        assert 1 <= f <= 16 and 1 <= few <= 64
        assert f == 1 or (tiles / f >= 2 and items < 2 * sms)
        assert few == 1 or tiles / few >= 2
        assert rows == (T * group if T * group <= 128 and T <= 128 // group else 256)
