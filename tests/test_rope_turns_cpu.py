"""Rotary frequencies as 64-bit fractions of a turn (csrc/rope_turns.h, host
code) against exact rational arithmetic."""
import os
import random
import struct
import subprocess
from fractions import Fraction

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234136")
MAIN = """
#include <cstdio>
#include <cstring>
#include "rope_turns.h"
int main() {
    unsigned long long u;
    while (std::scanf("%llx", &u) == 1) {
        double w;
        std::memcpy(&w, &u, 8);
        std::printf("%llx\\n", static_cast<unsigned long long>(dit::turns_per_step(w)));
    }
}
"""


def test_to_the_last_bit(tmp_path):
    rng = random.Random(5)
    values = [0.0, 1.0, -1.0, 0.5, 3.75, 6.283185307179586, 6.283185307179587, 1e-4, 1e-300, 5e-324, 2.0 ** 59, -0.3]
    values += [10000.0 ** (-i / 64) for i in range(64)]
    values += [rng.choice((-1, 1)) * rng.random() * 2.0 ** rng.randint(-70, 59) for _ in range(2000)]
    src, exe = tmp_path / "turns.cpp", tmp_path / "turns"
    src.write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "dit_long_sequence_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    text = "\n".join(struct.pack(">d", v).hex() for v in values)
    got = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
    assert len(got) == len(values)
    for v, g in zip(values, got):
        turns = Fraction(v) / TWO_PI * 2 ** 64
        off = (int(g, 16) - turns) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        # half a step for the rounding; 128 digits of 1 / 2 pi are |v| 2^-128 of a turn short
        assert off <= Fraction(1, 2) + abs(Fraction(v)) * Fraction(1, 2 ** 64), v
