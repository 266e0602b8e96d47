"""Frequencies of rotary positions as turns in units of 2^-64, without a GPU: the host code against exact rational
arithmetic, to the bound that it states."""
import math
import os
import shutil
import subprocess
from fractions import Fraction

import pytest

import attention_attn_fwd_08_gb300 as A
from attention_attn_fwd_08_gb300 import build

MAIN = r"""
#include <cstdio>
#include "turns.cuh"
int main() {
    double f;
    while (scanf("%la", &f) == 1)
        printf("%llu\n", attn::turn_fraction(attn::two_mul(attn::Two{f, 0}, attn::kTurnsPerRadian)));
}
"""


def test_frequencies_are_right_to_the_stated_bound(tmp_path):
    nvcc = build.nvcc()
    if not (os.path.exists(nvcc) or shutil.which(nvcc)):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "turns.cu", tmp_path / "turns"
    src.write_text(MAIN)
    subprocess.run([nvcc] + build.ARCH + ["-std=c++17", "-I" + build.CSRC, "-o", str(exe), str(src)], check=True)
    freqs = [0.0, 1.0, 2.0 ** 32, 2.0 ** 31 + 0.3, 7.1, 1e-9, 1e-300, math.pi, 2.0 ** -60, 2.0 ** -64]
    for theta in (10000.0, 500000.0, 1000000.0, 3.7):
        for d in (20, 64, 128, 256):
            freqs += A.attn_rope_freqs(d, theta).inv_freq
    out = subprocess.run([str(exe)], input="\n".join(f.hex() for f in freqs), capture_output=True, text=True, check=True).stdout
    got = [int(x) for x in out.split()]
    assert len(got) == len(freqs)
    # 1 / (2 pi) to 2^-200, by Machin's formula for pi in integers
    one = 1 << 240
    arctan = lambda k: sum((1 if i % 2 == 0 else -1) * (one // k ** (2 * i + 1) // (2 * i + 1)) for i in range(120))
    turn = Fraction(one, 2 * 4 * (4 * arctan(5) - arctan(239)))
    worst = 0
    for f, g in zip(freqs, got):
        d = (Fraction(f) * turn * 2 ** 64 - g) % 2 ** 64
        worst = max(worst, float(min(d, 2 ** 64 - d)))
    # one rounding; the product itself is right to 2^-104 of up to 2^30 turns, twice for the constant: 2^-9 units
    assert worst <= 0.5 + 2.0 ** -9, worst
