"""Frequencies as fractions of a turn (csrc/turns.h), compiled for the host, against whole-number arithmetic: the angle of the
rotation that alibi_paged_append applies, at every position that a table has room for."""
import os
import random
import subprocess
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cinttypes>
#include <cstdio>
#include "turns.h"
int main()
{
    double f;
    while (std::scanf("%la", &f) == 1) std::printf("%" PRIu64 "\n", alibi::turns_of(f));
}
"""


def two_pi():
    """2 pi to 2^-400, by Machin's formula in whole numbers."""
    one = 1 << 420

    def arctan_of_inverse(n):
        term, total, k = one // n, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total
    return Fraction(8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)), one)


TWO_PI = two_pi()


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    d = tmp_path_factory.mktemp("turns")
    src, exe = d / "turns.cpp", d / "turns"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "alibi_positional_bias_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)

    def ask(fs):
        out = subprocess.run([str(exe)], input="\n".join(float(f).hex() for f in fs), capture_output=True, text=True, check=True)
        return [int(x) for x in out.stdout.split()]
    return ask


def frequencies():
    rng = random.Random(1)
    fs = [0.0, -0.0, 1.0, -1.0, 1e6, -1e6, 999999.9999999999, 900.0, 1e-300, -1e-300, 5e-324, 2.0 ** -70, 6.283185307179586, 0.5, -3.0]
    fs += [10000.0 ** (-2.0 * i / 128) for i in range(64)]
    return fs + [rng.choice((-1, 1)) * 10.0 ** rng.uniform(-20, 6) for _ in range(2000)]


def test_units_of_a_turn(turns):
    fs = frequencies()
    for f, u in zip(fs, turns(fs)):
        off = (Fraction(u, 1 << 64) - Fraction(f) / TWO_PI) % 1
        assert min(off, 1 - off) <= Fraction(2, 1 << 64), f


def test_angles_of_far_positions(turns):
    # the upper 32 bits of n times the fraction, as a float of half turns: off by less than 2^-22 rad, the bound of the header
    fs = [f for f in frequencies() if abs(f) > 1e-3]
    worst = 0
    for f, u in zip(fs, turns(fs)):
        for n in (1, 65537, (1 << 24) - 1):
            left = (u * n >> 32) & 0xffffffff
            half = left - (1 << 32) if left >> 31 else left        # whole number below 2^31 in magnitude
            drop = max(0, abs(half).bit_length() - 24)             # rounded to the 24 bits of a float
            half = round(Fraction(half, 1 << drop)) << drop
            off = (Fraction(half, 1 << 32) - n * Fraction(f) / TWO_PI) % 1
            worst = max(worst, min(off, 1 - off) * TWO_PI)
    assert worst < Fraction(1, 1 << 22), float(worst)
