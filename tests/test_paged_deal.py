"""How the paged decode deals its work (csrc/paged_deal.h): the rule, compiled for the host."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "paged_deal.h"
using namespace alibi::paged;
int main()
{
    // clusters of two CTAs per SM that 152 SMs in groups of up to 20 hold
    int fit[kMostCluster + 1] = {0, 1};
    for (int c = 2; c <= kMostCluster; ++c) fit[c] = 7 * (40 / c) + 24 / c;
    long long units; int stages, d, groups;
    while (std::scanf("%lld %d %d %d", &units, &stages, &d, &groups) == 4)
        std::printf("%d %d\n", ctas_of_chunk(units, stages, 304, fit, step_us(d, groups)), fit[16]);
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("deal")
    src, exe = d / "deal.cpp", d / "deal"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "alibi_positional_bias_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        return [int(line.split()[0]) for line in out if line]
    return ask


def test_the_ways_of_the_measured_cases(rule):
    # units, stages, d, groups of rows: clusters where a few chunks fill the device, whole chunks where many do, shares between
    # (the fit above is rounder than the device's)
    cases = [(1, 512, 128, 1), (8, 2048, 128, 1), (4, 8192, 128, 1), (640, 256, 128, 1), (333, 512, 128, 1)]
    assert rule(cases) == [0] * 5
    assert all(c > 1 for c in rule([(40, 512, 128, 1), (32, 128, 128, 1), (80, 512, 128, 1), (128, 257, 128, 1), (32, 256, 64, 1)]))
    assert rule([(2560, 512, 128, 1), (160, 256, 128, 1), (6, 4, 64, 1), (10000, 3, 128, 4)]) == [1] * 4


def test_every_answer_is_one_that_can_be_launched(rule):
    cases = [(u, s, d, g) for u in (1, 2, 3, 7, 19, 38, 76, 150, 152, 153, 304, 305, 1000, 10 ** 6, 2 ** 31 - 1)
             for s in (1, 2, 4, 5, 8, 9, 64, 1000, 10 ** 6) for d in (16, 32, 64, 128) for g in (1, 2, 4)]
    for (u, s, d, g), c in zip(cases, rule(cases)):
        assert 0 <= c <= 16
        if c > 1:
            assert c <= -(-s // 4) and u <= 7 * (40 // c) + 24 // c
        if c == 0:
            assert s > 4  # a chunk that one step of a CTA's warps ends is not shared
