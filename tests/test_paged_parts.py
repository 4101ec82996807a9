"""How the prefill over pages cuts its work (csrc/paged_parts.h): the rules, compiled for the host, against the choices that the header's
tables of measurements state."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "alibi_positional_bias_gb300", "csrc")
SMS = 152
PROGRAM = r"""
#include <cstdio>
#include "paged_parts.h"
using namespace alibi::paged;
int main()
{
    int BH, G, T, L;
    while (std::scanf("%d %d %d %d", &BH, &G, &T, &L) == 4) {
        const int items = BH * ((T + 255) / 256), rest = items % 152;
        std::printf("%d %d %d\n", parts_of(rest, BH, T, T, L, 152).parts, together(BH, G, T, L, 152), rest);
    }
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("parts")
    src, exe = d / "parts.cpp", d / "parts"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        return [tuple(int(x) for x in line.split()) for line in out if line]
    return ask


def table():
    return open(os.path.join(CSRC, "paged_parts.h")).read()


def test_the_parts_of_the_measured_cases(rule):
    rows = re.findall(r"^//   ((?:\d+ x )+)(\d+) of (\d+) .*?\[(\d+)\] ", table(), re.M)
    assert len(rows) == 10
    cases = []
    for heads, T, L, _ in rows:
        BH = 1
        for n in re.findall(r"\d+", heads):
            BH *= int(n)
        cases.append((BH, 1, int(T), int(L)))
    assert [r[0] for r in rule(cases)] == [int(r[3]) for r in rows]


def test_the_heads_of_the_measured_cases(rule):
    rows = re.findall(r"(\d+) x (\d+) \(x (\d+)\) x (\d+) of (\d+) +\[([ta])\]", table())
    assert len(rows) == 12
    cases = [(int(B) * int(Hkv) * int(G), int(G), int(T), int(L)) for B, Hkv, G, T, L, _ in rows]
    assert [r[1] for r in rule(cases)] == [int(r[5] == "t") for r in rows]


def test_every_answer_is_one_that_can_be_launched(rule):
    cases = [(BH * G, G, T, L) for BH in (1, 2, 7, 19, 76, 151, 152, 153, 305, 10000) for G in (1, 2, 9) for T in (1, 127, 128, 129, 1000, 70000)
             for L in (1, 100, 129, 5000, 1 << 24)]
    for (BH, G, T, L), (parts, joined, rest) in zip(cases, rule(cases)):
        assert 1 <= parts <= 16 and (parts == 1 or rest * parts <= 3 * SMS)
        assert not joined or (G > 1 and T <= 128)
