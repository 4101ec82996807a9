"""The debug-checks build's predicate of the boxes that the paged kernels load (csrc/checks.h), compiled for the host: coordinates on
both sides of every boundary, and the bytes of boxes of one and of two parts of a row."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <cstdio>
#include "checks.h"
using namespace alibi::check;
static int fails = 0;
#define EXPECT(c) do { if (!(c)) { std::printf("FAIL line %d: %s\n", __LINE__, #c); ++fails; } } while (0)
int main()
{
    // pools of 10 pages of 3 heads of 64 slots of two parts; boxes of 16 slots
    const auto box = [](int slot, int half, int head, int page, int halves) { return page_box(slot, half, head, page, 16, halves, 64, 2, 3, 10); };
    EXPECT(box(0, 0, 0, 0, 2) && box(48, 1, 2, 9, 1) && box(16, 0, 1, 10, 2));  // page 10: zeros
    EXPECT(!box(64, 0, 0, 0, 1) && !box(8, 0, 0, 0, 1) && !box(-16, 0, 0, 0, 1));
    EXPECT(!box(0, 2, 0, 0, 1) && !box(0, 1, 0, 0, 2) && !box(0, -1, 0, 0, 1) && !box(0, 0, 0, 0, 0));
    EXPECT(!box(0, 0, 3, 0, 1) && !box(0, 0, -1, 0, 1) && !box(0, 0, 0, 11, 1) && !box(0, 0, 0, -1, 1));
    EXPECT(!page_box(0, 0, 0, 0, 128, 1, 64, 1, 1, 1));  // a box larger than its page
    // the decode's stage of 16 rows of d = 128 in one box, and a tile of the prefill: both halves
    EXPECT(page_box_bytes(16, 2, 64) == 4096 && page_box_bytes(16, 1, 64) == 2048 && page_box_bytes(128, 2, 64) == 32768);
    EXPECT(page_box_bytes(8, 1, 16) == 256 && page_box_align(8, 16) == 256 && page_box_align(8, 32) == 512);
    EXPECT(page_box_align(8, 64) == 1024 && page_box_align(128, 64) == 1024);
    // a window that ends after the first half has no room for both
    EXPECT(smem_range(4096, page_box_bytes(16, 1, 64), page_box_align(16, 64), 4096, 4096 + 2048));
    EXPECT(!smem_range(4096, page_box_bytes(16, 2, 64), page_box_align(16, 64), 4096, 4096 + 2048));
    EXPECT(smem_range(4096, page_box_bytes(16, 2, 64), page_box_align(16, 64), 4096, 4096 + 4096));
    std::printf(fails ? "%d failures\n" : "ok\n", fails);
    return fails != 0;
}
"""


def test_page_boxes_on_host(tmp_path):
    src, exe = tmp_path / "box.cpp", tmp_path / "box"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "alibi_positional_bias_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_no_caller_states_the_bytes_of_a_box():
    # the check derives them from the box itself: a caller that passed those of one half had the other one unchecked
    csrc = os.path.join(ROOT, "alibi_positional_bias_gb300", "csrc")
    text = open(os.path.join(csrc, "pages.cuh")).read()
    body = text[text.index("void load_box("):text.index("asm volatile(")]
    assert "uint32_t bytes" not in body and "check::page_box(" in body and "check::page_box_bytes(box, halves, WIDTH)" in body
