"""The 4-bit KV cache on the host: its layout (csrc/kv4.h against the documented formulas, every byte of a
block used once), the quantisation's own properties, and the entry points' refusals. No device work."""
import ctypes
import os
import shutil
import subprocess
from fractions import Fraction

import numpy as np
import pytest

import alibi_inputs as gen
import alibi_positional_bias_gb300 as ab
import kv4_ref as ref
from alibi_positional_bias_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "alibi_positional_bias_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "kv4.h"
using namespace alibi::kv4;
int main()
{
    for (int d : {16, 32, 64, 128}) {
        const int D = padded(d);
        std::printf("%d %d %d\n", d, D, block_bytes(D));
        for (int r = 0; r < kBlock; ++r) {
            for (int e = 0; e < D; e += 2) std::printf("%d %d\n", key_byte(D, r, e), value_byte(D, r, e));
            for (int n = 0; n < D / kGroup; ++n) std::printf("%d %d\n", scale_byte(D, r, 0, n), scale_byte(D, r, 1, n));
        }
    }
}
"""


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ab.load()


@pytest.fixture(scope="module")
def header_offsets(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("needs g++")
    tmp = tmp_path_factory.mktemp("kv4")
    src, exe = tmp / "p.cpp", tmp / "p"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    return [tuple(map(int, l.split())) for l in subprocess.run([str(exe)], capture_output=True, text=True,
                                                               check=True).stdout.splitlines()]


def test_header_matches_the_documented_layout(header_offsets):
    it = iter(header_offsets)
    for d in (16, 32, 64, 128):
        D = max(d, 32)
        assert next(it) == (d, D, 36 * D)
        used = np.zeros(36 * D, dtype=int)
        for r in range(32):
            for e in range(0, D, 2):
                kb, vb = next(it)
                assert (kb, vb) == (ref.key_byte(D, r, e), ref.value_byte(D, r, e)), (D, r, e)
                used[kb] += 1
                used[vb] += 1
            for n in range(D // 32):
                s = next(it)
                assert s == (ref.scale_byte(D, r, 0, n), ref.scale_byte(D, r, 1, n))
                for o in s:
                    used[o] += 1
                    used[o + 1] += 1
        assert (used == 1).all()  # every byte of a block belongs to one place
    assert next(it, None) is None


def test_block_bytes(lib):
    assert [ab.alibi_kv4_block_bytes(d) for d in (16, 32, 64, 128)] == [1152, 1152, 2304, 4608]
    for d, st in ((0, ab.ALIBI_ERR_INVALID), (-8, ab.ALIBI_ERR_INVALID), (48, ab.ALIBI_ERR_UNSUPPORTED),
                  (256, ab.ALIBI_ERR_UNSUPPORTED)):
        with pytest.raises(ab.AlibiError) as e:
            ab.alibi_kv4_block_bytes(d)
        assert e.value.status == st


def test_quotients_of_bf16_are_ties_or_far_from_them():
    # the claim behind the kernel's rounding: x / s with 8-bit significands is a multiple of 1/2
    # or at least 2^-10 away from one, for |x / s| <= 8 (smaller quotients round to code 8)
    worst = Fraction(1)
    for S in range(128, 256):
        for sh in range(-3, 4):  # x / s = X / S 2^sh
            for X in range(128, 256):
                y = Fraction(X, S) * Fraction(2) ** sh + Fraction(1, 2)
                f = y - (y.numerator // y.denominator)
                if f:
                    worst = min(worst, f, 1 - f)
    assert worst >= Fraction(1, 1024)


def test_reference_properties():
    rng = np.random.default_rng(5)
    x = gen.make_tensor(rng.standard_normal((64, 128)), (64, 128), "bf16").f32.astype(np.float64)
    u, s = ref.quantise(x)
    assert u.min() >= 0 and u.max() <= 15
    y = ref.held(x).reshape(64, 4, 32)
    g = x.reshape(64, 4, 32)
    i = np.abs(g).argmax(-1)
    assert (np.take_along_axis(y, i[..., None], -1) == np.take_along_axis(g, i[..., None], -1)).all()
    off = np.abs(y - g) / np.abs(s)[..., None]
    near = g / -s[..., None] < -7.5  # within s / 2 of -x_m: clamped to code 15
    assert off[~near].max() <= 0.5 and off.max() <= 1.0


def test_the_smoke_check_has_the_definition_of_its_own():
    import __graft_entry__ as entry
    rng = np.random.default_rng(8)
    x = gen.make_tensor(rng.standard_normal((50, 64)), (50, 64), "bf16").f32
    x[:8, 5] *= 2.0 ** np.arange(-4, 4)  # ties and clamped codes too
    x[9], x[10, 32:], x[11, 3], x[11, 4] = 0.0, 2.0 ** -101, 4.0, -4.0
    assert np.array_equal(entry.held_in_4_bits(x), ref.held(x.astype(np.float64)).astype(np.float32))


P = ctypes.c_void_p(0x10000)  # never dereferenced: arguments are checked before any CUDA call
MIS = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)


def test_write_and_read_argument_errors(lib):
    w, r = lib.alibi_kv4_write, lib.alibi_kv4_read
    I, U = ab.ALIBI_ERR_INVALID, ab.ALIBI_ERR_UNSUPPORTED
    for bad in ((None, P, P), (P, None, P), (P, P, None), (MIS, P, P), (P, MIS, P), (P, P, MIS)):
        assert w(*bad, None, None, 1, 1, 1, 32, 64, None) == I
        assert r(bad[2], bad[0], bad[1], None, None, 1, 1, 1, 32, 64, 0, None) == I
    assert w(P, P, P, ODD, None, 1, 1, 1, 32, 64, None) == I
    assert w(P, P, P, None, ODD, 1, 1, 1, 32, 64, None) == I
    for dims, st in (((0, 1, 1, 32, 64), I), ((1, 0, 1, 32, 64), I), ((1, 1, 0, 32, 64), I), ((1, 1, 1, 0, 64), I),
                     ((1, 1, 1, 32, 0), I), ((1, 1, 1, 48, 64), I), ((1, 1, 33, 32, 64), I),
                     ((-1, -1, 1, 32, 64), I), ((1, 1, 1, 32, 48), U), ((1, 1, 1, 32, 256), U),
                     ((1, 257, 1, 32, 64), U), ((1, 1, 1, (1 << 24) + 32, 64), U),
                     ((1 << 24, 128, 1, 32, 64), U)):
        assert w(P, P, P, None, None, *dims, None) == st, dims
        assert r(P, P, P, None, None, *dims, 0, None) == st, dims
    assert r(P, P, P, None, None, 1, 1, 1, 32, 64, 2, None) == I
    assert r(P, P, P, None, None, 1, 1, 1, 32, 64, -1, None) == I


def test_decode_argument_errors(lib):
    f = lib.alibi_attn_decode_kv4
    I, U = ab.ALIBI_ERR_INVALID, ab.ALIBI_ERR_UNSUPPORTED
    ok = (1, 2, 1, 1, 32, 32, 64)
    for ptrs in ((None, P, P, P, P), (P, None, P, P, P), (P, P, P, None, P), (MIS, P, P, P, P), (P, MIS, P, P, P),
                 (P, P, ODD, P, P), (P, P, P, MIS, P), (P, P, P, P, ODD)):
        assert f(*ptrs, *ok, None, None) == I, ptrs
    for dims, st in (((0, 2, 1, 1, 32, 32, 64), I), ((1, 0, 1, 1, 32, 32, 64), I), ((1, 2, 0, 1, 32, 32, 64), I),
                     ((1, 2, 1, 0, 32, 32, 64), I), ((1, 2, 1, 1, 0, 32, 64), I), ((1, 2, 1, 1, 32, 0, 64), I),
                     ((1, 3, 2, 1, 32, 32, 64), I),        # H not a multiple of Hkv
                     ((1, 2, 4, 1, 32, 32, 64), I),
                     ((1, 2, 1, 1, 33, 32, 64), I),        # L beyond the capacity
                     ((1, 2, 1, 1, 32, 40, 64), I),        # capacity not in whole blocks
                     ((1, 2, 1, 17, 32, 32, 64), U), ((1, 2, 1, 1, 32, 32, 96), U), ((1, 512, 1, 1, 32, 32, 64), U),
                     ((1, 2, 1, 1, 32, (1 << 24) + 32, 64), U), ((1 << 26, 128, 1, 1, 32, 32, 64), U)):
        assert f(P, P, None, P, P, *dims, None, None) == st, dims
    for bad in (-1.0, float("nan"), float("inf")):
        m = (ctypes.c_float * 2)(0.5, bad)
        assert f(P, P, None, P, P, *ok, m, None) == I


def test_decode_refuses_more_than_384_query_heads(lib):
    for H, Hkv in ((385, 385), (385, 1), (386, 193), (400, 50)):
        assert lib.alibi_attn_decode_kv4(P, P, None, P, P, 1, H, Hkv, 1, 32, 32, 64, None, None) == ab.ALIBI_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    import torch
    z = torch.zeros(1, 1, 1, 32, dtype=torch.bfloat16)
    c = torch.zeros(1, 1, 1, 1152, dtype=torch.uint8)
    with pytest.raises(ValueError):
        ab.alibi_kv4_write(z, z, c)
    with pytest.raises(ValueError):
        ab.alibi_kv4_read(c, z, z)
    with pytest.raises(ValueError):
        ab.alibi_attn_decode_kv4(z, c)
    for C in (0, -32, 33):
        with pytest.raises(ValueError):
            ab.alibi_kv4_cache(1, 1, C, 64)
