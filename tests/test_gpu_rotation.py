"""The rotation of alibi_paged_append at large frequencies and far positions, against angles reduced in whole numbers."""
from fractions import Fraction

import numpy as np
import pytest

import paged_ref as ref
from gpu_helpers import half_ulp_bf16, host64
from paged_ref import bf16, ints
from test_turns import TWO_PI

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("last", [1 << 24, 5000000, 70000])
def test_large_frequencies_at_far_positions(interleaved, last):
    # the kernel's bound before the store is that of paged_ref.rotated, 2^-20 (|x| + |y|) for an angle off by less than 2^-22;
    # the angles here are exact, their cosines and sines off by 2^-50
    import torch
    import alibi_positional_bias_gb300 as ab
    d, S, H, T = 64, 1024, 2, 5
    pos = last - T
    freqs = np.array([100.0, 900.0, 1000.0, 12345.678, 1e5, 999999.9, 1e6, -1e6, -31.4, 1.0, 27.0, 64.5, 3e4, 2.5e5, -777.0, 1e-3])
    R = 2 * len(freqs)
    table = torch.zeros(1, 16384, dtype=torch.int32, device="cuda")
    table[0, pos // S] = 1
    table[0, (pos + T - 1) // S] = 2 if (pos + T - 1) // S != pos // S else 1
    kp, vp = ref.pools(3, H, S, d, "heads")
    rng = np.random.default_rng(last)
    (k64, k), (_, v) = (bf16(rng.standard_normal((1, H, T, d)) * 2) for _ in range(2))
    ab.alibi_paged_append(k, v, kp, vp, table, pos=ints([pos]), rotate=R, freqs=freqs, interleaved=interleaved)
    ab.alibi_check_error()
    have = host64(torch.stack([kp[int(table[0, j // S]), :, j % S] for j in range(pos, pos + T)], 1))
    angle = np.array([[float(n * Fraction(f) % TWO_PI) for f in freqs] for n in range(pos, pos + T)])
    c, s = np.cos(angle), np.sin(angle)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    want = k64[0].copy()
    want[..., a] = k64[0][..., a] * c - k64[0][..., b] * s
    want[..., b] = k64[0][..., b] * c + k64[0][..., a] * s
    err = np.zeros_like(want)
    err[..., a] = err[..., b] = 2.0 ** -20 * (np.abs(k64[0][..., a]) + np.abs(k64[0][..., b]))
    off = np.abs(have - want)
    assert (off <= err + half_ulp_bf16(want) * (1 + 2.0 ** -6)).all(), (off - err - half_ulp_bf16(want)).max()
