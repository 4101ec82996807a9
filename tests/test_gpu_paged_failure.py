"""Failure paths of the paged attention kernels, without a GPU fault: a barrier that waits for an arrival that nobody makes lets a
bounded wait of 20 ms run out; the kernel waits for what it has in flight, returns and reports it, and the next call is right."""
import pytest

import paged_ref as ref
from paged_ref import bf16, ints
from test_gpu_fwd_paged import compare as compare_prefill
from test_gpu_paged import case

pytestmark = pytest.mark.gpu

# sequences, length and new tokens: two items of one tile for some CTAs; a few items in parts
TWO_ITEMS, PARTS = (200, 100, 100), (2, 1500, 300)


@pytest.fixture(scope="module")
def ab():
    import alibi_positional_bias_gb300 as ab
    ab.load()
    ab.alibi_check_error()
    return ab


def timed_out(ab):
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_TIMEOUT
    ab.alibi_check_error()  # the status word was cleared


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sizes,barrier", [(TWO_ITEMS, b) for b in range(9)] + [(PARTS, b) for b in (0, 1, 3, 4, 5, 7, 8)])
def test_prefill_timeout_drains_and_context_survives(ab, sizes, barrier, d):
    B, N, T = sizes
    q, k, v = case(B + d, B, 1, 1, T, N, d)
    kp, vp, table = ref.paged(k, v, [N] * B, 16)
    ab.alibi_selftest_fwd_paged_timeout(bf16(q)[1], kp, vp, table, barrier, lens=ints([N] * B), L=N)
    timed_out(ab)
    compare_prefill(ab, q, k, v, [N] * B, [T] * B)
