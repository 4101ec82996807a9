"""Failure paths of the paged attention kernels, without a GPU fault: a barrier that waits for an arrival that nobody makes lets a
bounded wait of 20 ms run out; the kernel waits for what it has in flight, returns and reports it, and the next call is right."""
import pytest

import paged_ref as ref
from paged_ref import bf16, ints
from test_gpu_fwd_paged import compare as compare_prefill
from test_gpu_paged import case, compare as compare_decode

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


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("sizes,barrier", [(TWO_ITEMS, b) for b in (0, 2, 3, 5, 6, 7)] + [(PARTS, b) for b in (0, 1, 4, 7)])
def test_prefill_rows_that_were_not_computed_are_nan(ab, sizes, barrier, d):
    # whatever was in out, and in the scratch of the parts, is not taken for a result
    import torch
    B, N, T = sizes
    q, k, v = case(B + d, B, 1, 1, T, N, d)
    counts = [T - b % 3 for b in range(B)]
    out, lse, args = compare_prefill(ab, q, k, v, [N] * B, counts)
    o, l = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    ab.alibi_selftest_fwd_paged_timeout(*args, barrier, lens=ints([N] * B), count=ints(counts), L=N, out=o, lse=l)
    timed_out(ab)
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    for b, c in enumerate(counts):
        # barriers 2 and 6 stop the CTAs that have two items, the last ones
        if barrier in (2, 6) and b < 2 * ctas - B:
            assert (o[b, :, :c].float() - out[b, :, :c].float()).abs().max() < 0.05
            assert (l[b, :, :c] - lse[b, :, :c]).abs().max() < 0.05
        else:
            assert bool(o[b, :, :c].isnan().all()) and bool(l[b, :, :c].isnan().all()), (b, c)
        assert bool((o[b, :, c:] == 7.0).all()) and bool((l[b, :, c:] == 7.0).all())


# (sequences, KV heads, heads of each, new tokens, length, d): whole chunks, clusters, equal shares that go on from chunk to chunk,
# two and four groups of rows
@pytest.mark.parametrize("B,Hkv,G,T,N,d", [(300, 2, 1, 1, 70, 128), (1, 4, 2, 1, 3000, 128), (1, 1, 1, 1, 9000, 128), (9, 37, 1, 1, 2000, 64),
                                           (3, 2, 3, 4, 500, 64), (5, 2, 5, 5, 700, 32), (2, 1, 40, 1, 300, 16)])
def test_decode_rows_of_a_wait_that_ran_out_are_nan(ab, B, Hkv, G, T, N, d):
    # a sum over some of the keys looks like a result
    q, k, v = case(B + N, B, Hkv, G, T, N, d)
    lens = [N - (7 * b) % (N // 2) for b in range(B)]
    kp, vp, table = ref.paged(k, v, lens, 16)
    out, lse = ab.alibi_selftest_decode_paged_timeout(bf16(q)[1], kp, vp, table, lens=ints(lens), L=N)
    timed_out(ab)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
    compare_decode(ab, q, k, v, lens)
