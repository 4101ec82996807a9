"""The prefill over the pages where it takes the rows of a group's heads together: few tokens of many heads to a KV head, against
attention in 64 bits within the bounds of tests/paged_ref.py."""
import numpy as np
import pytest

import oracle
import paged_ref as ref
from gpu_helpers import half_ulp_bf16, host64
from paged_ref import bf16, ints
from test_gpu_fwd_paged import check, compare
from test_gpu_paged import case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ab():
    import alibi_positional_bias_gb300 as ab
    ab.load()
    return ab


# (B, Hkv, G, T, N, d): whole blocks of rows, one block and a bit, a block that ends in a head, blocks cut into parts
CASES = [(20, 2, 16, 9, 400, 64), (9, 8, 8, 32, 513, 128), (40, 4, 4, 33, 300, 32), (3, 2, 64, 5, 1000, 16), (1, 2, 16, 24, 3000, 128),
         (2, 1, 40, 17, 2500, 64), (12, 4, 8, 128, 700, 64), (1, 1, 384, 1, 900, 128), (30, 3, 8, 1, 257, 128)]


@pytest.mark.parametrize("B,Hkv,G,T,N,d", CASES)
@pytest.mark.parametrize("slopes", ["usual", "none", "steep"])
def test_shapes(ab, B, Hkv, G, T, N, d, slopes):
    import torch
    q, k, v = case(N + T + G, B, Hkv, G, T, N, d)
    lens = [max(0, N - (37 * b) % N) for b in range(B)]
    counts = [min(n, T - (5 * b) % (T + 1)) for b, n in enumerate(lens)]
    H = Hkv * G
    m = {"usual": None, "none": np.zeros(H, np.float32), "steep": np.geomspace(1e-3, 30.0, H).astype(np.float32)}[slopes]
    out, lse, args = compare(ab, q, k, v, lens, counts, 16, m=None if m is None else m.astype(np.float64), slopes=m, L=N, M=-(-N // 16))
    for _ in range(2):  # the same bits for the same arguments
        o, l = out.clone(), lse.clone()
        ab.alibi_attn_fwd_paged(*args, lens=ints(lens), count=ints(counts), L=N, out=o, lse=l, slopes=m)
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("layout", ref.LAYOUTS)
@pytest.mark.parametrize("S", [8, 64, 1024])
def test_layouts_and_counts_beyond_the_length(ab, layout, S):
    # tokens before the first row see nothing
    q, k, v = case(S, 30, 2, 8, 20, 300, 64)
    lens = [10 * b % 301 for b in range(30)]
    compare(ab, q, k, v, lens, [20 - b % 21 for b in range(30)], S, layout=layout, L=300, M=-(-300 // S))


def test_every_length_of_a_few_tiles(ab):
    N = 300
    q, k, v = case(3, N + 1, 1, 8, 3, N, 64)
    compare(ab, q, k, v, list(range(N + 1)), [min(3, n) for n in range(N + 1)], 16)


@pytest.mark.parametrize("B,G,T,N,at", [(30, 16, 20, 300, 285), (30, 16, 20, 300, 100), (30, 16, 20, 300, 299), (1, 32, 24, 3000, 2990),
                                        (1, 32, 24, 3000, 500)])
def test_infinite_and_nan_rows(ab, B, G, T, N, at):
    import torch
    d, S = 64, 16
    q, k, v = case(N + T, B, 2, G, T, N, d)
    kp, vp, table = ref.paged(k, v, [N] * B, S)
    page, slot, t = int(table[0, at // S]), at % S, max(0, at - (N - T))
    vp[page, 0, slot, 3], vp[page, 0, slot, d - 1] = float("inf"), float("nan")
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, L=N)
    ab.alibi_check_error()
    o = out.float()
    assert not bool(torch.isfinite(o[0, :G, t:, 3]).any()) and bool(torch.isnan(o[0, :G, t:, d - 1]).all())
    v2 = v.copy()
    v2[0, 0, at, 3] = v2[0, 0, at, d - 1] = 0.0
    ro, rl, eo, el = ref.attention(q, k, v2, [N] * B, [T] * B, oracle.slopes(2 * G), weight=2.0 ** -8, chain=16, column=True)
    for e in (3, d - 1):
        o[0, :G, t:, e], ro[0, :G, t:, e] = 0, 0
    assert (np.abs(host64(o) - ro) <= eo + half_ulp_bf16(ro) * 1.02).all()
    assert (np.abs(host64(lse) - rl) <= el).all()
    kp[page, 0, slot] = float("nan")
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, L=N)
    assert bool(torch.isnan(out[0, :G, t:].float()).all()) and bool(torch.isnan(lse[0, :G, t:]).all())
    out[0, :G, t:] = 0
    ro[0, :G, t:] = 0
    assert (np.abs(host64(out) - ro) <= eo + half_ulp_bf16(ro) * 1.02).all()


@pytest.mark.parametrize("lens,counts", [(-1, 20), (301, 20), (300, -1), (300, 21)])
def test_lengths_and_counts_outside_the_bounds(ab, lens, counts):
    import torch
    B, bad = 30, 7
    q, k, v = case(9, B, 2, 16, 20, 300, 64)
    kp, vp, table = ref.paged(k, v, [300] * B, 16)
    L, C = [300] * B, [20 - b % 3 for b in range(B)]
    L[bad], C[bad] = lens, counts
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:3], 7.0, device="cuda")
    ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, lens=ints(L), count=ints(C), L=300, out=out, lse=lse)
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    good = [b for b in range(B) if b != bad]
    check(out[good], lse[good], q[good], k[good], v[good], [300] * (B - 1), [C[b] for b in good], oracle.slopes(32))
    for b in good:
        assert bool((out[b, :, C[b]:] == 7.0).all()) and bool((lse[b, :, C[b]:] == 7.0).all())


@pytest.mark.parametrize("number", [-1, 2 ** 31 - 1])
@pytest.mark.parametrize("B,G,T,N", [(30, 16, 20, 300), (3, 32, 24, 3000)])
def test_page_numbers_that_are_none(ab, number, B, G, T, N):
    q, k, v = case(10, B, 2, G, T, N, 64)
    kp, vp, table = ref.paged(k, v, [N] * B, 32)
    table[1, 3] = number
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, L=N)
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
    good = [b for b in range(B) if b != 1]
    check(out[good], lse[good], q[good], k[good], v[good], [N] * (B - 1), [T] * (B - 1), oracle.slopes(2 * G))


def test_follows_counts_in_a_graph(ab):
    import torch
    B, Hkv, G, T, N, d = 16, 2, 16, 20, 400, 64
    q, k, v = case(11, B, Hkv, G, T, N, d)
    args = (bf16(q)[1], *ref.paged(k, v, [N] * B, 16))
    lens, count = ints([N] * B), ints([T] * B)
    out, lse = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(q.shape[:3], device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ab.alibi_attn_fwd_paged(*args, lens=lens, count=count, out=out, lse=lse)
    for step in (0, 3, 8):
        L, C = [N - (step * 41 * b) % N for b in range(B)], [(T - step * b) % (T + 1) for b in range(B)]
        lens.copy_(ints(L))
        count.copy_(ints(C))
        out.fill_(7.0)
        g.replay()
        ab.alibi_check_error()
        check(out, lse, q, k, v, L, C, oracle.slopes(Hkv * G), step)
        for b in range(B):
            assert bool((out[b, :, C[b]:] == 7.0).all())
