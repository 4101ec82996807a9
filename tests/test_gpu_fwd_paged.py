"""The prefill over the pages (alibi_attn_fwd_paged) against attention in 64 bits within the bounds derived in
tests/paged_ref.py, with weights rounded to bf16 (2^-8) as the dense prefill's are."""
import numpy as np
import pytest

import oracle
import paged_ref as ref
from gpu_helpers import half_ulp_bf16, host64
from paged_ref import bf16, ints
from test_gpu_paged import case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ab():
    import alibi_positional_bias_gb300 as ab
    ab.load()
    return ab


def check(out, lse, q, k, v, lens, counts, m, what=""):
    # the values' products of a row are one chain of 16 keys a step; a weight is rounded to bf16 for them
    ro, rl, eo, el = ref.attention(q, k, v, lens, counts, m, weight=2.0 ** -8, chain=16, column=True)
    go, gl = host64(out), host64(lse)
    for b, c in enumerate(counts):
        o, e, r = go[b, :, :c], eo[b, :, :c], ro[b, :, :c]
        assert np.isfinite(o).all(), what
        lim = e + half_ulp_bf16(r) * (1 + 2.0 ** -6) + 2.0 ** -133
        assert (np.abs(o - r) <= lim).all(), (what, b, (np.abs(o - r) / lim).max())
        none = np.isinf(rl[b, :, :c])
        assert np.array_equal(none, np.isinf(gl[b, :, :c])) and (o[none] == 0).all()
        off = np.abs(gl[b, :, :c][~none] - rl[b, :, :c][~none])
        assert (off <= el[b, :, :c][~none]).all(), (what, b, (off - el[b, :, :c][~none]).max())


def compare(ab, q, k, v, lens, counts, S=16, m=None, slopes=None, L=None, M=None, layout="heads", unused=-1, what=""):
    import torch
    B, H, T = q.shape[:3]
    kp, vp, table = ref.paged(k, v, lens, S, seed=B + S, layout=layout, M=M, unused=unused)
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:3], 7.0, device="cuda")
    qd = bf16(q)[1]
    for b, c in enumerate(counts):
        qd[b, :, c:] = float("nan")
    ab.alibi_attn_fwd_paged(qd, kp, vp, table, lens=ints(lens), count=ints(counts), L=L, out=out, lse=lse, slopes=slopes)
    ab.alibi_check_error()
    check(out, lse, q, k, v, lens, counts, oracle.slopes(H) if m is None else m, what)
    for b, c in enumerate(counts):  # tokens from count on are left as they were
        assert bool((out[b, :, c:] == 7.0).all()) and bool((lse[b, :, c:] == 7.0).all())
    return out, lse, (qd, kp, vp, table)


@pytest.mark.parametrize("d,S", [(16, 8), (32, 16), (64, 16), (128, 64), (128, 16), (64, 1024), (128, 256)])
def test_first_prompts(ab, d, S):
    # prompts from their beginning, of lengths about the tiles' ends
    counts = [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 300, 0]
    q, k, v = case(d + S, len(counts), 1, 2, 300, 300, d)
    compare(ab, q, k, v, counts, counts, S)


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("T", [1, 5, 40, 129, 260])
def test_chunks_that_begin_anywhere(ab, d, T):
    # every place in a tile where a chunk can begin, and chunks that reach past their length
    B, N = 24, 420
    lens = [N - (53 * b) % N for b in range(B)]
    counts = [max(0, T - b % 3) for b in range(B)]
    q, k, v = case(T + d, B, 1, 1, T, N, d)
    compare(ab, q, k, v, lens, counts, 16)


@pytest.mark.parametrize("B,Hkv,G,T,N,d,S", [
    (1, 1, 1, 1000, 1000, 128, 16), (2, 3, 2, 100, 999, 64, 16), (1, 2, 4, 513, 2100, 128, 128), (3, 2, 3, 77, 1025, 32, 32),
    (1, 8, 1, 300, 5000, 128, 512), (2, 1, 9, 256, 700, 64, 8), (1, 3, 5, 17, 20001, 16, 64), (2, 40, 1, 260, 300, 128, 16),
    (70, 3, 1, 20, 100, 64, 16), (1, 1, 384, 30, 140, 16, 16)])
@pytest.mark.parametrize("layout", ["heads", "together"])
def test_shapes(ab, B, Hkv, G, T, N, d, S, layout):
    q, k, v = case(7 * N + d + G, B, Hkv, G, T, N, d)
    lens = [max(1, N - (37 * b) % N) for b in range(B)]
    counts = [min(n, T - (11 * b) % T) for b, n in enumerate(lens)]
    out, lse, args = compare(ab, q, k, v, lens, counts, S, layout=layout, M=-(-N // S) + 2, L=N + 3, unused=2 ** 31 - 1)
    import torch
    for _ in range(2):  # the same bits for the same arguments
        o, l = out.clone(), lse.clone()
        ab.alibi_attn_fwd_paged(*args, lens=ints(lens), count=ints(counts), L=N + 3, out=o, lse=l)
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("layout", ref.LAYOUTS)
@pytest.mark.parametrize("d,S", [(16, 8), (64, 32), (128, 128)])
def test_layouts(ab, layout, d, S):
    import torch
    q, k, v = case(S + d, 2, 3, 2, 150, 300, d)
    out, lse, _ = compare(ab, q, k, v, [300, 217], [150, 90], S, layout=layout)
    plain, plain_lse, _ = compare(ab, q, k, v, [300, 217], [150, 90], S)
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)


def test_without_lengths_or_counts(ab):
    import torch
    q, k, v = case(1, 2, 2, 2, 100, 320, 64)
    kp, vp, table = ref.paged(k, v, [320, 320], 32)
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table)
    ab.alibi_check_error()
    check(out, lse, q, k, v, [320, 320], [100, 100], oracle.slopes(4))
    o, l = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, L=290)
    check(o, l, q, k, v, [290, 290], [100, 100], oracle.slopes(4))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, l = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, stream=stream)
    stream.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)


def test_agrees_with_the_dense_prefill(ab):
    # whole prompts of one length, one key head per query head: what alibi_attn_fwd computes
    q, k, v = case(2, 2, 4, 1, 700, 700, 128)
    out, lse, _ = compare(ab, q, k, v, [700, 700], [700, 700], 64)
    o, l = ab.alibi_attn_fwd(*(bf16(x)[1] for x in (q, k, v)))
    check(o, l, q, k, v, [700, 700], [700, 700], oracle.slopes(4))


def test_more_new_tokens_than_length(ab):
    # queries before the first row see nothing: out 0, lse -inf
    q, k, v = case(3, 4, 2, 2, 300, 200, 64)
    lens, counts = [0, 1, 130, 200], [300, 300, 290, 201]
    out, lse, _ = compare(ab, q, k, v, lens, counts)
    for b, (n, c) in enumerate(zip(lens, counts)):
        assert bool((out[b, :, :c - n] == 0).all()) and bool((lse[b, :, :c - n] == -np.inf).all())


def test_caller_slopes_and_no_bias(ab):
    q, k, v = case(4, 1, 2, 4, 200, 900, 128)
    for m in (np.zeros(8), np.linspace(0.0, 2.0, 8), oracle.slopes(8)[::-1], np.array([1e4, 3e4, 2.7, 2.8, 1, 2, 30, 1e30])):
        m32 = m.astype(np.float32)
        compare(ab, q, k, v, [777], [150], m=m32.astype(np.float64), slopes=m32, what=m)


def test_large_logits(ab):
    # scores of some hundreds in either order along the cache: the maximum moves often
    q, k, v = case(5, 1, 2, 2, 140, 1024, 128)
    ramp = np.linspace(0.0, 20.0, 1024)
    for r in (ramp, ramp[::-1]):
        kk = bf16(k * r[None, None, :, None])[0]
        compare(ab, bf16(4 * q)[0], kk, v, [1001], [139], m=np.zeros(4), slopes=np.zeros(4, np.float32))


@pytest.mark.parametrize("d,S", [(16, 16), (64, 8), (128, 128)])
@pytest.mark.parametrize("N,T,at", [(300, 300, 299), (300, 300, 130), (500, 260, 400), (500, 260, 255), (700, 200, 512)])
def test_infinite_and_nan_rows_that_a_query_does_not_see(ab, d, S, N, T, at):
    # one row's key is NaN and two of its values are not finite: queries before it know nothing of that
    import torch
    q, k, v = case(d + N, 1, 1, 2, T, N, d)
    kp, vp, table = ref.paged(k, v, [N], S)
    page, slot, first = int(table[0, at // S]), at % S, N - T
    t = max(0, at - first)  # the first query that sees the row
    vp[page, 0, slot, 3], vp[page, 0, slot, d - 1] = float("inf"), float("nan")
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, L=N)
    ab.alibi_check_error()
    o = out.float()
    assert not bool(torch.isfinite(o[:, :, t:, 3]).any()) and bool(torch.isnan(o[:, :, t:, d - 1]).all())
    o[:, :, t:, 3] = o[:, :, t:, d - 1] = 0
    # the other elements, and all of the queries before, are those without it
    v2 = v.copy()
    v2[0, 0, at, 3] = v2[0, 0, at, d - 1] = 0.0
    ro, rl, eo, el = ref.attention(q, k, v2, [N], [T], oracle.slopes(2), weight=2.0 ** -8, chain=16, column=True)
    ro[:, :, t:, 3] = ro[:, :, t:, d - 1] = 0
    assert (np.abs(host64(o) - ro) <= eo + half_ulp_bf16(ro) * 1.02).all()
    assert (np.abs(host64(lse) - rl) <= el).all()
    kp[page, 0, slot] = float("nan")
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, L=N)
    assert bool(torch.isnan(out[:, :, t:].float()).all()) and bool(torch.isnan(lse[:, :, t:]).all())
    assert (np.abs(host64(out[:, :, :t]) - ro[:, :, :t]) <= eo[:, :, :t] + half_ulp_bf16(ro[:, :, :t]) * 1.02).all()


@pytest.mark.parametrize("lens,counts,bad", [
    ([300, -1, 300], [200, 200, 200], 1), ([300, 301, 300], [200, 200, 200], 1), ([300, 300, 300], [200, -1, 200], 1),
    ([300, 300, 300], [200, 301, 200], 1), ([300, 2 ** 31 - 1, 300], [200, 2, 200], 1), ([300, 300, -2 ** 31], [1, 1, 0], None)])
def test_lengths_and_counts_outside_the_bounds(ab, lens, counts, bad):
    import torch
    q, k, v = case(9, 3, 2, 2, 300, 300, 64)
    kp, vp, table = ref.paged(k, v, [300] * 3, 16)
    qd = bf16(q)[1]
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:3], 7.0, device="cuda")
    ab.alibi_attn_fwd_paged(qd, kp, vp, table, lens=ints(lens), count=ints(counts), L=300, out=out, lse=lse)
    if bad is None:  # nothing to compute where nothing is new
        ab.alibi_check_error()
    else:
        with pytest.raises(ab.AlibiError) as e:
            ab.alibi_check_error()
        assert e.value.status == ab.ALIBI_ERR_RANGE
        c = counts[bad] if 0 <= counts[bad] <= 300 else 300
        assert bool(out[bad, :, :c].isnan().all()) and bool(lse[bad, :, :c].isnan().all())
        assert bool((out[bad, :, c:] == 7.0).all())
    ab.alibi_check_error()
    good = [b for b in range(3) if b != bad and lens[b] == 300]
    check(out[good], lse[good], q[good], k[good], v[good], [300] * len(good), [counts[b] for b in good], oracle.slopes(4))


@pytest.mark.parametrize("number", [-1, -2 ** 31, 2 ** 31 - 1, "one past"])
@pytest.mark.parametrize("S", [8, 16, 128, 256])
def test_page_numbers_that_are_none(ab, number, S):
    q, k, v = case(10, 3, 2, 2, 150, 600, 64)
    kp, vp, table = ref.paged(k, v, [600] * 3, S)
    table[1, 300 // S] = kp.shape[0] if number == "one past" else number
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, L=600)
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
    check(out[::2], lse[::2], q[::2], k[::2], v[::2], [600] * 2, [150] * 2, oracle.slopes(4))


# (B, Hkv, G, T, N, d): a bound on the lengths far beyond them makes the kernel share few items' tiles among all SMs
SHARED = [(1, 1, 1, 300, 3000, 128), (1, 1, 2, 40, 9000, 64), (3, 2, 2, 260, 1500, 128), (2, 4, 1, 700, 700, 64), (5, 2, 3, 129, 400, 16),
          (1, 1, 1, 1, 5, 128), (40, 4, 1, 30, 300, 64)]


@pytest.mark.parametrize("B,Hkv,G,T,N,d", SHARED)
@pytest.mark.parametrize("spread", ["equal", "ragged", "one long", "longer chunks"])
def test_shared_items(ab, B, Hkv, G, T, N, d, spread):
    import torch
    q, k, v = case(N + B + T, B, Hkv, G, T, N, d)
    lens = {"equal": [N] * B, "ragged": [N - (b * 7919) % N for b in range(B)], "one long": [N] + [b % 9 for b in range(1, B)],
            "longer chunks": [N - (b * 7919) % N for b in range(B)]}[spread]
    counts = [T - (13 * b) % T for b in range(B)]
    if spread != "longer chunks":
        counts = [min(n, c) for n, c in zip(lens, counts)]
    out, lse, args = compare(ab, q, k, v, lens, counts, 32, L=100000, M=-(-100000 // 32), what=spread)
    for _ in range(3):  # the same bits for the same arguments
        o, l = out.clone(), lse.clone()
        ab.alibi_attn_fwd_paged(*args, lens=ints(lens), count=ints(counts), L=100000, out=o, lse=l)
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("N,T,at", [(300, 300, 130), (500, 260, 400), (2000, 260, 1990), (2000, 260, 700), (2000, 260, 1745)])
def test_infinite_and_nan_rows_of_shared_items(ab, N, T, at):
    import torch
    d, S, L = 64, 16, 100000
    q, k, v = case(d + N, 1, 1, 2, T, N, d)
    kp, vp, table = ref.paged(k, v, [N], S, M=-(-L // S))
    page, slot = int(table[0, at // S]), at % S
    t = max(0, at - (N - T))
    vp[page, 0, slot, 3] = float("nan")
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, lens=ints([N]), L=L)
    ab.alibi_check_error()
    o = out.float()
    assert bool(torch.isnan(o[:, :, t:, 3]).all())
    o[:, :, t:, 3] = 0
    v2 = v.copy()
    v2[0, 0, at, 3] = 0.0
    ro, rl, eo, el = ref.attention(q, k, v2, [N], [T], oracle.slopes(2), weight=2.0 ** -8, chain=16, column=True)
    ro[:, :, t:, 3] = 0
    assert (np.abs(host64(o) - ro) <= eo + half_ulp_bf16(ro) * 1.02).all()
    assert (np.abs(host64(lse) - rl) <= el).all()


def test_page_numbers_that_are_none_in_shared_items(ab):
    q, k, v = case(10, 3, 2, 2, 150, 600, 64)
    kp, vp, table = ref.paged(k, v, [600] * 3, 16, M=6250)
    table[1, 5] = -1
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, lens=ints([600] * 3), L=100000)
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
    check(out[::2], lse[::2], q[::2], k[::2], v[::2], [600] * 2, [150] * 2, oracle.slopes(4))


@pytest.mark.parametrize("B,T", [(3, 300), (200, 40)])
def test_slots_past_the_length_that_are_not_finite(ab, B, T):
    # freshly allocated pages hold anything: NaN everywhere but in the rows of the sequences (which ref.paged does), of
    # prompts whose first tiles are their last
    q, k, v = case(T, B, 2, 1, T, T, 128)
    lens = [T - (7 * b) % T for b in range(B)]
    compare(ab, q, k, v, lens, lens, 64)


def test_offsets_beyond_32_bits(ab):
    import torch
    S, H, d = 64, 8, 128
    P = (1 << 32) // (S * H * d) + 10
    q, k, v = case(11, 1, H, 1, 100, 200, d)
    kp, vp = (torch.empty(P, H, S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = ints([[P - 1, 0, P - 2, P // 2]])
    ab.alibi_paged_append(bf16(k)[1], bf16(v)[1], kp, vp, table)
    out, lse = ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, L=200)
    ab.alibi_check_error()
    check(out, lse, q, k, v, [200], [100], oracle.slopes(H))
    del kp, vp
    torch.cuda.empty_cache()


def test_prompts_in_chunks_then_decode_in_graphs(ab):
    # prompts of two lengths appended and attended in chunks of 100 tokens, each chunk one replay of a graph that follows
    # positions and counts; then the decode of a token
    import torch
    B, Hkv, G, d, S, step = 2, 2, 2, 64, 16, 100
    total = [390, 145]
    N = max(total) + 1
    q, k, v = case(12, B, Hkv, G, N, N, d)
    M = -(-N // S)
    kp, vp = ref.pools(B * M, Hkv, S, d, "slots")
    table = ints(np.random.default_rng(1).permutation(B * M).reshape(B, M))
    (_, kd), (_, vd), (_, qd) = bf16(k), bf16(v), bf16(q)
    pos, count, lens = ints([0, 0]), ints([0, 0]), ints([0, 0])
    ks, vs = torch.zeros(B, Hkv, step, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, Hkv, step, d, dtype=torch.bfloat16, device="cuda")
    qs = torch.zeros(B, Hkv * G, step, d, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros_like(qs), torch.zeros(B, Hkv * G, step, device="cuda")

    def run():
        ab.alibi_paged_append(ks, vs, kp, vp, table, pos=pos, count=count)
        torch.add(pos, count, out=lens)
        ab.alibi_attn_fwd_paged(qs, kp, vp, table, lens=lens, count=count, out=out, lse=lse)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for at in range(0, max(total), step):
        now = [max(0, min(step, n - at)) for n in total]
        first = [min(at, n) for n in total]
        pos.copy_(ints(first))
        count.copy_(ints(now))
        for b in range(B):
            c, f = now[b], first[b]
            ks[b, :, :c], vs[b, :, :c], qs[b, :, :c] = kd[b, :, f:f + c], vd[b, :, f:f + c], qd[b, :, f:f + c]
        out.fill_(7.0)
        g.replay()
        ab.alibi_check_error()
        part = np.zeros((B, Hkv * G, step, d))
        for b in range(B):
            part[b, :, :now[b]] = q[b, :, first[b]:first[b] + now[b]]
            assert bool((out[b, :, now[b]:] == 7.0).all())
        check(out, lse, part, k, v, [f + c for f, c in zip(first, now)], now, oracle.slopes(Hkv * G), at)
    last = torch.stack([kd[b, :, n:n + 1] for b, n in enumerate(total)]), torch.stack([vd[b, :, n:n + 1] for b, n in enumerate(total)])
    ab.alibi_paged_append(*last, kp, vp, table, pos=ints(total))
    ql = np.stack([q[b, :, n:n + 1] for b, n in enumerate(total)])
    o, l = ab.alibi_attn_decode_paged(bf16(ql)[1], kp, vp, table, lens=ints([n + 1 for n in total]))
    ab.alibi_check_error()
    check(o, l, ql, k, v, [n + 1 for n in total], [1, 1], oracle.slopes(Hkv * G))


def test_calls_on_two_streams_at_once(ab):
    import torch
    jobs = []
    for s in range(2):
        q, k, v = case(20 + s, 2, 4, 2, 600, 1500, 128)
        cache = ref.paged(k, v, [1500, 1300], 64, seed=s)
        args = (bf16(q)[1], *cache)
        lens = ints([1500, 1300])
        jobs.append((args, lens, ab.alibi_attn_fwd_paged(*args, lens=lens), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[ab.alibi_attn_fwd_paged(*args, lens=lens, stream=st) for args, lens, _, st in jobs] for _ in range(10)]
    torch.cuda.synchronize()
    ab.alibi_check_error()
    for outs in got:
        for (o, l), (_, _, want, _) in zip(outs, jobs):
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])
