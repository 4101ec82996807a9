"""The paged cache: appending tokens (alibi_paged_append), with and without rotation, and the decode over the pages
(alibi_attn_decode_paged), against plain forms in 64 bits within the bounds derived in tests/paged_ref.py."""
import threading

import numpy as np
import pytest

import oracle
import paged_ref as ref
from gpu_helpers import half_ulp_bf16, host64
from paged_ref import bf16, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ab():
    import alibi_positional_bias_gb300 as ab
    ab.load()
    return ab


def case(seed, B, Hkv, G, T, N, d, strong=4.0):
    """q, k, v as exact bf16 values, a few strong key channels."""
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((B, Hkv, N, d))
    k[..., :: max(1, d // 4)] *= strong
    return tuple(bf16(a)[0] for a in (rng.standard_normal((B, Hkv * G, T, d)), k, rng.standard_normal((B, Hkv, N, d))))


def check(out, lse, want, what=""):
    ro, rl, eo, el = want
    assert tuple(out.shape) == ro.shape and tuple(lse.shape) == rl.shape
    go, gl = host64(out), host64(lse)
    assert np.isfinite(go).all(), what
    lim = eo + half_ulp_bf16(ro) * (1 + 2.0 ** -6) + 2.0 ** -133
    assert (np.abs(go - ro) <= lim).all(), (what, (np.abs(go - ro) / lim).max())
    none = np.isinf(rl)
    assert np.array_equal(none, np.isinf(gl)) and (gl[none] < 0).all() and (go[none] == 0).all()
    off = np.abs(gl[~none] - rl[~none])
    assert (off <= el[~none]).all(), (what, (off - el[~none]).max())


def compare(ab, q, k, v, lens, S=16, m=None, slopes=None, L=None, M=None, layout="heads", unused=-1, what=""):
    B, H, T = q.shape[:3]
    kp, vp, table = ref.paged(k, v, lens, S, seed=B + S, layout=layout, M=M, unused=unused)
    out, lse = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints(lens), L=L, slopes=slopes)
    ab.alibi_check_error()
    # a query before the first row is row T of a longer count in `attention`'s sense: positions len - T + t
    check(out, lse, ref.attention(q, k, v, lens, [T] * B, oracle.slopes(H) if m is None else m), what)
    return out, lse, (kp, vp, table)


# ------------------------------------------------------------------------ decode

@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("S", [8, 16, 64])
def test_every_length_of_a_few_pages(ab, d, S):
    # one sequence per length 0 .. 150: every place in a page, a tile and a stage where a sequence can end
    N = 150
    q, k, v = case(N + d + S, N + 1, 1, 2, 1, N, d)
    compare(ab, q, k, v, list(range(N + 1)), S)


@pytest.mark.parametrize("B,Hkv,G,T,N,d,S", [
    (1, 1, 1, 1, 33, 128, 16), (2, 3, 1, 1, 517, 128, 32), (1, 4, 1, 1, 4099, 64, 16), (3, 2, 3, 1, 1025, 32, 128),
    (1, 2, 8, 1, 2047, 128, 1024), (1, 1, 9, 1, 543, 64, 8), (2, 1, 40, 1, 320, 128, 16), (1, 1, 71, 2, 97, 64, 16),
    (2, 2, 4, 2, 1023, 128, 64), (1, 2, 2, 4, 801, 64, 256), (1, 2, 5, 3, 417, 128, 16), (2, 1, 1, 16, 255, 128, 16),
    (1, 3, 16, 1, 641, 16, 16), (1, 1, 1, 1, 20001, 128, 32), (1, 2, 4, 1, 50017, 64, 128), (5, 7, 1, 1, 95, 128, 16),
    (40, 8, 2, 1, 65, 64, 16), (2, 2, 3, 16, 300, 32, 512), (1, 1, 33, 1, 130, 16, 8), (300, 1, 1, 1, 40, 128, 16)])
def test_shapes(ab, B, Hkv, G, T, N, d, S):
    q, k, v = case(7 * N + d + G, B, Hkv, G, T, N, d)
    lens = [max(0, N - (37 * b) % N) for b in range(B)]
    compare(ab, q, k, v, lens, S)
    compare(ab, q, k, v, lens, S, M=-(-N // S) + 3, L=N + 5)  # planned for more than there is
    compare(ab, q, k, v, [N] * B, S, unused=2 ** 31 - 1)


@pytest.mark.parametrize("layout", ref.LAYOUTS)
@pytest.mark.parametrize("d,S", [(16, 8), (64, 32), (128, 16), (128, 128)])
def test_layouts(ab, layout, d, S):
    q, k, v = case(S + d, 3, 5, 2, 2, 300, d)
    out, lse, _ = compare(ab, q, k, v, [300, 1, 217], S, layout=layout)
    import torch
    plain, plain_lse, _ = compare(ab, q, k, v, [300, 1, 217], S)
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)


@pytest.mark.parametrize("T", [2, 5, 16])
def test_more_new_tokens_than_length(ab, T):
    # queries before the first row see nothing: out 0, lse -inf
    q, k, v = case(T, 6, 2, 2, T, 32, 64)
    kp, vp, table = ref.paged(k, v, [0, 1, 2, T - 1, T, T + 1], 16)
    out, lse = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints([0, 1, 2, T - 1, T, T + 1]))
    ab.alibi_check_error()
    for b, n in enumerate([0, 1, 2, T - 1, T, T + 1]):
        c = min(n, T)
        assert bool((out[b, :, :T - c] == 0).all()) and bool((lse[b, :, :T - c] == -np.inf).all())
        if c:
            want = ref.attention(q[b:b + 1, :, T - c:], k[b:b + 1], v[b:b + 1], [n], [c], oracle.slopes(4))
            check(out[b:b + 1, :, T - c:], lse[b:b + 1, :, T - c:], want)


def test_three_dimensional_query_and_given_outputs(ab):
    import torch
    q, k, v = case(3, 2, 2, 2, 1, 64, 64)
    out4, lse4, cache = compare(ab, q, k, v, [64, 33])
    out, lse = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 4, device="cuda")
    got = ab.alibi_attn_decode_paged(bf16(q[:, :, 0])[1], *cache, lens=ints([64, 33]), out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert torch.equal(out, out4[:, :, 0]) and torch.equal(lse, lse4[:, :, 0])


def test_caller_slopes_and_no_bias(ab):
    q, k, v = case(4, 1, 2, 4, 1, 1000, 128)
    for m in (np.zeros(8), np.linspace(0.0, 2.0, 8), oracle.slopes(8)[::-1], np.array([1e4, 3e4, 1e-6, 0, 1, 2, 3, 1e30])):
        m32 = m.astype(np.float32)
        compare(ab, q, k, v, [777], m=m32.astype(np.float64), slopes=m32)


def test_large_logits(ab):
    # scores of some hundreds in either order along the cache: the reference moves often
    q, k, v = case(5, 2, 2, 2, 1, 1024, 128)
    ramp = np.linspace(0.0, 20.0, 1024)
    for r in (ramp, ramp[::-1]):
        kk = bf16(k * r[None, None, :, None])[0]
        compare(ab, bf16(4 * q)[0], kk, v, [1024, 999], m=np.zeros(4), slopes=np.zeros(4, np.float32))


def test_pages_that_sequences_share(ab):
    # a common prefix: the first pages of all sequences are the same
    import torch
    q, k, v = case(6, 3, 2, 2, 1, 100, 64)
    k[1:, :, :64], v[1:, :, :64] = k[:1, :, :64], v[:1, :, :64]
    lens = [100, 70, 65]
    kp, vp, table = ref.paged(k, v, lens, 16)
    table[1:, :4] = table[:1, :4]
    out, lse = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints(lens))
    ab.alibi_check_error()
    check(out, lse, ref.attention(q, k, v, lens, [1] * 3, oracle.slopes(4)))
    assert torch.isfinite(out.float()).all()


# (B, Hkv, G, T, N, d): few chunks, about as many as CTAs, and many; short and long
WAYS = [(1, 1, 1, 1, 9000, 128), (1, 3, 4, 1, 3000, 64), (1, 2, 8, 4, 700, 128), (7, 5, 1, 1, 900, 128), (33, 5, 2, 1, 500, 64),
        (70, 5, 1, 1, 200, 128), (130, 3, 1, 1, 300, 32), (1, 1, 1, 1, 120000, 16), (2, 40, 1, 1, 2000, 128), (150, 8, 1, 1, 70, 128)]


@pytest.mark.parametrize("B,Hkv,G,T,N,d", WAYS)
@pytest.mark.parametrize("spread", ["equal", "ragged", "one long"])
def test_ways_of_dealing(ab, B, Hkv, G, T, N, d, spread):
    q, k, v = case(N + B, B, Hkv, G, T, N, d)
    lens = {"equal": [N] * B, "ragged": [N - (b * 7919) % N for b in range(B)], "one long": [N] + [b % 9 for b in range(1, B)]}[spread]
    if T > 1:
        lens = [max(T, n) for n in lens]
    out, lse, cache = compare(ab, q, k, v, lens, 32, L=N)
    import torch
    for _ in range(3):  # the same bits for the same arguments
        o, l = ab.alibi_attn_decode_paged(bf16(q)[1], *cache, lens=ints(lens), L=N)
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("G,T", [(1, 3), (4, 2), (2, 16), (12, 2)])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_infinite_and_nan_rows_that_a_query_does_not_see(ab, G, T, d):
    # the newest token's key and value are infinite or NaN: only the queries that see it may know
    import torch
    N = 150
    q, k, v = case(d + T, 2, 1, G, T, N, d)
    for bad in (float("inf"), float("nan")):
        kp, vp, table = ref.paged(k, v, [N, N - 17], 16)
        for b, n in enumerate((N, N - 17)):
            page, slot = int(table[b, (n - 1) // 16]), (n - 1) % 16
            kp[page, :, slot, 0] = float("nan")
            vp[page, :, slot] = bad
            vp[page, :, slot, 1] = -bad
        out, lse = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints([N, N - 17]))
        ab.alibi_check_error()
        want = ref.attention(q[:, :, :-1], k, v, [N - 1, N - 18], [T - 1] * 2, oracle.slopes(G))
        check(out[:, :, :-1], lse[:, :, :-1], want, (bad, d))
        assert bool(torch.isnan(out[:, :, -1].float()).all()) and bool(torch.isnan(lse[:, :, -1]).all())


def test_infinite_values_that_are_seen(ab):
    import torch
    q, k, v = case(8, 1, 1, 2, 2, 40, 64)
    kp, vp, table = ref.paged(k, v, [40], 16)
    vp[int(table[0, 39 // 16]), 0, 38 % 16, 5] = float("inf")  # row 38: both queries see it
    vp[int(table[0, 39 // 16]), 0, 39 % 16, 6] = float("-inf")  # row 39: the second one does
    out, _ = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints([40]))
    o = out.float()
    assert bool((o[0, :, :, 5] == np.inf).all()) and bool((o[0, :, 1, 6] == -np.inf).all()) and bool(torch.isfinite(o[0, :, 0, 6]).all())
    o[0, :, :, 5] = o[0, :, 1, 6] = 0
    assert bool(torch.isfinite(o).all())


@pytest.mark.parametrize("B,N,L", [(5, 300, 300), (5, 300, 5000), (200, 60, 60), (1, 300, 9000)])
def test_lengths_outside_the_bound(ab, B, N, L):
    q, k, v = case(9, B, 2, 2, 1, N, 64)
    kp, vp, table = ref.paged(k, v, [N] * B, 16, M=-(-L // 16))
    good, _ = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints([N] * B), L=L)
    ab.alibi_check_error()
    lens = [N] * B
    lens[0] = -1
    if B > 3:
        lens[3] = L + 1
    out, lse = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints(lens), L=L)
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    ab.alibi_check_error()  # collected
    for b in range(B):
        if lens[b] == N:
            assert bool((out[b] == good[b]).all())
        else:
            assert bool(out[b].isnan().all()) and bool(lse[b].isnan().all())


@pytest.mark.parametrize("B,N,at", [(4, 300, 0), (4, 300, 18), (1, 9000, 300), (150, 70, 4)])
@pytest.mark.parametrize("number", [-1, -2 ** 31, 2 ** 31 - 1, "one past"])
def test_page_numbers_that_are_none(ab, B, N, at, number):
    q, k, v = case(10, B, 2, 2, 1, N, 64)
    kp, vp, table = ref.paged(k, v, [N] * B, 16)
    good, _ = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints([N] * B))
    ab.alibi_check_error()
    table[B // 2, at] = kp.shape[0] if number == "one past" else number
    out, lse = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints([N] * B))
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    for b in range(B):
        if b == B // 2:
            assert bool(out[b].isnan().all()) and bool(lse[b].isnan().all())
        else:
            assert bool((out[b] == good[b]).all())


def test_offsets_beyond_32_bits(ab):
    # pools of more than 2^32 elements, of which only the pages in use are written
    import torch
    S, H, d = 64, 8, 128
    P = (1 << 32) // (S * H * d) + 10
    q, k, v = case(11, 2, H, 1, 1, 200, d)
    kp, vp = (torch.empty(P, H, S, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = [P - 1, 0, P - 2, P // 2, P - 3, 1, P // 2 + 1, P - 4]
    table = ints([pages[:4], pages[4:]])
    ab.alibi_paged_append(bf16(k)[1], bf16(v)[1], kp, vp, table)
    for b in range(2):
        for i in range(4):
            n = min(S, 200 - i * S)
            assert torch.equal(kp[int(table[b, i]), :, :n], bf16(k[b, :, i * S:i * S + n])[1])
            assert torch.equal(vp[int(table[b, i]), :, :n], bf16(v[b, :, i * S:i * S + n])[1])
    out, lse = ab.alibi_attn_decode_paged(bf16(q)[1], kp, vp, table, lens=ints([200, 137]))
    ab.alibi_check_error()
    check(out, lse, ref.attention(q, k, v, [200, 137], [1, 1], oracle.slopes(H)))
    del kp, vp
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------ append

def append_want(kp, vp, table, S, k, v, pos, count, M):
    """The pools after an append of rows k, v (tensors), by the definition."""
    kp, vp = kp.clone(), vp.clone()
    for b in range(k.shape[0]):
        if pos[b] < 0 or count[b] < 0 or count[b] > k.shape[2] or pos[b] + count[b] > M * S:
            continue
        for t in range(count[b]):
            page = int(table[b, (pos[b] + t) // S])
            if 0 <= page < kp.shape[0]:
                kp[page, :, (pos[b] + t) % S] = k[b, :, t]
                vp[page, :, (pos[b] + t) % S] = v[b, :, t]
    return kp, vp


def same_bits(a, b):
    import torch
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


@pytest.mark.parametrize("B,H,T,d,S,pos,count", [
    (1, 1, 1, 128, 16, [0], [1]), (3, 2, 1, 64, 8, [0, 17, 63], [1, 1, 0]), (2, 40, 1, 128, 16, [5, 47], [1, 1]),
    (2, 3, 37, 16, 16, [0, 9], [37, 20]), (1, 5, 100, 32, 32, [3], [97]), (2, 33, 65, 128, 64, [63, 0], [65, 1]),
    (1, 1, 500, 64, 1024, [200], [500]), (4, 7, 3, 128, 128, [0, 1, 127, 250], [3, 3, 3, 3]), (1, 300, 2, 16, 8, [7], [2])])
@pytest.mark.parametrize("layout", ref.LAYOUTS)
def test_append(ab, B, H, T, d, S, pos, count, layout):
    import torch
    M = max(-(-(p + c) // S) for p, c in zip(pos, count)) + 1
    kp, vp = ref.pools(B * M + 2, H, S, d, layout)
    table = ints(np.random.default_rng(T).permutation(B * M + 2)[:B * M].reshape(B, M))
    rng = np.random.default_rng(B + T)
    (_, k), (_, v) = (bf16(rng.standard_normal((B, H, T, d))) for _ in range(2))
    want = append_want(kp, vp, table, S, k, v, pos, count, M)
    ab.alibi_paged_append(k, v, kp, vp, table, pos=ints(pos), count=ints(count))
    ab.alibi_check_error()
    assert same_bits(kp, want[0]) and same_bits(vp, want[1])
    # rows as a projection gives them, [B, T, H, d], and as parts of one tensor
    kp2, vp2 = ref.pools(B * M + 2, H, S, d, layout)
    both = torch.stack((k, v), 3).transpose(1, 2).contiguous()  # [B, T, H, 2, d]
    ab.alibi_paged_append(both[..., 0, :].transpose(1, 2), both[..., 1, :].transpose(1, 2), kp2, vp2, table, pos=ints(pos), count=ints(count))
    assert same_bits(kp2, want[0]) and same_bits(vp2, want[1])


def test_append_without_positions_or_counts(ab):
    kp, vp = ref.pools(10, 2, 16, 64, "heads")
    table = ints([[3, 1, 4], [9, 2, 6]])
    rng = np.random.default_rng(0)
    (_, k), (_, v) = (bf16(rng.standard_normal((2, 2, 40, 64))) for _ in range(2))
    want = append_want(kp, vp, table, 16, k, v, [0, 0], [40, 40], 3)
    ab.alibi_paged_append(k, v, kp, vp, table)
    ab.alibi_check_error()
    assert same_bits(kp, want[0]) and same_bits(vp, want[1])


@pytest.mark.parametrize("pos,count,bad", [
    ([0, -1, 5], [4, 4, 4], True), ([0, 29, 5], [4, 4, 4], True), ([0, 28, 5], [4, 4, 4], False), ([0, 2, 5], [4, -1, 4], True),
    ([0, 2, 5], [4, 5, 4], True), ([0, 2 ** 31 - 1, 5], [4, 4, 4], True), ([0, -2 ** 31, 5], [4, 4, 4], True), ([0, 32, 5], [4, 0, 4], False)])
def test_append_outside_the_table(ab, pos, count, bad):
    kp, vp = ref.pools(12, 3, 8, 32, "heads")
    table = ints(np.arange(12).reshape(3, 4))
    rng = np.random.default_rng(0)
    (_, k), (_, v) = (bf16(rng.standard_normal((3, 3, 4, 32))) for _ in range(2))
    want = append_want(kp, vp, table, 8, k, v, pos, count, 4)
    ab.alibi_paged_append(k, v, kp, vp, table, pos=ints(pos), count=ints(count))
    if bad:
        with pytest.raises(ab.AlibiError) as e:
            ab.alibi_check_error()
        assert e.value.status == ab.ALIBI_ERR_RANGE
    ab.alibi_check_error()
    assert same_bits(kp, want[0]) and same_bits(vp, want[1])


@pytest.mark.parametrize("number", [-1, -2 ** 31, 12, 2 ** 31 - 1])
def test_append_to_page_numbers_that_are_none(ab, number):
    kp, vp = ref.pools(12, 3, 8, 32, "heads")
    table = ints(np.arange(12).reshape(3, 4))
    table[1, 1] = number
    rng = np.random.default_rng(0)
    (_, k), (_, v) = (bf16(rng.standard_normal((3, 3, 20, 32))) for _ in range(2))
    want = append_want(kp, vp, table, 8, k, v, [0] * 3, [20] * 3, 4)
    ab.alibi_paged_append(k, v, kp, vp, table)
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    assert same_bits(kp, want[0]) and same_bits(vp, want[1])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,R,H,G,T,pos", [
    (16, 16, 3, 1, 5, [0, 7]), (32, 16, 2, 2, 40, [1, 100]), (64, 64, 5, 4, 33, [1000, 70000]), (128, 128, 2, 3, 20, [0, 16000000]),
    (128, 32, 1, 8, 1, [131071, 5]), (128, 96, 20, 1, 3, [63, 65536]), (64, 48, 2, 40, 1, [0, 1])])
def test_append_rotated(ab, d, R, H, G, T, pos, interleaved):
    import torch
    S, M = 1024, 16384  # 2^24 tokens to a table
    B, count = 2, [T, max(1, T - 2)]
    table = torch.zeros(B, M, dtype=torch.int32, device="cuda")
    for b in range(B):
        table[b, pos[b] // S:pos[b] // S + 2] = ints([2 * b, 2 * b + 1])
    kp, vp = ref.pools(4, H, S, d, "slots")
    before = kp.clone(), vp.clone()
    rng = np.random.default_rng(d + T)
    (k64, k), (_, v), (q64, q) = (bf16(rng.standard_normal((B, h, T, d)) * 2) for h in (H, H, H * G))
    q_out = torch.full_like(q, 7.0)
    freqs = None if R != 96 else np.linspace(-3.0, 900.0, R // 2)
    got = ab.alibi_paged_append(k, v, kp, vp, table, pos=ints(pos), count=ints(count), rotate=R, freqs=freqs,
                                interleaved=interleaved, q=q, q_out=q_out)
    ab.alibi_check_error()
    assert got is q_out
    for b in range(B):
        c, n = count[b], pos[b] + np.arange(count[b])
        for x64, have in ((k64, torch.stack([kp[int(table[b, j // S]), :, j % S] for j in n], 1)), (q64, q_out[b, :, :c])):
            want, err = ref.rotated(x64[b, :, :c], n, R, freqs=freqs, interleaved=interleaved)
            off = np.abs(host64(have) - want)
            assert (off <= err + half_ulp_bf16(want) * (1 + 2.0 ** -6)).all(), (off - err - half_ulp_bf16(want)).max()
            assert np.array_equal(host64(have)[..., R:], x64[b, :, :c, R:])
        assert bool((q_out[b, :, c:] == 7.0).all())
        for t, j in enumerate(n):
            assert torch.equal(vp[int(table[b, j // S]), :, j % S], v[b, :, t])
            for x in (kp, vp):
                x[int(table[b, j // S]), :, j % S] = float("nan")
    assert same_bits(kp, before[0]) and same_bits(vp, before[1])  # nothing else was written


def test_rotation_made_here_and_without_queries(ab):
    import torch
    table = ints([[0, 1]])
    rng = np.random.default_rng(3)
    (k64, k), (_, v), (_, q) = (bf16(rng.standard_normal((1, h, 20, 64))) for h in (2, 2, 6))
    pools = [ref.pools(2, 2, 16, 64, "heads") for _ in range(2)]
    a = ab.alibi_paged_append(k, v, *pools[0], table, rotate=64, base=500.0, q=q)
    assert ab.alibi_paged_append(k, v, *pools[1], table, rotate=64, base=500.0) is None
    assert a.shape == q.shape and same_bits(pools[0][0], pools[1][0]) and same_bits(pools[0][1], pools[1][1])
    assert torch.equal(a[:, :, 0], q[:, :, 0])  # position 0 does not turn
    # given frequencies: the same as those of the base
    f = [500.0 ** (-2 * i / 64) for i in range(32)]
    third = ref.pools(2, 2, 16, 64, "heads")
    assert torch.equal(a, ab.alibi_paged_append(k, v, *third, table, rotate=64, freqs=f, q=q.transpose(1, 2).contiguous().transpose(1, 2)))
    assert same_bits(third[0], pools[0][0])


# ------------------------------------------------------------------- run together

def test_serving_steps_in_a_graph(ab):
    # prompts of two lengths, then steps of append and decode from one captured graph that follows the lengths
    import torch
    B, Hkv, G, d, S, steps, P = 2, 2, 3, 64, 16, 40, [90, 33]
    N = max(P) + steps
    q, k, v = case(15, B, Hkv, G, steps, N, d)
    M = -(-N // S)
    kp, vp = ref.pools(B * M, Hkv, S, d, "slots")
    table = ints(np.random.default_rng(5).permutation(B * M).reshape(B, M))
    (_, kd), (_, vd) = bf16(k), bf16(v)
    ab.alibi_paged_append(kd[:, :, :90], vd[:, :, :90], kp, vp, table, count=ints(P))
    lens = ints(P)
    qs, ks, vs = bf16(q[:, :, :1])[1], kd[:, :, :1].contiguous(), vd[:, :, :1].contiguous()

    def step():
        ab.alibi_paged_append(ks, vs, kp, vp, table, pos=lens)
        lens.add_(1)
        return ab.alibi_attn_decode_paged(qs, kp, vp, table, lens=lens)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out, lse = step()
    for i in range(steps):
        qs.copy_(bf16(q[:, :, i:i + 1])[1])
        for b in range(B):
            ks[b].copy_(kd[b, :, P[b] + i:P[b] + i + 1])
            vs[b].copy_(vd[b, :, P[b] + i:P[b] + i + 1])
        g.replay()
        torch.cuda.synchronize()
        check(out, lse, ref.attention(q[:, :, i:i + 1], k, v, [p + i + 1 for p in P], [1] * B, oracle.slopes(Hkv * G)), i)
    ab.alibi_check_error()


def test_two_graphs_and_streams_at_once(ab):
    # two captured decodes that split their work, replayed at the same time, and direct calls from host threads
    import torch
    jobs = []
    for s in range(2):
        q, k, v = case(20 + s, 1, 4, 4, 1, 20000 + 77 * s, 64)
        n = k.shape[2]
        cache = ref.paged(k, v, [n], 64, seed=s)
        qd, lens, stream = bf16(q)[1], ints([n]), torch.cuda.Stream()
        want = ab.alibi_attn_decode_paged(qd, *cache, lens=lens)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            got = ab.alibi_attn_decode_paged(qd, *cache, lens=lens)
        jobs.append((g, stream, got, want, (qd, *cache), lens))
    for _ in range(20):
        for g, stream, *_ in jobs:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for _, _, got, want, _, _ in jobs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    failed = []

    def work(job):
        try:
            _, stream, _, want, args, lens = job
            for _ in range(20):
                o, l = ab.alibi_attn_decode_paged(*args, lens=lens, stream=stream)
                stream.synchronize()
                if not (torch.equal(o, want[0]) and torch.equal(l, want[1])):
                    failed.append("differs")
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_calls_wait_for_each_other(ab):
    # each call begins while the one before it ends, and waits before it reads: lengths, table and rows of the call before
    import torch
    q, k, v = case(30, 4, 8, 2, 1, 3000, 128)
    S = 32
    M = -(-3000 // S)
    kd, vd, qd = bf16(k)[1], bf16(v)[1], bf16(q)[1]
    table0 = ints(np.random.default_rng(1).permutation(4 * M).reshape(4, M))
    want = None
    for _ in range(10):
        kp, vp = ref.pools(4 * M, 8, S, 128, "heads")
        table, lens = torch.full_like(table0, -1), torch.full((4,), -5, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        table.copy_(table0)
        ab.alibi_paged_append(kd, vd, kp, vp, table)
        lens.fill_(3000)
        out, lse = ab.alibi_attn_decode_paged(qd, kp, vp, table, lens=lens)
        ab.alibi_check_error()
        if want is None:
            want = out, lse
            check(out, lse, ref.attention(q, k, v, [3000] * 4, [1] * 4, oracle.slopes(16)))
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
