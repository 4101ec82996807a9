"""Decode over the 4-bit KV cache with more than 256 query heads, where the groups of 32 elements of a row differ
widely in magnitude, where queries and keys lie at the ends of bf16's range, and with large logits and slopes: against
attention in 64 bits over the held values, within bounds that hold for each group by itself
(kv4_ref.decode_by_group)."""
import numpy as np
import pytest

import alibi_inputs as gen
import kv4_ref as ref
import oracle
from gpu_helpers import half_ulp_bf16, host64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ab():
    import alibi_positional_bias_gb300 as ab
    ab.load()
    return ab


def exact_bf16(x):
    return gen.make_tensor(np.asarray(x, dtype=np.float32), np.shape(x), "bf16").f32.astype(np.float64)


def compare(ab, q, k, v, lens, m=None, what=""):
    """q, k, v: exact bf16 values; the whole of out and lse against the bounds of each group."""
    import torch
    B, H = q.shape[:2]
    C = -(-k.shape[2] // 32) * 32
    cache = torch.from_numpy(np.concatenate([ref.pack(k[b:b + 1, :, :n], v[b:b + 1, :, :n], C)
                                             for b, n in enumerate(lens)])).cuda()
    qd = torch.from_numpy(gen.make_tensor(q.astype(np.float32), q.shape, "bf16").bf16.view(np.int16)).view(torch.bfloat16).cuda()
    slopes = None if m is None else np.asarray(m, dtype=np.float32)
    out, lse = ab.alibi_attn_decode_kv4(qd, cache, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), slopes=slopes)
    ab.alibi_check_error()
    ro, rl, eo, el = ref.decode_by_group(q, ref.held(k), ref.held(v), lens,
                                         oracle.slopes(H) if m is None else slopes.astype(np.float64))
    go, gl = host64(out), host64(lse)
    assert np.isfinite(go).all() and np.isfinite(gl).all(), what
    lim = eo + half_ulp_bf16(ro) * (1 + 2.0 ** -6) + 2.0 ** -133
    assert (np.abs(go - ro) <= lim).all(), (what, (np.abs(go - ro) / lim).max())
    assert (np.abs(gl - rl) <= el).all(), (what, (np.abs(gl - rl) / el).max())


def case(seed, B, Hkv, G, T, N, d):
    rng = np.random.default_rng(seed)
    return (exact_bf16(rng.standard_normal(s)) for s in ((B, Hkv * G, T, d), (B, Hkv, N, d), (B, Hkv, N, d)))


# Whole chunks (the first two), clusters, and slices with a merge kernel; one row per lane and two
SHAPES = [(2, 2, 1, 1, 96, 64), (1, 2, 3, 2, 200, 128), (1, 8, 1, 1, 3000, 128), (1, 1, 1, 1, 20000, 64), (1, 2, 8, 1, 3000, 64)]


@pytest.mark.parametrize("power", [16, 24, 32, 40, 100, -40])
@pytest.mark.parametrize("B,Hkv,G,T,N,d", SHAPES)
def test_a_value_group_far_larger_or_smaller_than_the_others(ab, B, Hkv, G, T, N, d, power):
    q, k, v = case(power + N, B, Hkv, G, T, N, d)
    v[..., :32] *= 2.0 ** power
    lens = [N - 5 * b for b in range(B)]
    compare(ab, q, k, exact_bf16(v), lens, what="default slopes")
    compare(ab, q, k, exact_bf16(v), lens, m=np.zeros(Hkv * G), what="flat")
    compare(ab, q * 0, k, exact_bf16(v), lens, m=np.zeros(Hkv * G), what="equal weights")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("apart", [10, 20, 50])
def test_groups_apart_by_powers_of_two_in_turn(ab, apart, d):
    # group n of token j has values about 2^(apart (n + j) mod 3): the largest group changes from token to token
    q, k, v = case(apart, 1, 2, 2, 1, 320, d)
    n, j = np.arange(d) // 32, np.arange(320)
    v = exact_bf16(v * 2.0 ** (apart * ((n[None, :] + j[:, None]) % 3 - 1)))
    for m in (None, np.zeros(4)):
        compare(ab, q, k, v, [317], m=m)


@pytest.mark.parametrize("d", [64, 128])
def test_a_group_that_only_far_tokens_fill(ab, d):
    # the newest tokens have zeros in group 1 and large values in group 0; the far ones, whose weights are 2^-30 of the
    # newest ones', alone fill group 1
    q, k, v = case(3, 1, 1, 1, 1, 256, d)
    v[..., 224:, 32:64] = 0.0
    v[..., 224:, :32] *= 2.0 ** 30
    compare(ab, q, k, exact_bf16(v), [256], m=np.full(1, 30 * np.log(2) / 64))


@pytest.mark.parametrize("B,Hkv,G,T,N,d", SHAPES)
@pytest.mark.parametrize("sk,sq", [(1e34, 1e-34), (7e37, 1e-37), (2.0 ** 112, 2.0 ** -112), (1e37, 1e-38), (1e20, 1e-20)])
def test_keys_at_the_upper_end_of_the_range(ab, B, Hkv, G, T, N, d, sk, sq):
    q, k, v = case(N, B, Hkv, G, T, N, d)
    lens = [N - 5 * b for b in range(B)]
    big = 255 * 2.0 ** 120  # bf16's largest number
    compare(ab, exact_bf16(q * sq), exact_bf16(np.clip(k * sk, -big, big)), v, lens)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_the_largest_keys(ab, d):
    # keys of +-bf16's largest number; queries of 2^-126 to 2^-120, whose logits are some tens
    rng = np.random.default_rng(d)
    big = 255 * 2.0 ** 120
    k = exact_bf16(rng.choice([-big, big], size=(1, 2, 160, d)))
    q = exact_bf16(rng.standard_normal((1, 4, 1, d)) * 2.0 ** -126)
    v = exact_bf16(rng.standard_normal((1, 2, 160, d)))
    compare(ab, q, k, v, [150])
    compare(ab, exact_bf16(q * 32), k, v, [150])


@pytest.mark.parametrize("power", [12, 30, 45, 90])
@pytest.mark.parametrize("d", [64, 128])
def test_query_groups_of_very_different_magnitude(ab, d, power):
    # group 0 of the query is 2^power larger and that of the keys as much smaller: every group has its part of the logits
    q, k, v = case(power, 2, 2, 2, 2, 320, d)
    q[..., :32] *= 2.0 ** power
    k[..., :32] *= 2.0 ** -power
    compare(ab, exact_bf16(q), exact_bf16(k), v, [320, 77])


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("sk,sq", [(1e38, 1e6), (1e38, 1e38), (1e30, 1e20)])
def test_large_keys_that_large_queries_do_not_meet(ab, d, sk, sq):
    # q.k = 0 although the largest of both are out of range together: where one has values the other has zeros
    q, k, v = case(d, 1, 2, 2, 1, 128, d)
    q[..., ::2] = 0.0
    k[..., 1::2] = 0.0
    compare(ab, exact_bf16(np.clip(q, -3, 3) * sq), exact_bf16(np.clip(k, -3, 3) * sk), v, [120])


@pytest.mark.parametrize("Hkv,G,T,d", [(40, 8, 1, 64), (37, 7, 2, 32), (48, 8, 1, 128), (1, 384, 1, 64), (43, 6, 5, 16)])
def test_more_than_256_query_heads(ab, Hkv, G, T, d):
    q, k, v = case(Hkv, 2, Hkv, G, T, 64, d)
    compare(ab, q, k, v, [64, 37])
    compare(ab, q, k, v, [50, 64], m=np.linspace(0.0, 1.5, Hkv * G))


@pytest.mark.parametrize("G,d", [(1, 64), (8, 64), (2, 128), (8, 128), (1, 32)])
@pytest.mark.parametrize("step", [2.0 ** 18, 3e8, 7e9, 1e15, 1e33])
def test_logits_far_beyond_whole_numbers_in_fp32(ab, G, d, step):
    # logits that grow towards the oldest token, up to some 25 `step`: the reference moves in nearly every block, by numbers
    # that fp32 rounds to more than one. Only the oldest tokens, whose keys are equal in bf16, have a weight: two products off
    # by 2^-11 at most, a mean and a rounding of 2^-9
    rng = np.random.default_rng(d)
    N = 700
    q = np.ones((1, G, 1, d))
    k = exact_bf16(np.broadcast_to(3.0 * step * np.linspace(1.0, 1.0 / 400.0, N)[:, None], (1, 1, N, d)))
    v = exact_bf16(rng.standard_normal((1, 1, N, d)) * 2.0 ** 100)
    compare(ab, q, k, v, [N], m=np.zeros(G))
    import torch
    cache = torch.from_numpy(ref.pack(k, v, 704)).cuda()
    qd = torch.ones(1, G, 1, d, dtype=torch.bfloat16, device="cuda")
    out, _ = ab.alibi_attn_decode_kv4(qd, cache, lens=torch.tensor([N], dtype=torch.int32, device="cuda"),
                                      slopes=np.zeros(G, dtype=np.float32))
    logits = ref.held(k)[0, 0].sum(-1)
    first = ref.held(v)[0, 0, logits == logits.max()]
    assert np.abs(host64(out)[0, :, 0] - first.mean(0)).max() <= (2.0 ** -9 + 2.0 ** -10) * np.abs(first).max()


@pytest.mark.parametrize("T,d", [(1, 64), (3, 128), (1, 32)])
def test_large_slopes_at_every_length_of_a_block(ab, T, d):
    # the bias of the query's own token is 0 wherever in a block it stands, and that of the one before it the slope
    B = 33
    q, k, v = case(T, B, 1, 6, T, 320, d)
    compare(ab, q, k, v, list(range(288, 288 + B)), m=[0.0, 3.0, 1e3, 1e4, 1e10, 1e30])


def magnitudes(rng, x, lo, hi):
    """x times powers of two: none, one for all, one per group of 32, one per token, or with most elements zero."""
    d, kind = x.shape[-1], rng.integers(0, 5)
    if kind == 1:
        return x * 2.0 ** rng.integers(lo, hi)
    if kind == 2:
        return x * np.repeat(2.0 ** rng.integers(lo // 2, hi // 2, size=max(1, d // 32)), min(32, d))
    if kind == 3:
        return x * 2.0 ** rng.integers(lo // 3, hi // 3, size=x.shape[:-1] + (1,))
    return x * (rng.random(x.shape) < 0.2) if kind == 4 else x


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(ab, seed):
    rng = np.random.default_rng(1000 + seed)
    d = int(rng.choice([16, 32, 64, 128]))
    B, Hkv, N = int(rng.integers(1, 5)), int(rng.integers(1, 4)), max(1, int(np.exp(rng.uniform(0.0, np.log(3000.0)))))
    G, T = int(rng.choice([1, 1, 2, 3, 5, 8, 11])), int(rng.choice([1, 1, 1, 2, 4, 7, 16]))
    q, k, v = (rng.standard_normal(s) for s in ((B, Hkv * G, T, d), (B, Hkv, N, d), (B, Hkv, N, d)))
    s = int(rng.integers(-60, 110)) if seed % 2 else 0
    k, q, v = k * 2.0 ** s, q * 2.0 ** max(-120, -s), magnitudes(rng, v, -90, 110)
    if seed % 3 == 0:
        g = np.repeat(2.0 ** rng.integers(-40, 40, size=max(1, d // 32)), min(32, d))
        q, k = q * g, k / g
    big = 255 * 2.0 ** 120
    q, k, v = (exact_bf16(np.clip(x, -big, big)) for x in (q, k, v))
    lens = [int(rng.choice([N, rng.integers(1, N + 1), min(N, int(rng.integers(1, 4)))])) for _ in range(B)]
    lens = [max(n, T) for n in lens] if N >= T else [N] * B
    if N < T:
        q, T = q[:, :, :1], 1
    m = None if seed % 5 < 2 else rng.choice([0.0, 1e-3, 0.3, 5.0, 1e4]) * rng.random(Hkv * G)
    compare(ab, q, k, v, lens, m=m, what=(B, Hkv, G, T, N, d, lens))
