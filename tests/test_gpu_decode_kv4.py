"""Decode over the 4-bit KV cache (alibi_attn_decode_kv4) against attention in 64 bits over the values that
the cache holds, within the bounds derived in tests/kv4_ref.py."""
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


def bf16(x):
    import torch
    t = gen.make_tensor(np.asarray(x, dtype=np.float32), np.shape(x), "bf16")
    return t.f32.astype(np.float64), torch.from_numpy(t.bf16.view(np.int16)).view(torch.bfloat16).cuda()


def up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(seed, B, Hkv, G, T, N, d, strong=4.0):
    """q, k, v as exact bf16 values, a few strong key channels."""
    rng = np.random.default_rng(seed)
    k = rng.standard_normal((B, Hkv, N, d))
    k[..., :: max(1, d // 4)] *= strong
    x = lambda a: gen.make_tensor(a, a.shape, "bf16").f32.astype(np.float64)  # noqa: E731
    return x(rng.standard_normal((B, Hkv * G, T, d))), x(k), x(rng.standard_normal((B, Hkv, N, d)))


def compare(ab, q, k, v, lens, m=None, C=None, L=None, kernel_slopes=None, what=""):
    """The kernel's out and lse against the reference; rows past each length are 0xFF bytes (NaN scales)."""
    B, H = q.shape[:2]
    N = k.shape[2]
    full = [N] * B if lens is None else lens
    C = -(-N // 32) * 32 if C is None else C
    cache = up(np.concatenate([ref.pack(k[b:b + 1, :, :full[b]], v[b:b + 1, :, :full[b]], C) for b in range(B)]))
    out, lse = ab.alibi_attn_decode_kv4(bf16(q)[1], cache, lens=None if lens is None else ints(lens), L=L,
                                        slopes=kernel_slopes)
    ab.alibi_check_error()
    ro, rl, eo, el = ref.decode(q, ref.held(k), ref.held(v), full, oracle.slopes(H) if m is None else m)
    assert tuple(out.shape) == q.shape and tuple(lse.shape) == q.shape[:-1]
    go, gl = host64(out), host64(lse)
    assert np.isfinite(go).all(), what
    lim = eo + half_ulp_bf16(ro) * (1 + 2.0 ** -6) + 2.0 ** -133
    assert (np.abs(go - ro) <= lim).all(), (what, (np.abs(go - ro) / lim).max())
    none = np.isinf(rl)
    assert np.array_equal(none, np.isinf(gl)) and (gl[none] < 0).all() and (go[none] == 0).all()
    off = np.abs(gl[~none] - rl[~none])
    assert (off <= el[~none]).all(), (what, off.max())
    return out, lse


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("N", [32, 64, 160])
def test_every_length_of_a_few_blocks(ab, d, N):
    # one sequence per length 0 .. N: every place in a block and a tile where a sequence can end
    q, k, v = case(N + d, N + 1, 1, 2, 1, N, d)
    compare(ab, q, k, v, list(range(N + 1)))


@pytest.mark.parametrize("B,Hkv,G,T,N,d", [
    (1, 1, 1, 1, 32, 128), (2, 3, 1, 1, 512, 128), (1, 4, 1, 1, 4096, 64), (3, 2, 3, 1, 1024, 32), (1, 2, 8, 1, 2048, 128),
    (1, 1, 9, 1, 544, 64), (2, 1, 40, 1, 320, 128), (1, 1, 71, 2, 96, 64), (2, 2, 4, 2, 1024, 128), (1, 2, 2, 4, 800, 64),
    (1, 2, 5, 3, 416, 128), (2, 1, 1, 16, 256, 128), (1, 3, 16, 1, 640, 16), (1, 1, 1, 1, 20000, 128), (1, 2, 4, 1, 50016, 64),
    (5, 7, 1, 1, 96, 128), (40, 8, 2, 1, 64, 64)])
def test_shapes(ab, B, Hkv, G, T, N, d):
    q, k, v = case(7 * N + d + G, B, Hkv, G, T, N, d)
    lens = [max(0, N - (37 * b) % N) for b in range(B)]
    compare(ab, q, k, v, lens)
    compare(ab, q, k, v, lens, C=N + 96, L=N + 5)  # planned for more than there is
    if N % 32 == 0:
        compare(ab, q, k, v, None)


@pytest.mark.parametrize("T", [2, 5, 16])
def test_more_new_tokens_than_length(ab, T):
    # queries before the first row see nothing: out 0, lse -inf
    q, k, v = case(T, 6, 2, 2, T, 32, 64)
    out, lse = compare(ab, q, k, v, [0, 1, 2, T - 1, T, T + 1])
    assert bool((out[0] == 0).all()) and bool((lse[0] == -np.inf).all())
    assert bool((lse[1, :, :-1] == -np.inf).all()) and bool((lse[1, :, -1] > -np.inf).all())


def test_three_dimensional_query(ab):
    q, k, v = case(3, 2, 2, 2, 1, 64, 64)
    out4, lse4 = compare(ab, q, k, v, [64, 33])
    import torch
    cache = up(ref.pack(k, v))
    out, lse = ab.alibi_attn_decode_kv4(bf16(q[:, :, 0])[1], cache, lens=ints([64, 33]))
    assert out.shape == (2, 4, 64) and lse.shape == (2, 4)
    assert torch.equal(out, out4[:, :, 0]) and torch.equal(lse, lse4[:, :, 0])


def test_caller_slopes_and_no_bias(ab):
    q, k, v = case(4, 1, 2, 4, 1, 1000 // 32 * 32, 128)
    for m in (np.zeros(8), np.linspace(0.0, 2.0, 8), oracle.slopes(8)[::-1]):
        m32 = m.astype(np.float32)
        compare(ab, q, k, v, [777], m=m32.astype(np.float64), kernel_slopes=m32)


def test_large_logits(ab):
    # scores of some hundreds in either order along the cache: the running maximum moves often
    q, k, v = case(5, 2, 2, 2, 1, 1024, 128)
    for order in (1, -1):
        ramp = np.linspace(0.1, 60.0, 1024)[::order, None]
        k2 = gen.make_tensor(k / np.abs(k).max() * ramp, k.shape, "bf16").f32.astype(np.float64)
        compare(ab, q, k2, v, [1024, 900], m=np.zeros(4), kernel_slopes=np.zeros(4), what=f"order {order}")


@pytest.mark.parametrize("sk,sv,sq", [(1e-30, 1.0, 1.0), (1.0, 1e-28, 1.0), (1.0, 1e30, 1.0), (1e18, 1.0, 1e-18),
                                      (1e-18, 1e25, 1e18), (1.0, 1.0, 1e-30), (1.0, 1e37, 1e-3), (1e-25, 1.0, 1e25)])
def test_magnitudes(ab, sk, sv, sq):
    q, k, v = case(6, 1, 2, 2, 1, 96, 64)
    x = lambda a: gen.make_tensor(a, a.shape, "bf16").f32.astype(np.float64)  # noqa: E731
    compare(ab, x(q * sq), x(k * sk), x(v * sv), [90])


def test_values_of_very_different_magnitude_between_tokens(ab):
    # value scales that jump by 2^60 from token to token, with weights that make the small ones matter: every
    # second token's values are huge, but their keys put them 2^-80 below the others
    rng = np.random.default_rng(14)
    q, k, v = case(8, 1, 1, 1, 1, 128, 64)
    u = rng.standard_normal(64)
    q[:] = u / np.linalg.norm(u) * 8.0
    k[:] = 0.0
    k[:, :, 1::2] = -u / np.linalg.norm(u) * 56.0  # logit -56
    v[:, :, 1::2] *= 2.0 ** 60
    x = lambda a: gen.make_tensor(a, a.shape, "bf16").f32.astype(np.float64)  # noqa: E731
    compare(ab, x(q), x(k), x(v), [127], m=np.zeros(1), kernel_slopes=np.zeros(1))
    compare(ab, x(q), x(k), x(v), [128], m=np.zeros(1), kernel_slopes=np.zeros(1))


def test_zero_query_and_zero_values(ab):
    q, k, v = case(9, 1, 2, 1, 1, 320, 128)
    compare(ab, q * 0, k, v, [300])
    out, _ = compare(ab, q, k, v * 0, [300])
    assert bool((out == 0).all())
    compare(ab, q, k * 0, v, [300])


def test_nan_in_a_row_that_is_seen_and_in_rows_that_are_not(ab):
    q, k, v = case(10, 1, 3, 2, 3, 64, 64)
    k[0, 1, 40, 3] = np.nan          # seen by all queries of KV head 1
    v[0, 2, 49, 5] = np.inf          # length 50: row 49 is seen by the last query (t = 2) of KV head 2 alone
    cache = up(ref.pack(k, v))
    out, lse = ab.alibi_attn_decode_kv4(bf16(q)[1], cache, lens=ints([50]))
    ab.alibi_check_error()
    kc, vc = k.copy(), v.copy()
    kc[0, 1, 40], vc[0, 2, 49] = 0, 0
    ro, rl, eo, el = ref.decode(q, ref.held(kc), ref.held(vc), [50], oracle.slopes(6))
    go, gl = host64(out), host64(lse)
    assert np.isnan(go[0, 2:4]).all() and np.isnan(gl[0, 2:4]).all()
    assert np.isnan(go[0, 4:6, 2, :32]).all()      # the poisoned group
    fine = np.ones(go.shape, dtype=bool)
    fine[0, 2:4] = False
    fine[0, 4:6, 2, :] = False
    assert (np.abs(go - ro) <= eo + half_ulp_bf16(ro) * (1 + 2.0 ** -6))[fine].all()
    assert (np.abs(gl - rl) <= el)[0, [0, 1, 4, 5]].all()


@pytest.mark.parametrize("lens", [[33, 20, 5], [20, -1, 5], [20, 5, 2 ** 31 - 1], [-2 ** 31, 64, 1]])
def test_lengths_outside_the_bound(ab, lens):
    # the offending sequence gets NaN and is reported, the others their values
    import torch
    B, L = 3, 32
    q, k, v = case(11, B, 2, 2, 1, 64, 64)
    good = [0 <= l <= L for l in lens]
    out, lse = ab.alibi_attn_decode_kv4(bf16(q)[1], up(ref.pack(k, v)), lens=ints(lens), L=L)
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    want, wl = ab.alibi_attn_decode_kv4(bf16(q)[1], up(ref.pack(k, v)), lens=ints([l if g else 0 for l, g in zip(lens, good)]),
                                        L=L)
    ab.alibi_check_error()
    for b in range(B):
        if good[b]:
            assert torch.equal(out[b], want[b]) and torch.equal(lse[b], wl[b])
        else:
            assert bool(torch.isnan(out[b]).all()) and bool(torch.isnan(lse[b]).all())


def test_lse_may_be_left_out_and_outputs_given(ab):
    import ctypes
    import torch
    q, k, v = case(12, 1, 2, 2, 1, 64, 128)
    qd, cache = bf16(q)[1], up(ref.pack(k, v))
    want, wl = ab.alibi_attn_decode_kv4(qd, cache)
    out, lse = torch.full_like(want, 3.0), torch.full_like(wl, 3.0)
    r = ab.alibi_attn_decode_kv4(qd, cache, out=out, lse=lse)
    assert r[0] is out and r[1] is lse and torch.equal(out, want) and torch.equal(lse, wl)
    out.fill_(3.0)
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = ab.load().alibi_attn_decode_kv4(P(qd), P(cache), None, P(out), None, 1, 4, 2, 1, 64, 64, 128, None,
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    ab.alibi_check_error()
    assert st == 0 and torch.equal(out, want)


@pytest.mark.parametrize("B,Hkv,G,N,d", [(1, 2, 2, 8192, 128), (3, 4, 1, 700 // 32 * 32, 64)])
def test_repeated_calls_give_the_same_bits(ab, B, Hkv, G, N, d):
    import torch
    q, k, v = case(13, B, Hkv, G, 1, N, d)
    qd, cache = bf16(q)[1], up(ref.pack(k, v))
    first = ab.alibi_attn_decode_kv4(qd, cache)
    for _ in range(20):
        again = ab.alibi_attn_decode_kv4(qd, cache)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    ab.alibi_check_error()


def test_serving_steps_prompt_write_then_decode_in_a_graph(ab):
    # the run as a server makes it: a prompt is written, then every step writes one token and attends; the step is
    # captured once, with positions and lengths in device memory, and replayed over block boundaries
    import torch
    B, Hkv, G, N, d, P = 3, 2, 2, 160, 64, [5, 64, 90]
    steps = 40
    q, k, v = case(15, B, Hkv, G, steps, N, d)
    cache = ab.alibi_kv4_cache(B, Hkv, N, d)
    cache.fill_(0xFF)
    (_, kd), (_, vd) = bf16(k), bf16(v)
    ab.alibi_kv4_write(kd[:, :, :90].contiguous(), vd[:, :, :90].contiguous(), cache, count=ints(P))
    lens = ints(P)
    qs, ks, vs = bf16(q[:, :, :1])[1], kd[:, :, :1].contiguous(), vd[:, :, :1].contiguous()

    def step():
        ab.alibi_kv4_write(ks, vs, cache, pos=lens)
        lens.add_(1)
        return ab.alibi_attn_decode_kv4(qs, cache, lens=lens)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out, lse = step()
    kh, vh = ref.held(k), ref.held(v)
    for i in range(steps):
        qs.copy_(bf16(q[:, :, i:i + 1])[1])
        for b in range(B):
            ks[b].copy_(kd[b, :, P[b] + i:P[b] + i + 1])
            vs[b].copy_(vd[b, :, P[b] + i:P[b] + i + 1])
        g.replay()
        torch.cuda.synchronize()
        ro, rl, eo, el = ref.decode(q[:, :, i:i + 1], kh, vh, [p + i + 1 for p in P], oracle.slopes(Hkv * G))
        go, gl = host64(out), host64(lse)
        assert (np.abs(go - ro) <= eo + half_ulp_bf16(ro) * (1 + 2.0 ** -6)).all(), i
        assert (np.abs(gl - rl) <= el).all(), i
    ab.alibi_check_error()


@pytest.mark.parametrize("B,Hkv,G,N,d,T", [(2, 6, 2, 300, 64, 1), (1, 2, 4, 30000, 128, 1), (64, 8, 1, 2000, 128, 20),
                                           (1, 32, 1, 6000, 64, 3), (24, 7, 1, 40000, 32, 1)])
def test_calls_one_after_another_wait_for_each_other(ab, B, Hkv, G, N, d, T):
    # Every kernel begins while the one before it ends: write, decode, read back and torch's own kernels on the same
    # rows, positions and outputs give the same bits with and without a wait between any two of them.
    import torch
    g = torch.Generator(device="cuda").manual_seed(N)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    C, steps, D = -(-(N + 13 * T) // 32) * 32, 12, min(T, 16)
    k, v, new = rand(B, Hkv, N, d), rand(B, Hkv, N, d), rand(steps, 3, B, Hkv, T, d)
    q = rand(steps, B, Hkv * G, D, d)
    results = []
    for wait in (True, False):
        sync = torch.cuda.synchronize if wait else lambda: None
        cache = ab.alibi_kv4_cache(B, Hkv, C, d)
        cache.fill_(0xFF)
        ab.alibi_kv4_write(k, v, cache)
        pos, lens = ints([N] * B), ints([N + T] * B)
        row, kr, vr, qx = torch.empty_like(new[0, 0]), torch.empty_like(new[0, 0]), torch.empty_like(new[0, 0]), q[0].clone()
        got = []
        for i in range(steps):
            row.copy_(new[i, 0])
            sync()
            ab.alibi_kv4_write(row, new[i, 1], cache, pos=pos)
            sync()
            qx.copy_(q[i])
            sync()
            out, lse = ab.alibi_attn_decode_kv4(qx, cache, lens=lens, L=C)
            sync()
            qx.zero_()
            row.fill_(float("nan"))
            sync()
            ab.alibi_kv4_read(cache, kr, vr, pos=pos)
            sync()
            again = ab.alibi_attn_decode_kv4(q[i], cache, lens=lens, L=C)
            sync()
            ab.alibi_kv4_write(new[i, 2], kr, cache, pos=pos)  # over what the decode before it reads
            sync()
            got += [out, lse, again[0], again[1], kr.clone(), vr.clone()]
            pos += T
            lens += T
            sync()
        torch.cuda.synchronize()
        got.append(cache)
        results.append(got)
    ab.alibi_check_error()
    for i, (a, b) in enumerate(zip(*results)):
        assert torch.equal(a, b), i
    for out, again in zip(results[0][0:-1:6], results[0][2:-1:6]):
        assert torch.equal(out, again)


def test_drafted_tokens_equal_single_steps(ab):
    # four new tokens at once see what four single calls with growing lengths see
    q, k, v = case(16, 2, 2, 2, 4, 352, 128)
    compare(ab, q, k, v, [350, 37])
    cache = up(ref.pack(k, v))
    out, lse = (host64(t) for t in ab.alibi_attn_decode_kv4(bf16(q)[1], cache, lens=ints([350, 37])))
    for t in range(4):
        o1, l1 = (host64(x) for x in ab.alibi_attn_decode_kv4(bf16(q[:, :, t:t + 1])[1], cache,
                                                              lens=ints([347 + t, 34 + t])))
        assert np.abs(o1[:, :, 0] - out[:, :, t]).max() <= 2.0 ** -6 and np.abs(l1[:, :, 0] - lse[:, :, t]).max() <= 1e-4


def test_agrees_with_the_bf16_decode_and_the_fp32_prefill(ab):
    # over the values read back: the bf16 decode within the rounding of those values, the fp32 prefill's last row
    # within the kernel's own bounds
    import torch
    B, H, N, d = 2, 6, 224, 64
    q, k, v = case(17, B, H, 1, 1, N, d)
    qd, cache = bf16(q)[1], up(ref.pack(k, v))
    out, lse = ab.alibi_attn_decode_kv4(qd, cache)
    kf, vf = torch.empty(B, H, N, d, device="cuda"), torch.empty(B, H, N, d, device="cuda")
    ab.alibi_kv4_read(cache, kf, vf)
    qf = torch.zeros_like(kf)
    qf[:, :, -1] = qd[:, :, 0].float()
    o32, l32 = ab.alibi_attn_fwd_f32(qf, kf, vf)
    ab.alibi_check_error()
    ro, rl, eo, el = ref.decode(q, ref.held(k), ref.held(v), [N] * B, oracle.slopes(H))
    assert (np.abs(host64(out) - host64(o32[:, :, -1:])) <= eo + half_ulp_bf16(ro) * (1 + 2.0 ** -6) + 1e-5).all()
    assert (np.abs(host64(lse) - host64(l32[:, :, -1:])) <= el + 1e-5).all()
    kb, vb = torch.empty_like(kf, dtype=torch.bfloat16), torch.empty_like(kf, dtype=torch.bfloat16)
    ab.alibi_kv4_read(cache, kb, vb)
    o16 = ab.alibi_attn_decode(qd[:, :, 0].contiguous(), kb, vb)
    # keys off by 2^-8 relative: logits by up to 2^-8 sum |q k| / sqrt(d)
    x = 2.0 ** -8 * (np.abs(q[:, :, 0, None]) * np.abs(ref.held(k))).sum(-1).max() / np.sqrt(d)
    assert np.abs(host64(o16) - host64(out)[:, :, 0]).max() <= (2 * x + 2.0 ** -7) * np.abs(v).max()


def test_two_streams_and_two_graphs_at_once(ab):
    # calls in flight at the same time share nothing: each gives what it gives alone
    import torch
    jobs = []
    for i, (B, Hkv, G, N, d) in enumerate([(1, 2, 2, 20000, 128), (1, 3, 1, 30016, 64)]):
        q, k, v = case(20 + i, B, Hkv, G, 1, N, d)
        qd, cache = bf16(q)[1], up(ref.pack(k, v))
        want = ab.alibi_attn_decode_kv4(qd, cache)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = ab.alibi_attn_decode_kv4(qd, cache)
        jobs.append((qd, cache, want, g, got, torch.cuda.Stream()))
    for _ in range(20):
        eager = []
        for qd, cache, want, g, got, s in jobs:
            with torch.cuda.stream(s):
                g.replay()
                eager.append(ab.alibi_attn_decode_kv4(qd, cache))
        torch.cuda.synchronize()
        for (qd, cache, want, g, got, s), e in zip(jobs, eager):
            assert all(torch.equal(a, b) for a, b in zip(want, got)) and all(torch.equal(a, b) for a, b in zip(want, e))
    ab.alibi_check_error()


def test_calls_from_several_host_threads(ab):
    # the library's calls release the interpreter's lock: four threads, each on a stream of its own, give what one gives
    import threading

    import torch
    jobs, failed = [], []
    for i, (B, Hkv, G, N, d) in enumerate([(1, 2, 2, 20000, 128), (1, 32, 1, 3000, 64), (3, 4, 8, 100, 32), (2, 40, 1, 5000, 128)]):
        g = torch.Generator(device="cuda").manual_seed(i)
        k, v = (torch.randn(B, Hkv, N, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        q = torch.randn(B, Hkv * G, 1, d, generator=g, device="cuda", dtype=torch.bfloat16)
        cache = ab.alibi_kv4_cache(B, Hkv, -(-N // 32) * 32, d)
        ab.alibi_kv4_write(k, v, cache)
        jobs.append((k, v, q, cache, ab.alibi_attn_decode_kv4(q, cache, L=N)))
    torch.cuda.synchronize()

    def work(k, v, q, cache, want):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    mine = torch.full_like(cache, 0xFF)
                    ab.alibi_kv4_write(k, v, mine)
                    out, lse = ab.alibi_attn_decode_kv4(q, mine, L=k.shape[2])
                    kr, vr = ab.alibi_kv4_read(mine, torch.empty_like(k), torch.empty_like(v))
                    k2, v2 = ab.alibi_kv4_read(cache, torch.empty_like(k), torch.empty_like(v))
                    stream.synchronize()
                    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
                    assert torch.equal(kr, k2) and torch.equal(vr, v2)
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    ab.alibi_check_error()


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_made_for_another_stream_belong_to_it(ab, handle):
    # Memory that the current stream has just let go of may still be in use there, so a call on another stream must
    # not get its outputs from it; and memory that it writes is handed out again behind it.
    import torch
    q, k, v = case(24, 2, 2, 2, 1, 96, 128)
    qd, cache = bf16(q)[1], up(ref.pack(k, v))
    want, want_lse = ab.alibi_attn_decode_kv4(qd, cache)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    gone = [torch.empty_like(want), torch.empty_like(want_lse)]
    was = {t.data_ptr() for t in gone}
    del gone
    out, lse = ab.alibi_attn_decode_kv4(qd, cache, stream=side.cuda_stream if handle else side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert out.data_ptr() not in was and lse.data_ptr() not in was
    assert torch.cuda.current_stream() != side
    mine = {out.data_ptr(), lse.data_ptr()}
    del out, lse
    with torch.cuda.stream(side):
        assert {torch.empty_like(want).data_ptr(), torch.empty_like(want_lse).data_ptr()} & mine
    same = ab.alibi_attn_decode_kv4(qd, cache, stream=torch.cuda.current_stream())[0]
    torch.cuda.synchronize()
    assert torch.equal(same, want)
    ab.alibi_check_error()


@pytest.mark.parametrize("B,Hkv,G,N,d", [(2, 5, 1, 300, 64), (1, 32, 2, 2048, 128), (1, 2, 8, 30000, 128),
                                         (24, 7, 1, 14336, 32), (24, 7, 1, 40000, 32)])
def test_graph_of_every_way_follows_lengths_on_the_device(ab, B, Hkv, G, N, d):
    # captured once for the capacity, replayed while the lengths change (whole chunks, clusters, slices, shares)
    import torch
    g = torch.Generator(device="cuda").manual_seed(N)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    cache = ab.alibi_kv4_cache(B, Hkv, -(-N // 32) * 32, d)
    ab.alibi_kv4_write(rand(B, Hkv, N, d), rand(B, Hkv, N, d), cache)
    q, lens = rand(B, Hkv * G, 1, d), ints([N] * B)
    ab.alibi_attn_decode_kv4(q, cache, lens=lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = ab.alibi_attn_decode_kv4(q, cache, lens=lens)
    for new in ([N] * B, [1 + b for b in range(B)], [N - 13 * b for b in range(B)], [0] * B, [(N * b) // B for b in range(B)]):
        lens.copy_(ints(new))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        want, wl = ab.alibi_attn_decode_kv4(q, cache, lens=lens)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        assert bool((lse[[b for b in range(B) if new[b] == 0]] == -np.inf).all())
    ab.alibi_check_error()


FIRST_CALL = """
import torch
import alibi_positional_bias_gb300 as ab
B, H, N, d = {0}
k = torch.randn(B, H, N, d, device="cuda", dtype=torch.bfloat16)
v, q = torch.randn_like(k), torch.randn(B, H, 1, d, device="cuda", dtype=torch.bfloat16)
cache = torch.full((B, H, -(-N // 32), 36 * max(d, 32)), 255, dtype=torch.uint8, device="cuda")
kr, vr = torch.empty_like(k), torch.empty_like(v)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    ab.alibi_kv4_write(k, v, cache)
    out, lse = ab.alibi_attn_decode_kv4(q, cache, L=N)
    ab.alibi_kv4_read(cache, kr, vr)
graph.replay()
want, wl = ab.alibi_attn_decode_kv4(q, cache, L=N)
torch.cuda.synchronize()
assert torch.equal(out, want) and torch.equal(lse, wl) and bool(torch.isfinite(out).all())
ab.alibi_check_error()
"""


@pytest.mark.parametrize("shape", [(1, 6, 100, 64), (1, 32, 3000, 128), (1, 2, 60000, 128), (24, 7, 40000, 32)])
def test_first_calls_of_a_process_in_a_graph(shape):
    # whole chunks, clusters, slices and shares, captured before the library has made any call on the device
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(shape)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_every_way_with_a_nan_far_back(ab):
    # a NaN value whose weight has long vanished still reaches its group, as 0 x NaN does in the bf16 decode; NaN rows past
    # the length do not
    import torch
    for B, Hkv, N, d in ((1, 3, 200, 128), (1, 32, 4096, 128), (1, 2, 20000, 64), (24, 7, 14336, 32), (1, 2, 130000, 64),
                         (24, 7, 40000, 32)):
        k = torch.randn(B, Hkv, N, d, device="cuda", dtype=torch.bfloat16)
        v = torch.randn(B, Hkv, N, d, device="cuda", dtype=torch.bfloat16)
        v[:, 1, 3, 2] = float("nan")
        v[:, 0, N - 1, 2] = float("nan")
        k[:, 0, N - 1, 2] = float("nan")
        cache = ab.alibi_kv4_cache(B, Hkv, -(-N // 32) * 32, d)
        ab.alibi_kv4_write(k, v, cache)
        q = torch.randn(B, Hkv, 1, d, device="cuda", dtype=torch.bfloat16)
        out, lse = ab.alibi_attn_decode_kv4(q, cache, lens=ints([N - 1] * B), slopes=[1.0] * Hkv)
        ab.alibi_check_error()
        nan = torch.isnan(out)
        assert bool(nan[:, 1, 0, :32].all()) and not bool(nan[:, 1, 0, 32:].any())
        assert not bool(nan[:, [0] + list(range(2, Hkv))].any()) and not bool(torch.isnan(lse).any())


def test_very_large_slopes(ab):
    # only the query's own token is left, whatever the slope
    import torch
    q, k, v = case(40, 1, 4, 1, 1, 300, 64)
    cache = up(ref.pack(k, v))
    out, lse = ab.alibi_attn_decode_kv4(bf16(q)[1], cache, lens=ints([300]), slopes=[1e20, 1e30, 3e38, 3.4e38])
    ab.alibi_check_error()
    want = torch.from_numpy(ref.held(v)[:, :, 299].astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(out[:, :, 0].cpu(), want)
    x = (q[:, :, 0] * ref.held(k)[:, :, 299]).sum(-1) / 8.0
    assert np.abs(host64(lse)[:, :, 0] - x).max() <= 1e-5


def test_more_heads_than_grid_rows(ab):
    # 71680 (b, head) pairs
    import torch
    B, H, N, d = 1024, 70, 32, 16
    rng = np.random.default_rng(30)
    q, k, v = (gen.make_tensor(rng.standard_normal(s), s, "bf16").f32.astype(np.float64)
               for s in ((B, H, 1, d), (B, H, N, d), (B, H, N, d)))
    lens = rng.integers(0, N + 1, size=B)
    out, lse = ab.alibi_attn_decode_kv4(bf16(q)[1], up(ref.pack(k, v)), lens=ints(lens.tolist()))
    ab.alibi_check_error()
    pick = [0, 1, 511, 936, 937, 1023]
    ro, rl, eo, el = ref.decode(q[pick], ref.held(k[pick]), ref.held(v[pick]), lens[pick], oracle.slopes(H))
    assert (np.abs(host64(out)[pick] - ro) <= eo + half_ulp_bf16(ro) * (1 + 2.0 ** -6)).all()
    seen = ~np.isinf(rl)
    assert (np.abs(host64(lse)[pick][seen] - rl[seen]) <= el[seen]).all()
    assert np.array_equal(np.isinf(host64(lse)), np.broadcast_to((lens == 0)[:, None, None], (B, H, 1)))


def test_offsets_beyond_32_bits(ab):
    # 8 KV heads of 2^21 tokens: the last head's rows lie past 2^31 bytes. All rows are zeros but the newest
    import torch
    Hkv, C, d, n = 8, 1 << 21, 128, 48
    cache = ab.alibi_kv4_cache(1, Hkv, C, d)
    cache.zero_()  # scale 0: every value 0
    q, k, v = case(31, 1, Hkv, 1, 1, n, d)
    ab.alibi_kv4_write(bf16(k)[1], bf16(v)[1], cache, pos=ints([C - n]))
    m = np.full(Hkv, 2.0 ** -6)
    out, lse = ab.alibi_attn_decode_kv4(bf16(q)[1], cache, slopes=m.astype(np.float32))
    ab.alibi_check_error()
    # rows before the newest n: values 0 and logits -m (i - j), down to where they vanish
    pad = 8192
    K = np.concatenate([np.zeros((1, Hkv, pad, d)), ref.held(k)], axis=2)
    V = np.concatenate([np.zeros((1, Hkv, pad, d)), ref.held(v)], axis=2)
    ro, rl, eo, el = ref.decode(q, K, V, [pad + n], m)
    assert (np.abs(host64(out) - ro) <= eo + half_ulp_bf16(ro) * (1 + 2.0 ** -6)).all()
    assert (np.abs(host64(lse) - rl) <= el).all()
    del cache
    torch.cuda.empty_cache()


def run_picked(ab, seed, B, Hkv, G, T, N, d, lens, L, picks, steep=None):
    """A case too large for a whole reference: keys and values are made and written on the GPU, and the rows of some
    (sequence, KV head) pairs are compared; all outputs have to be finite, and empty where no token is."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    C = -(-N // 32) * 32
    k, v, q = rand(B, Hkv, N, d), rand(B, Hkv, N, d), rand(B, Hkv * G, T, d)
    cache = ab.alibi_kv4_cache(B, Hkv, C, d)
    cache.fill_(0xFF)
    true = [N] * B if lens is None else lens
    ab.alibi_kv4_write(k, v, cache, count=ints(true))
    m = None if steep is None else np.full(Hkv * G, steep, dtype=np.float32)
    out, lse = ab.alibi_attn_decode_kv4(q, cache, lens=None if lens is None else ints(lens), L=L, slopes=m)
    ab.alibi_check_error()
    assert bool(torch.isfinite(out).all())
    empty = torch.tensor([[n - T + t < 0 for t in range(T)] for n in true], device="cuda")[:, None]
    assert torch.equal(torch.isinf(lse), empty.expand_as(lse)) and bool((out.transpose(2, 3)[empty[:, :, None].expand(
        B, Hkv * G, d, T)] == 0).all())
    slopes = oracle.slopes(Hkv * G) if m is None else m.astype(np.float64)
    for b, h in picks:
        n, rows = true[b], slice(h * G, (h + 1) * G)
        x = [host64(t) for t in (q[b:b + 1, rows], k[b:b + 1, h:h + 1, :max(n, 1)], v[b:b + 1, h:h + 1, :max(n, 1)])]
        ro, rl, eo, el = ref.decode(x[0], ref.held(x[1]), ref.held(x[2]), [n], slopes[rows])
        go, gl = host64(out[b:b + 1, rows]), host64(lse[b:b + 1, rows])
        assert (np.abs(go - ro) <= eo + half_ulp_bf16(ro) * (1 + 2.0 ** -6)).all(), (b, h)
        seen = ~np.isinf(rl)
        assert (np.abs(gl[seen] - rl[seen]) <= el[seen]).all(), (b, h)


# Whole chunks, clusters, slices and equal shares (the ways on 152 SMs: tests/test_kv4_deal.py); more and fewer than 32
# sequences; very unequal lengths; lengths far below the bound that the work was planned for
@pytest.mark.parametrize("B,Hkv,G,T,N,d,kind,L", [
    (24, 7, 1, 1, 14336, 32, "ragged", None),      # whole, more CTAs than SMs
    (40, 5, 8, 1, 16384, 64, "ragged", None),      # two columns per lane
    (40, 5, 8, 1, 16384, 64, None, 16384),         # one length for all
    (8, 38, 1, 1, 4096, 128, "ragged", None),      # whole, one round
    (40, 2, 1, 1, 8192, 128, "ragged", None),      # clusters
    (24, 7, 1, 1, 40000, 32, "ragged", None),      # shares
    (24, 7, 1, 1, 40000, 32, "one long", 40000),
    (24, 7, 1, 1, 40000, 32, "short", 40000),
    (40, 4, 8, 1, 30000, 64, "ragged", None),      # shares, two columns per lane, more than 32 sequences
    (40, 4, 8, 1, 30000, 64, None, 30000),         # one length for all
    (50, 1, 1, 1, 128000, 32, "ragged", None),     # slices, more than 32 sequences
    (50, 1, 2, 3, 64000, 64, "one long", 64000),
    (50, 1, 2, 3, 64000, 64, "short", 64000),
    (2, 1, 4, 2, 80000, 64, "ragged", None),       # slices
    (40, 2, 2, 3, 8192, 64, "one long", 8192),     # one sequence of 8192 among sequences of one token
    (3, 2, 1, 1, 16384, 128, "one long", 16384),
    (24, 7, 1, 1, 14336, 32, "one long", 14336),
    (6, 4, 2, 2, 16384, 64, "short", 16384),       # planned for 16384, a few tokens each
    (40, 4, 1, 1, 20000, 32, "short", 20000),
    (24, 9, 1, 1, 14000, 32, "short", 14000),
    (1, 2, 64, 2, 4096, 64, None, 4096),           # 16 chunks of a head
    (1, 1, 1, 1, 300000, 32, None, 300000),
])
def test_ways_of_dealing(ab, B, Hkv, G, T, N, d, kind, L):
    lens = {None: None, "ragged": [max(0, N - 1 - (N * 7 * b // 11) % N) if b % 5 else b % 3 for b in range(B)],
            "one long": [N if b == B // 2 else 1 for b in range(B)], "short": [(7 * b) % 40 for b in range(B)]}[kind]
    picks = sorted({(0, 0), (B - 1, Hkv - 1), (B // 2, 0), (B // 3, Hkv // 2), (B // 2, Hkv - 1)})
    run_picked(ab, 1000 + B + N, B, Hkv, G, T, N, d, lens, L, picks)


@pytest.mark.parametrize("B,Hkv,G,T,N,d", [(24, 7, 1, 1, 14336, 32), (3, 4, 8, 1, 8192, 128), (40, 5, 2, 4, 1000, 64),
                                             (24, 7, 1, 1, 40000, 32), (1, 1, 1, 1, 80000, 64)])
def test_ways_of_dealing_without_bias(ab, B, Hkv, G, T, N, d):
    # no bias: no block's weights vanish, long sums of small weights
    lens = [N - 17 * b for b in range(B)]
    run_picked(ab, 77, B, Hkv, G, T, N, d, lens, None, [(0, 0), (B - 1, Hkv - 1)], steep=0.0)


def test_repeated_calls_of_every_way_give_the_same_bits(ab):
    import torch
    for B, Hkv, N, d in ((24, 7, 14336, 32), (4, 2, 8192, 128), (8, 38, 600, 64), (24, 7, 40000, 32), (1, 1, 80000, 64)):
        k = torch.randn(B, Hkv, N, d, device="cuda", dtype=torch.bfloat16)
        cache = ab.alibi_kv4_cache(B, Hkv, -(-N // 32) * 32, d)
        ab.alibi_kv4_write(k, torch.flip(k, dims=[2]).contiguous(), cache)
        q = torch.randn(B, Hkv, 1, d, device="cuda", dtype=torch.bfloat16)
        lens = ints([N - 31 * b for b in range(B)])
        first = ab.alibi_attn_decode_kv4(q, cache, lens=lens)
        for _ in range(10):
            again = ab.alibi_attn_decode_kv4(q, cache, lens=lens)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    ab.alibi_check_error()


def test_binding_refusals(ab):
    import torch
    q = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    c = ab.alibi_kv4_cache(2, 2, 64, 64)
    for bad in (q.float(), q.half()):
        with pytest.raises(TypeError):
            ab.alibi_attn_decode_kv4(bad, c)
    for bad in (q[:1], q[..., :32].contiguous(), q[0, 0], q.transpose(0, 1)):
        with pytest.raises(ValueError):
            ab.alibi_attn_decode_kv4(bad, c)
    with pytest.raises(TypeError):
        ab.alibi_attn_decode_kv4(q, c, lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ab.alibi_attn_decode_kv4(q, c, lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        ab.alibi_attn_decode_kv4(q, c, slopes=[0.5] * 3)
    with pytest.raises(TypeError):
        ab.alibi_attn_decode_kv4(q, c, out=q.float())
    for L in (0, 65, -1):
        with pytest.raises(ab.AlibiError):
            ab.alibi_attn_decode_kv4(q, c, L=L)
    with pytest.raises(ab.AlibiError):  # 3 query heads over 2 KV heads
        ab.alibi_attn_decode_kv4(q[:, :3].contiguous(), c)
    with pytest.raises(ab.AlibiError):  # 17 new tokens
        ab.alibi_attn_decode_kv4(torch.zeros(2, 4, 17, 64, dtype=torch.bfloat16, device="cuda"), c)
