"""Writing the 4-bit KV cache and reading it back (alibi_kv4_write, alibi_kv4_read): byte for byte against
the plain form of tests/kv4_ref.py."""
import numpy as np
import pytest

import alibi_inputs as gen
import kv4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ab():
    import alibi_positional_bias_gb300 as ab
    ab.load()
    return ab


def bf16(x):
    """Exact bf16 values (float64) and the CUDA tensor of them."""
    import torch
    t = gen.make_tensor(np.asarray(x, dtype=np.float32), np.shape(x), "bf16")
    return t.f32.astype(np.float64), torch.from_numpy(t.bf16.view(np.int16)).view(torch.bfloat16).cuda()


def ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(B, H, C, d, byte=0xA5):
    return np.full((B, H, C // 32, ref.block_bytes(d)), byte, dtype=np.uint8)


def up(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check_write(ab, k, v, cache, pos, count):
    """Write k, v into a copy of the numpy cache on the GPU and compare every byte."""
    (kf, kd), (vf, vd) = bf16(k), bf16(v)
    B, _, T, _ = kf.shape
    dev = up(cache)
    ab.alibi_kv4_write(kd, vd, dev, pos=None if pos is None else ints(pos), count=None if count is None else ints(count))
    ab.alibi_check_error()
    want = cache.copy()
    ref.write(want, kf, vf, [0] * B if pos is None else pos, [T] * B if count is None else count)
    assert np.array_equal(dev.cpu().numpy(), want)
    return dev, kf, vf


def check_read(ab, dev, k, v, pos, count):
    """Read the rows back in both types; tokens past the counts keep what was there."""
    import torch
    B, H, T, d = k.shape
    hk, hv = ref.held(k), ref.held(v)
    for dt in (torch.float32, torch.bfloat16):
        ko = torch.full((B, H, T, d), 7.0, dtype=dt, device="cuda")
        vo = torch.full_like(ko, -3.0)
        r = ab.alibi_kv4_read(dev, ko, vo, pos=None if pos is None else ints(pos),
                              count=None if count is None else ints(count))
        ab.alibi_check_error()
        assert r[0] is ko and r[1] is vo
        for got, h, was in ((ko, hk, 7.0), (vo, hv, -3.0)):
            want = torch.from_numpy(h.astype(np.float32)).to(dt)  # exact in fp32; one rounding to bf16
            for b in range(B):
                n = T if count is None else count[b]
                assert torch.equal(got[b, :, :n].cpu(), want[b, :, :n])
                assert bool((got[b, :, n:] == was).all())


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("B,H,T,C,pos,count", [
    (1, 1, 1, 32, None, None), (1, 2, 1, 64, [31], None), (1, 2, 1, 64, [32], None), (2, 3, 1, 96, [95, 0], [1, 0]),
    (1, 1, 32, 32, None, None), (2, 2, 33, 96, [31, 1], [33, 2]), (3, 2, 70, 160, [90, 0, 17], [70, 69, 0]),
    (1, 3, 128, 128, None, None), (2, 1, 15, 32, [17, 16], [15, 15]), (1, 2, 200, 256, [56], [200]),
    (2, 3, 3, 64, [30, 61], None), (3, 1, 2, 64, [64, 62, 31], [0, 2, 1]), (4, 2, 4, 64, [0, 30, 60, 64], [4, 4, 4, 0]),
    (3, 2, 40, 96, [96, 57, 8], [0, 39, 40])])
def test_write_and_read(ab, d, B, H, T, C, pos, count):
    rng = np.random.default_rng(B + 10 * T + d)
    k, v = rng.standard_normal((B, H, T, d)) * 3, rng.standard_normal((B, H, T, d))
    dev, kf, vf = check_write(ab, k, v, filled(B, H, C, d), pos, count)
    check_read(ab, dev, kf, vf, pos, count)


@pytest.mark.parametrize("d", [16, 32])
@pytest.mark.parametrize("T,start", [(1000, 0), (1000, 31), (97, 64), (16, 120), (33, 1)])
def test_runs_of_blocks_equal_single_ones(ab, d, T, start):
    # many heads, so that a CTA takes a run of blocks, against the same rows of few heads, a block each
    import torch
    B, H, C = 40, 60, 1056
    k = torch.randn(B, H, T, d, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(B, H, T, d, device="cuda", dtype=torch.bfloat16)
    pos = ints([start + (3 * b if start + 3 * (B - 1) + T <= C else b % 2) for b in range(B)])
    count = ints([T - b % 7 for b in range(B)])
    cache = ab.alibi_kv4_cache(B, H, C, d)
    cache.fill_(0xA5)
    ab.alibi_kv4_write(k, v, cache, pos=pos, count=count)
    kr, vr = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    ab.alibi_kv4_read(cache, kr, vr, pos=pos, count=count)
    for b, h in ((0, 0), (1, 59), (17, 30), (39, 59), (6, 1)):
        one = ab.alibi_kv4_cache(1, 1, C, d)
        one.fill_(0xA5)
        rows = [x[b:b + 1, h:h + 1].contiguous() for x in (k, v)]
        ab.alibi_kv4_write(*rows, one, pos=pos[b:b + 1].clone(), count=count[b:b + 1].clone())
        assert torch.equal(one, cache[b:b + 1, h:h + 1])
        got = [torch.full_like(x, 7.0) for x in rows]
        ab.alibi_kv4_read(one, *got, pos=pos[b:b + 1].clone(), count=count[b:b + 1].clone())
        assert torch.equal(got[0], kr[b:b + 1, h:h + 1]) and torch.equal(got[1], vr[b:b + 1, h:h + 1])
    ab.alibi_check_error()


def test_appending_tokens_equals_writing_them_at_once(ab):
    import torch
    rng = np.random.default_rng(3)
    B, H, N, d = 2, 3, 100, 64
    (_, k), (_, v) = bf16(rng.standard_normal((B, H, N, d))), bf16(rng.standard_normal((B, H, N, d)))
    whole, steps = up(filled(B, H, 128, d)), up(filled(B, H, 128, d))
    ab.alibi_kv4_write(k, v, whole)
    at = 0
    for n in (1, 30, 1, 1, 33, 16, 18):
        ab.alibi_kv4_write(k[:, :, at:at + n].contiguous(), v[:, :, at:at + n].contiguous(), steps, pos=ints([at] * B))
        at += n
    ab.alibi_check_error()
    assert at == N and torch.equal(whole, steps)


def test_every_quotient_of_two_bf16(ab):
    # x_m with each of the 128 significands, and every bf16 x with |x| in (2^-12 |x_m|, |x_m|], of both signs: every
    # tie and every near tie that a group can hold
    rows = []
    for S in range(128, 256):
        xm = S * 2.0 ** -7
        x = np.concatenate([np.arange(128, 256) * 2.0 ** (-7 - e) for e in range(13)])
        x = x[x <= xm]
        x = np.concatenate([x, -x[x < xm]])
        x = np.concatenate([x, np.zeros(-len(x) % 31)]).reshape(-1, 31)
        sign = 1.0 if S % 2 else -1.0  # -x_m is the scale's element when no +x_m is there
        rows.append(np.concatenate([sign * x, np.full((len(x), 1), sign * xm)], axis=1))
    x = np.concatenate(rows)
    x = np.concatenate([x, np.zeros((-len(x) % 32, 32))])[None, None]
    dev, kf, vf = check_write(ab, x, -x, filled(1, 1, x.shape[2], 32), None, None)
    check_read(ab, dev, kf, vf, None, None)


def test_values_at_the_edges(ab):
    big, tiny = 3.3895313892515355e38, 2.0 ** -133  # largest and smallest bf16
    g = []
    for vals in ([0.0], [-0.0, 0.0], [1.0, -1.0], [-1.0, 1.0], [big, -big], [-big, tiny], [tiny, -tiny], [2.0 ** -100],
                 [-(2.0 ** -100), 2.0 ** -101], [2.0 ** -100 * (1 - 2.0 ** -8)], [2.0 ** -99, 2.0 ** -110],
                 [np.inf, 1.0], [-np.inf, 2.0], [np.nan, 1.0], [np.inf, -np.inf], [5.0] * 32, [-5.0] * 32,
                 [1.0, 2.0 ** -5, -(2.0 ** -4), 0.9375, -0.9375]):
        r = np.zeros(32)
        r[-len(vals):] = vals
        g.append(r)
    x = np.stack(g).astype(np.float32)
    for d, rows in ((32, x), (128, np.concatenate([x, x, x, x], axis=1)[:, np.roll(np.arange(128), 32)])):
        (kf, kd), (vf, vd) = bf16(rows[None, None]), bf16(-rows[None, None])
        import torch
        dev = up(filled(1, 1, 32, d))
        ab.alibi_kv4_write(kd, vd, dev)
        ko = torch.empty(kf.shape, dtype=torch.float32, device="cuda")
        vo = torch.empty_like(ko)
        ab.alibi_kv4_read(dev, ko, vo)
        ab.alibi_check_error()
        for got, f in ((ko, kf), (vo, vf)):
            want = ref.held(f)
            got = got.cpu().numpy().astype(np.float64)
            assert np.array_equal(np.isnan(got), np.isnan(want))
            assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))
    # one NaN poisons its own group only
    r = np.ones((1, 1, 1, 128))
    r[..., 40] = np.nan
    h = ref.held(r)
    assert np.isnan(h[..., 32:64]).all() and np.isfinite(np.delete(h, np.s_[32:64], axis=-1)).all()


@pytest.mark.parametrize("pos,count", [([-1, 0, 3], [1, 1, 1]), ([0, 63, 0], [2, 2, 2]), ([0, 0, 5], [4, -1, 4]),
                                       ([0, 0, 0], [4, 5, 1]), ([2 ** 31 - 1, 0, 0], [4, 4, 4]),
                                       ([-2 ** 31, 61, 60], [4, 4, 4])])
def test_spans_outside_the_cache_are_left_out(ab, pos, count):
    # the offending sequence is left out whole and reported; the others are written and read as always
    import torch
    rng = np.random.default_rng(8)
    B, H, T, C, d = 3, 2, 4, 64, 64
    (kf, kd), (vf, vd) = bf16(rng.standard_normal((B, H, T, d))), bf16(rng.standard_normal((B, H, T, d)))
    fits = [p >= 0 and 0 <= c <= T and p + c <= C for p, c in zip(pos, count)]
    assert not all(fits)
    cache = filled(B, H, C, d)
    dev = up(cache)
    ab.alibi_kv4_write(kd, vd, dev, pos=ints(pos), count=ints(count))
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    ref.write(cache, kf, vf, [p if f else 0 for p, f in zip(pos, fits)], [c if f else 0 for c, f in zip(count, fits)])
    assert np.array_equal(dev.cpu().numpy(), cache)
    ko, vo = torch.full_like(kd, 9.0), torch.full_like(kd, 9.0)
    ab.alibi_kv4_read(dev, ko, vo, pos=ints(pos), count=ints(count))
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    for b in range(B):
        n = count[b] if fits[b] else 0
        want = torch.from_numpy(ref.held(kf[b, :, :n]).astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(ko[b, :, :n].cpu(), want) and bool((ko[b, :, n:] == 9.0).all())
    ab.alibi_check_error()  # collected: nothing is left


def test_graph_replay_follows_positions_on_the_device(ab):
    import torch
    rng = np.random.default_rng(9)
    B, H, C, d = 2, 2, 64, 128
    (_, k), (_, v) = bf16(rng.standard_normal((B, H, 1, d))), bf16(rng.standard_normal((B, H, 1, d)))
    pos = ints([0, 29])
    dev, want = up(filled(B, H, C, d)), filled(B, H, C, d)
    ab.alibi_kv4_write(k, v, dev, pos=pos, count=ints([0, 0]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ab.alibi_kv4_write(k, v, dev, pos=pos)
        pos.add_(1)
    for i in range(5):
        (kf, kn), (vf, vn) = bf16(rng.standard_normal((B, H, 1, d))), bf16(rng.standard_normal((B, H, 1, d)))
        k.copy_(kn), v.copy_(vn)
        g.replay()
        torch.cuda.synchronize()
        ref.write(want, kf, vf, [i, 29 + i], [1, 1])
    ab.alibi_check_error()
    assert np.array_equal(dev.cpu().numpy(), want)


def test_calls_on_two_streams(ab):
    import torch
    rng = np.random.default_rng(10)
    B, H, T, d = 1, 4, 500, 64
    jobs = []
    for i in range(2):
        (kf, kd), (vf, vd) = bf16(rng.standard_normal((B, H, T, d))), bf16(rng.standard_normal((B, H, T, d)))
        jobs.append((kf, vf, kd, vd, up(filled(B, H, 512, d)), torch.cuda.Stream(), torch.empty(B, H, T, d, device="cuda"),
                     torch.empty(B, H, T, d, device="cuda")))
    torch.cuda.synchronize()
    for kf, vf, kd, vd, dev, s, ko, vo in jobs:
        ab.alibi_kv4_write(kd, vd, dev, stream=s)
        ab.alibi_kv4_read(dev, ko, vo, stream=s)
    torch.cuda.synchronize()
    ab.alibi_check_error()
    for kf, vf, _, _, _, _, ko, vo in jobs:
        assert np.array_equal(ko.cpu().numpy(), ref.held(kf).astype(np.float32))
        assert np.array_equal(vo.cpu().numpy(), ref.held(vf).astype(np.float32))


def test_offsets_beyond_32_bits(ab):
    # 8 heads of 2^21 tokens of d = 128: 2.4 GB of cache; the last rows of the last head lie past 2^31 bytes
    import torch
    H, C, d = 8, 1 << 21, 128
    cache = ab.alibi_kv4_cache(1, H, C, d)
    assert cache.numel() > 1 << 31
    cache[:, -1, -2:] = 0xA5
    rng = np.random.default_rng(11)
    (kf, kd), (vf, vd) = bf16(rng.standard_normal((1, H, 35, d))), bf16(rng.standard_normal((1, H, 35, d)))
    ab.alibi_kv4_write(kd, vd, cache, pos=ints([C - 35]))
    ko = torch.empty(1, H, 35, d, device="cuda")
    vo = torch.empty_like(ko)
    ab.alibi_kv4_read(cache, ko, vo, pos=ints([C - 35]))
    ab.alibi_check_error()
    assert np.array_equal(ko.cpu().numpy(), ref.held(kf).astype(np.float32))
    assert np.array_equal(vo.cpu().numpy(), ref.held(vf).astype(np.float32))
    want = filled(1, 1, 64, d)
    ref.write(want, kf[:, -1:], vf[:, -1:], [29], [35])
    assert np.array_equal(cache[:, -1:, -2:].cpu().numpy(), want)
    del cache
    torch.cuda.empty_cache()


def test_long_prompt_against_the_plain_form(ab):
    # a prompt that takes many blocks of every launch shape, from an odd row on, one head in full
    import torch
    rng = np.random.default_rng(12)
    B, H, T, C, d = 2, 5, 3001, 4096, 128
    (kf, kd), (vf, vd) = bf16(rng.standard_normal((B, H, T, d))), bf16(rng.standard_normal((B, H, T, d)))
    cache = filled(B, H, C, d)
    dev = up(cache)
    pos, count = [1, 1095], [3000, 3001]
    ab.alibi_kv4_write(kd, vd, dev, pos=ints(pos), count=ints(count))
    ko = torch.zeros(B, H, T, d, device="cuda")
    vo = torch.zeros_like(ko)
    ab.alibi_kv4_read(dev, ko, vo, pos=ints(pos), count=ints(count))
    ab.alibi_check_error()
    for b in range(B):
        n = count[b]
        assert np.array_equal(ko[b, :, :n].cpu().numpy(), ref.held(kf[b, :, :n]).astype(np.float32))
        assert np.array_equal(vo[b, :, :n].cpu().numpy(), ref.held(vf[b, :, :n]).astype(np.float32))
    assert bool((ko[0, :, 3000:] == 0).all())
    got = dev.cpu().numpy()
    assert (got[0, :, 94:] == 0xA5).all() and (got[1, :, :34] == 0xA5).all()  # blocks outside both spans


def test_binding_refusals(ab):
    import torch
    k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    c = ab.alibi_kv4_cache(2, 3, 32, 64)
    with pytest.raises(TypeError):
        ab.alibi_kv4_write(k.float(), k, c)
    with pytest.raises(ValueError):
        ab.alibi_kv4_write(k, k[:, :, :3], c)
    with pytest.raises(ValueError):
        ab.alibi_kv4_write(k.transpose(1, 2), k.transpose(1, 2), c)        # not contiguous
    with pytest.raises(ValueError):
        ab.alibi_kv4_write(k, k, c[:, :2])
    with pytest.raises(ValueError):
        ab.alibi_kv4_write(k, k, ab.alibi_kv4_cache(2, 3, 32, 128))
    with pytest.raises(TypeError):
        ab.alibi_kv4_write(k, k, c, pos=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ab.alibi_kv4_write(k, k, c, count=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ab.alibi_kv4_write(k, k, c, pos=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        ab.alibi_kv4_read(c, k, k.float())
    with pytest.raises(TypeError):
        ab.alibi_kv4_read(c, k.half(), k.half())
    with pytest.raises(ab.AlibiError):
        ab.alibi_kv4_write(torch.zeros(2, 3, 33, 64, dtype=torch.bfloat16, device="cuda"),
                           torch.zeros(2, 3, 33, 64, dtype=torch.bfloat16, device="cuda"), c)  # T beyond C
