"""The paged calls at sizes that the other files do not combine: random calls over every option, very many sequences, the most
query rows to one KV head, and the first calls of a process inside a graph's capture."""
import os
import subprocess
import sys

import numpy as np
import pytest

import oracle
import paged_ref as ref
import test_gpu_fwd_paged as prefill
import test_gpu_paged as decode
from paged_ref import ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ab():
    import alibi_positional_bias_gb300 as ab
    ab.load()
    return ab


def draw(rng, most):
    """Sizes of a call whose scores number at most `most`."""
    while True:
        B, Hkv, G = (int(2 ** rng.uniform(0, x)) for x in (3, 3, 4))
        d, S = int(rng.choice([16, 32, 64, 128])), int(2 ** rng.integers(3, 11))
        T, N = int(2 ** rng.uniform(0, 9)), int(2 ** rng.uniform(0, 13))
        if B * Hkv * G * min(T, N) * N <= most and B * Hkv * N * d <= 1 << 22:
            break
    H = Hkv * G
    m = [None, np.zeros(H), np.exp(rng.uniform(-9, 0, H)), np.exp(rng.uniform(0, 3, H))][int(rng.integers(4))]
    m = None if m is None else m.astype(np.float32)
    lens = [int(n) for n in rng.integers(0, N + 1, B)]
    lens[int(rng.integers(B))] = N
    layout = ref.LAYOUTS[int(rng.integers(len(ref.LAYOUTS)))]
    M = -(-N // S) + int(rng.integers(3))
    L = None if rng.integers(2) else int(rng.integers(N, M * S + 1))
    return dict(B=B, Hkv=Hkv, G=G, T=T, N=N, d=d, S=S, lens=lens, layout=layout, M=M, L=L,
                m=None if m is None else m.astype(np.float64), slopes=m)


@pytest.mark.parametrize("seed", range(40))
def test_random_decodes(ab, seed):
    rng = np.random.default_rng(1000 + seed)
    c = draw(rng, 1 << 21)
    T = 1 + c["T"] % 16 if seed % 2 else 1
    q, k, v = decode.case(seed, c["B"], c["Hkv"], c["G"], T, c["N"], c["d"], strong=float(rng.uniform(1, 4)))
    decode.compare(ab, q, k, v, c["lens"], c["S"], m=c["m"], slopes=c["slopes"], L=c["L"], M=c["M"], layout=c["layout"],
                   unused=[-1, 2 ** 31 - 1][seed % 2], what=str({x: c[x] for x in "B Hkv G N d S lens L M layout".split()}))


@pytest.mark.parametrize("seed", range(40))
def test_random_prefills(ab, seed):
    rng = np.random.default_rng(2000 + seed)
    c = draw(rng, 1 << 22)
    T = c["T"]
    counts = [int(n) for n in rng.integers(0, T + 1, c["B"])]
    counts = [min(n, x) if rng.integers(4) else n for n, x in zip(counts, c["lens"])]  # most begin at or past the first row
    q, k, v = prefill.case(seed, c["B"], c["Hkv"], c["G"], T, c["N"], c["d"], strong=float(rng.uniform(1, 4)))
    prefill.compare(ab, q, k, v, c["lens"], counts, c["S"], m=c["m"], slopes=c["slopes"], L=c["L"], M=c["M"], layout=c["layout"],
                    unused=[-1, 2 ** 31 - 1][seed % 2], what=str({x: c[x] for x in "B Hkv G T N d S lens L M layout".split()}))


@pytest.mark.parametrize("d", [16, 128])
def test_very_many_sequences(ab, d):
    # one token each but for every seventh, which has none: out is its value, exactly
    import torch
    B, S = 70001, 8
    kp, vp = ref.pools(B, 1, S, d, "heads")
    table = torch.randperm(B, device="cuda").to(torch.int32)[:, None].contiguous()
    k, v, q = (torch.randn(B, 1, 1, d, device="cuda").bfloat16() for _ in range(3))
    count = (torch.arange(B, device="cuda") % 7 != 0).to(torch.int32)
    ab.alibi_paged_append(k, v, kp, vp, table, count=count)
    want = torch.where(count[:, None, None, None] == 1, v, torch.zeros_like(v))
    some = count == 1
    for call, more in ((ab.alibi_attn_decode_paged, {}), (ab.alibi_attn_fwd_paged, {"count": count})):
        out, lse = call(q, kp, vp, table, lens=count, **more)
        ab.alibi_check_error()
        assert torch.equal(out[some], want[some]) and bool(torch.isfinite(lse[some]).all())
        if not more:
            assert torch.equal(out, want) and bool((lse[~some] == -np.inf).all())
    bad = ~some
    assert bool((kp[table[bad, 0].long(), :, 0] != kp[table[bad, 0].long(), :, 0]).all())  # pools are NaN where nothing was written


@pytest.mark.parametrize("T,N,d", [(16, 70, 64), (16, 33, 128), (13, 200, 16)])
def test_most_query_rows_of_a_head(ab, T, N, d):
    q, k, v = decode.case(N, 2, 1, 384, T, N, d)
    decode.compare(ab, q, k, v, [N, N // 2], 16)


FIRST_CALL = """
import torch
import alibi_positional_bias_gb300 as ab
B, Hkv, G, N, T, d = {0}
k, v = (torch.randn(B, Hkv, N, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
q1, q2 = (torch.randn(B, Hkv * G, t, d, device="cuda", dtype=torch.bfloat16) for t in (1, T))
S, M = 16, -(-N // 16)
pools = [torch.zeros(B * M, Hkv, S, d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
table = torch.randperm(B * M, device="cuda").to(torch.int32).view(B, M)
turned = torch.empty_like(q2)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    ab.alibi_paged_append(k, v, *pools, table)
    a = ab.alibi_attn_decode_paged(q1, *pools, table, L=N)
    b = ab.alibi_attn_fwd_paged(q2, *pools, table, L=N)
    ab.alibi_paged_append(k[:, :, -T:], v[:, :, -T:], *pools, table, rotate=16, q=q2, q_out=turned)
graph.replay()
torch.cuda.synchronize()
ab.alibi_paged_append(k, v, *pools, table)
wa, wb = ab.alibi_attn_decode_paged(q1, *pools, table, L=N), ab.alibi_attn_fwd_paged(q2, *pools, table, L=N)
wt = ab.alibi_paged_append(k[:, :, -T:], v[:, :, -T:], *pools, table, rotate=16, q=q2)
torch.cuda.synchronize()
for x, y in zip((*a, *b, turned), (*wa, *wb, wt)):
    assert torch.equal(x, y) and bool(torch.isfinite(x).all())
ab.alibi_check_error()
"""


@pytest.mark.parametrize("shape", [(1, 6, 1, 100, 3, 64), (1, 32, 1, 3000, 300, 128), (1, 2, 4, 60000, 20, 128), (9, 37, 1, 3000, 17, 32)])
def test_first_calls_of_a_process_in_a_graph(shape):
    # captured before the library has made any call on the device
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(shape)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("power", [-95, -40, 60, 96])
def test_magnitudes_of_values(ab, power):
    # out is linear in the values: with them times a power of two it is that power times the same bits
    import torch
    for B, Hkv, G, N, d in ((1, 2, 2, 700, 128), (1, 1, 4, 20000, 64), (2, 8, 1, 4100, 128)):
        q, k, v = decode.case(N, B, Hkv, G, 1, N, d)
        qd, (kp, vp, table) = decode.bf16(q)[1], ref.paged(k, v, [N] * B, 16)
        big = torch.ldexp(vp, torch.tensor(power, device="cuda")).to(torch.bfloat16)
        for call, x in ((ab.alibi_attn_decode_paged, qd), (ab.alibi_attn_fwd_paged, qd.expand(-1, -1, 5, -1).contiguous())):
            (a, la), (b, lb) = call(x, kp, vp, table, L=N), call(x, kp, big, table, L=N)
            ab.alibi_check_error()
            assert torch.equal(la, lb) and bool(torch.isfinite(b).all())
            # bf16 and fp32 numbers this far from their ends scale exactly, but for the smallest elements of `out`
            want = torch.ldexp(a.float(), torch.tensor(power, device="cuda"))
            assert torch.allclose(b.float(), want, rtol=2.0 ** -8, atol=2.0 ** (power - 20)), (power, N)


def test_two_graphs_of_prefills_in_parts_at_once(ab):
    # captured prefills whose items are cut into parts, replayed at the same time, each in its own scratch
    import torch
    jobs = []
    for s in range(2):
        q, k, v = decode.case(30 + s, 1, 2, 2, 40, 9000 + 77 * s, 64)
        n = k.shape[2]
        args = (decode.bf16(q)[1], *ref.paged(k, v, [n], 64, seed=s))
        want = ab.alibi_attn_fwd_paged(*args, lens=ints([n]))
        torch.cuda.synchronize()
        g, stream, lens = torch.cuda.CUDAGraph(), torch.cuda.Stream(), ints([n])
        with torch.cuda.graph(g, stream=stream):
            got = ab.alibi_attn_fwd_paged(*args, lens=lens)
        jobs.append((g, stream, got, want, args, lens))
    for _ in range(20):
        for g, stream, *_ in jobs:
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    ab.alibi_check_error()
    for _, _, got, want, _, _ in jobs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
