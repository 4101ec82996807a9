"""Sequences of a prefill over pages that have no new tokens (alibi.h: not looked at): whatever their lengths and page numbers say,
nothing is reported and their outputs stay, in every way that the work is cut."""
import pytest

import oracle
import paged_ref as ref
from paged_ref import bf16, ints
from test_gpu_fwd_paged import check
from test_gpu_paged import case

pytestmark = pytest.mark.gpu


# (KV heads, heads of each, new tokens, length, bound): whole items, parts of items, heads of a group together, together in parts
@pytest.mark.parametrize("Hkv,G,T,N,L", [(2, 1, 300, 300, 300), (2, 2, 260, 1500, 9000), (8, 4, 20, 400, 400), (2, 8, 16, 900, 20000)])
@pytest.mark.parametrize("idle", [-1, -2 ** 31, 2 ** 31 - 1, "one past", 0])
def test_idle_sequences_are_not_looked_at(Hkv, G, T, N, L, idle):
    import torch
    import alibi_positional_bias_gb300 as ab
    ab.alibi_check_error()
    B, S = 4, 16
    q, k, v = case(N + T, B, Hkv, G, T, N, 64)
    kp, vp, table = ref.paged(k, v, [N] * B, S, M=-(-L // S))
    table[1::2] = -1
    lens, counts = [N, L + 1 if idle == "one past" else idle] * 2, [T, 0] * 2
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:3], 7.0, device="cuda")
    ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, lens=ints(lens), count=ints(counts), L=L, out=out, lse=lse)
    ab.alibi_check_error()
    assert bool((out[1::2] == 7.0).all()) and bool((lse[1::2] == 7.0).all())
    check(out[::2], lse[::2], q[::2], k[::2], v[::2], [N] * 2, [T] * 2, oracle.slopes(Hkv * G))
    # one that has new tokens is reported beside them
    lens[2], counts[2] = -1, 1
    ab.alibi_attn_fwd_paged(bf16(q)[1], kp, vp, table, lens=ints(lens), count=ints(counts), L=L, out=out, lse=lse)
    with pytest.raises(ab.AlibiError) as e:
        ab.alibi_check_error()
    assert e.value.status == ab.ALIBI_ERR_RANGE
    assert bool(out[2, :, :1].isnan().all()) and bool(lse[2, :, :1].isnan().all()) and bool((out[1::2] == 7.0).all())
