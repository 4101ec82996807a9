"""A first call from a host thread that has made no other: the tensor maps are encoded with a current context."""
import threading

import numpy as np
import pytest

import paged_ref as ref
from paged_ref import bf16, ints

pytestmark = pytest.mark.gpu


def in_thread(f):
    got = []

    def work():
        try:
            got.append(f())
        except Exception as e:  # noqa: BLE001
            got.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not isinstance(got[0], Exception), got[0]
    return got[0]


@pytest.mark.parametrize("call", ["fwd", "bwd", "decode_paged", "fwd_paged", "append"])
def test_first_call_of_a_thread(call):
    import torch
    import alibi_positional_bias_gb300 as ab
    rng = np.random.default_rng(0)
    N, d = 150, 64
    (k64, k), (v64, v), (_, q) = (bf16(rng.standard_normal((1, 2, N, d))) for _ in range(3))
    kp, vp, table = ref.paged(k64, v64, [N], 16)
    stream = torch.cuda.Stream()
    out, lse = torch.empty_like(q), torch.empty(1, 2, N, device="cuda")
    one, one_lse = torch.empty_like(q[:, :, :1]), torch.empty(1, 2, 1, device="cuda")
    grads = [torch.empty_like(q) for _ in range(3)]
    dense = ab.alibi_attn_fwd(q, k, v)
    torch.cuda.synchronize()
    f = {
        "fwd": lambda: ab.alibi_attn_fwd(q, k, v, out=out, lse=lse, stream=stream),
        "bwd": lambda: ab.alibi_attn_bwd(q, k, v, *dense, q, *grads, stream=stream),
        "decode_paged": lambda: ab.alibi_attn_decode_paged(q[:, :, -1:].contiguous(), kp, vp, table, lens=ints([N]), out=one, lse=one_lse,
                                                           stream=stream),
        "fwd_paged": lambda: ab.alibi_attn_fwd_paged(q, kp, vp, table, L=N, out=out, lse=lse, stream=stream),
        "append": lambda: ab.alibi_paged_append(k, v, kp, vp, table, stream=stream),
    }[call]
    want = f()
    want = [x.clone() for x in want] if want is not None else []
    torch.cuda.synchronize()
    got = in_thread(f)
    torch.cuda.synchronize()
    ab.alibi_check_error()
    for a, b in zip(got or [], want):
        assert torch.equal(a, b)
