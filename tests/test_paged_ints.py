"""Positions, counts and lengths of the paged calls that are no tensors: refused by name, as every other argument."""
import numpy as np
import pytest
import torch

import alibi_positional_bias_gb300 as ab
from test_paged_binding import fake, on  # noqa: F401


@pytest.mark.parametrize("value", [[0, 1], 5, np.zeros(2, np.int32)])
def test_no_tensors(fake, value):  # noqa: F811
    k, kp, table = on(2, 2, 3, 64), on(4, 2, 16, 64), on(2, 4, dtype=torch.int32)
    q = on(2, 4, 1, 64)
    given = dict(out=q, lse=on(2, 4, 1, dtype=torch.float32))
    for name, call in [("pos", lambda: ab.alibi_paged_append(k, k, kp, kp, table, pos=value)),
                       ("count", lambda: ab.alibi_paged_append(k, k, kp, kp, table, count=value)),
                       ("lens", lambda: ab.alibi_attn_decode_paged(q, kp, kp, table, lens=value, **given)),
                       ("lens", lambda: ab.alibi_attn_fwd_paged(q, kp, kp, table, lens=value, **given)),
                       ("count", lambda: ab.alibi_attn_fwd_paged(q, kp, kp, table, count=value, **given))]:
        with pytest.raises(TypeError, match=name):
            call()
    assert not fake.calls
