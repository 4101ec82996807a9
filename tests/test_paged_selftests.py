"""What the self-tests of the paged kernels' failure paths refuse, without a GPU."""
import pytest

import alibi_positional_bias_gb300 as ab
from test_paged_binding import P, lib, pages  # noqa: F401

INVALID = ab.ALIBI_ERR_INVALID


@pytest.mark.parametrize("change", [dict(barrier=-1), dict(barrier=9), dict(wait_us=0), dict(wait_us=999), dict(wait_us=1000001),
                                    dict(q=None), dict(T=0), dict(L=65)])
def test_prefills_that_are_refused(lib, change):  # noqa: F811
    x = dict(q=P, lens=P, count=P, out=P, lse=P, B=1, H=2, T=1, L=64, barrier=0, wait_us=20000)
    x.update(change)
    assert lib.alibi_selftest_fwd_paged_timeout(x["q"], pages(), x["lens"], x["count"], x["out"], x["lse"], x["B"], x["H"], x["T"],
                                                x["L"], x["barrier"], x["wait_us"], None) == INVALID


@pytest.mark.parametrize("change", [dict(wait_us=0), dict(wait_us=999), dict(wait_us=1000001), dict(q=None), dict(T=0), dict(L=65)])
def test_decodes_that_are_refused(lib, change):  # noqa: F811
    x = dict(q=P, lens=P, out=P, lse=P, B=1, H=2, T=1, L=64, wait_us=20000)
    x.update(change)
    assert lib.alibi_selftest_decode_paged_timeout(x["q"], pages(), x["lens"], x["out"], x["lse"], x["B"], x["H"], x["T"], x["L"],
                                                   x["wait_us"], None) == INVALID
