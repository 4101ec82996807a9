"""Kernels that are launched as programmatic dependents begin while the kernel before them, which may write what they
read, still runs. The read-only load path (__ldg, ld.global.nc, and what the compiler may turn loads through const
__restrict__ pointers into) is defined only for data that nothing writes during the kernel's whole life, however late
in it the load stands, so their sources do not use it. No GPU involved."""
import os
import re

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "alibi_positional_bias_gb300", "csrc")


def code(name: str) -> str:
    """The source without comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def dependents() -> list:
    """Sources with a kernel that waits for the one before it."""
    return [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and "griddep_wait()" in code(n)]


def test_the_sources_are_found():
    assert {"alibi_kv4.cu", "alibi_decode_kv4.cu", "alibi_bwd_tc.cu"} <= set(dependents())


@pytest.mark.parametrize("name", dependents())
def test_no_read_only_loads(name):
    # the kernels that wait take their parameters as one struct; a kernel with __restrict__ pointers must not wait
    text = code(name)
    assert "__ldg" not in text and "ld.global.nc" not in text
    for body in re.split(r"__global__", text)[1:]:
        head, _, rest = body.partition("{")
        if "__restrict__" in head:
            assert "griddep_wait()" not in rest.split("__global__")[0].split("\n}\n")[0], head
