"""The 4-bit cache's calls under the debug-checks build (-DALIBI_CHECKS): the bulk copies' addresses and sizes are
tested before every copy, and every call of the selection comes back with a clean status word and the results of
the plain forms."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

SWEEPS = [
    "test_gpu_kv4.py::test_write_and_read",
    "test_gpu_kv4.py::test_offsets_beyond_32_bits",
    "test_gpu_decode_kv4.py::test_every_length_of_a_few_blocks",
    "test_gpu_decode_kv4.py::test_shapes",
    "test_gpu_decode_kv4.py::test_ways_of_dealing",
    "test_gpu_decode_kv4.py::test_offsets_beyond_32_bits",
]


def test_checks_build_passes_the_cache_sweeps():
    from alibi_positional_bias_gb300 import _build
    _build.build(checks=True)
    env = dict(os.environ, ALIBI_CHECKS="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        *[os.path.join(HERE, s) for s in SWEEPS]],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    summary = [ln for ln in r.stdout.splitlines() if " passed" in ln][-1]
    assert int(summary.split(" passed")[0].split()[-1]) >= 99, summary  # every case of the selection ran
