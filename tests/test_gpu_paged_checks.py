"""The paged cache's calls under the debug-checks build (-DALIBI_CHECKS): every box's coordinates and destination are tested
before its copy, and every call of the selection comes back with a clean status word and the results of the plain forms."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)

SWEEPS = [
    "test_gpu_paged.py::test_every_length_of_a_few_pages",
    "test_gpu_paged.py::test_shapes",
    "test_gpu_paged.py::test_layouts",
    "test_gpu_paged.py::test_ways_of_dealing",
    "test_gpu_paged.py::test_offsets_beyond_32_bits",
    "test_gpu_paged.py::test_append",
    "test_gpu_fwd_paged.py::test_first_prompts",
    "test_gpu_fwd_paged.py::test_chunks_that_begin_anywhere",
    "test_gpu_fwd_paged.py::test_shapes",
    "test_gpu_fwd_paged.py::test_shared_items",
    "test_gpu_fwd_paged.py::test_infinite_and_nan_rows_that_a_query_does_not_see",
    "test_gpu_fwd_paged_together.py::test_shapes",
    "test_gpu_fwd_paged_together.py::test_infinite_and_nan_rows",
]


def test_checks_build_passes_the_paged_sweeps():
    from alibi_positional_bias_gb300 import _build
    _build.build(checks=True)
    env = dict(os.environ, ALIBI_CHECKS="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        *[os.path.join(HERE, s) for s in SWEEPS]],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    summary = [ln for ln in r.stdout.splitlines() if " passed" in ln][-1]
    assert int(summary.split(" passed")[0].split()[-1]) >= 200, summary  # every case of the selection ran
