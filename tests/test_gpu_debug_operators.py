"""The debug build (AWQ_B200_DEBUG=1: every guarded access checks its range
first) under the tests of the operators between the linear layers: the cache
calls must report AWQ_OK, and all outputs match as they do in the normal
build. Ragged batches, groups split between CTAs and taken whole, both row tiles
and ring depths, long parts, ranges of blocks per CTA, the norm's and the SiLU's
copy-ahead rows. No case provokes an out-of-range access."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ENV = {**os.environ, "AWQ_B200_DEBUG": "1"}


def test_the_debug_build_is_the_one_that_runs():
    r = subprocess.run([sys.executable, "-c", "import weight_only_bit_awq_b200 as a; print(a.LIB_PATH)"], cwd=ROOT, env=ENV,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("libawq_b200_debug.so"), r.stdout + r.stderr


@pytest.mark.parametrize("file,which", [
    ("test_gpu_norm_act.py", "test_rmsnorm or silu or walks_rows"),
    ("test_gpu_kv8.py", "bit_exact or several_tokens or is_split or short_sequences or sharing_out or drafts or bad_contents or pieces"),
    ("test_gpu_kv8_long.py", "sixteen or unit_counts"),
])
def test_operators_in_the_debug_build(file, which):
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", os.path.join("tests", file),
                        "-k", which], cwd=ROOT, env=ENV, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-3000:]
