"""The feed-forward suites under the debug library, whose kernels check every
load's coordinates, TMEM columns and stored rows (as test_gpu_debug_checks does
for the GEMMs')."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITES = ["tests/test_gpu_gated_gemm.py", "tests/test_gpu_gated_few_tokens.py", "tests/test_gpu_not_finite.py",
          "tests/test_gpu_gated_backward.py", "tests/test_gpu_checkpoint.py", "tests/test_gpu_block.py"]


def test_the_feed_forward_suites_pass_every_device_check():
    if os.environ.get("DG_DEBUG_LIBRARY", "0") not in ("", "0"):
        pytest.skip("already running under the debug library")
    from moe_grouped_gemm_fp8_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, DG_DEBUG_LIBRARY="1")
    r = subprocess.run([sys.executable, "-m", "pytest", *SUITES, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"],
                       env=env, cwd=ROOT, timeout=1800, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-6000:] + r.stderr[-3000:]
