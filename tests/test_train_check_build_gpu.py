"""The training-side suites on the check build (libtkg_check.so): every kernel verifies its ring slots, tiles,
accumulators, widths and TMA coordinates, and each case asserts a clean device status."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def test_training_suites_pass_on_the_check_build():
    from dense_block_scaled_gb300 import build
    lib = build.build(check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_linear_ce_gpu.py", "tests/test_grouped_grad_gpu.py", "-k",
                        "matches or match or widths or pieces or capacity or many_groups or accumulation"],
                       cwd=ROOT, env=dict(os.environ, TKG_LIBRARY=lib), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
