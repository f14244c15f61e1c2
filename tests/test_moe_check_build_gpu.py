"""Routing on the check build (libtkg_check.so): candidates, choices and rows are verified to be inside, and each case
asserts a clean device status.  Among them are the cases whose candidates once stood past the last expert."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("files,which", [
    (["tests/test_moe_masked_biases_gpu.py"], "1- or 300- or groups or many"),
    (["tests/test_moe_route_gpu.py"], "33-bf16 or 513-bf16 or 1000-f32 or rules or many_tokens or ties or decide or biases or masked or nan"),
    (["tests/test_moe_random_gpu.py", "tests/test_moe_block_gpu.py"], "test"),
])
def test_routing_passes_on_the_check_build(files, which):
    from dense_block_scaled_gb300 import build
    lib = build.build(check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *files, "-k",
                        which], cwd=ROOT, env=dict(os.environ, TKG_LIBRARY=lib), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout, r.stdout[-500:]
