"""The forms of the training-side kernel that only long sums and few tokens reach (sums in parts, two blocks to an SM),
and the suites of values and long sums, on the check build (libtkg_check.so), with every invariant verified."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("files,which", [
    (["tests/test_linear_ce_gpu.py"], "long_sums or few_tokens or precision or last_bits"),
    (["tests/test_linear_ce_values_gpu.py", "tests/test_long_sums_gpu.py"], "test"),
])
def test_forms_pass_on_the_check_build(files, which):
    from dense_block_scaled_gb300 import build
    lib = build.build(check=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *files, "-k",
                        which], cwd=ROOT, env=dict(os.environ, TKG_LIBRARY=lib), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
