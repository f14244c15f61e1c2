"""The 64-bit exponential that decides between near ties of routing, against a longer type's (80 bits or 128 on the host):
off by at most 2 units in the last place (of subnormal results 2 steps of 2^-1074), over its whole range, at the
boundaries of its reduction, and at infinities and NaN."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from dense_block_scaled_gb300 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def exp64(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("exp64") / "libexp64.so")
    r = subprocess.run([build._nvcc(), *build.ARCH, "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", build.CSRC,
                        os.path.join(HERE, "cuda", "exp64_values.cu"), "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    fn = ctypes.CDLL(lib).exp64_values
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_void_p]

    def values(x):
        x = torch.as_tensor(np.ascontiguousarray(x, dtype=np.float64)).cuda()
        y = torch.full_like(x, 7.0)
        assert fn(x.data_ptr(), y.data_ptr(), x.numel(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        return y.cpu().numpy()
    return values


def units(got, x):
    """How far off, in units of the exact value's last place."""
    with np.errstate(over="ignore", under="ignore"):
        exact = np.exp(x.astype(np.longdouble))
    step = np.spacing(np.minimum(exact, np.finfo(np.float64).max).astype(np.float64)).astype(np.longdouble)
    return np.abs((got.astype(np.longdouble) - exact) / step).astype(np.float64)


@pytest.mark.parametrize("lo,hi", [(-745.0, -708.0), (-708.0, -40.0), (-40.0, -1.0), (-1.0, 1.0), (1.0, 40.0), (40.0, 709.7)])
def test_over_the_range(exp64, lo, hi):
    rng = np.random.default_rng(3)
    x = np.concatenate([np.linspace(lo, hi, 100_000), rng.uniform(lo, hi, 200_000)])
    off = units(exp64(x), x)
    print(f"exp64 on [{lo}, {hi}]: off by {off.max():.3f} units at most")
    assert off.max() <= 2


def test_boundaries_of_the_reduction(exp64):
    # arguments around (n + 1/2) log 2, where r is largest, and n log 2, where it is smallest
    n = np.arange(-1074, 1024)
    x = np.concatenate([(n + h) * np.log(2.0) * (1 + d * 2.0 ** -52) for h in (0.0, 0.5) for d in (-2, -1, 0, 1, 2)])
    x = x[(x > -745) & (x < 709.7)]
    assert units(exp64(x), x).max() <= 2


def test_small_arguments(exp64):
    x = np.concatenate([s * 2.0 ** np.arange(-1074.0, 1.0) for s in (-1.0, 1.0)])
    assert units(exp64(x), x).max() <= 2 and (exp64(np.array([0.0, -0.0])) == 1).all()


def test_ends_infinities_and_nan(exp64):
    x = np.array([np.inf, -np.inf, np.nan, -np.nan, 710.0, 800.0, 801.0, 1e300, -746.0, -800.0, -801.0, -1e300])
    y = exp64(x)
    assert np.isnan(y[2:4]).all() and not np.isnan(np.delete(y, [2, 3])).any()
    assert (y[[0, 4, 5, 6, 7]] == np.inf).all() and (y[[1, 8, 9, 10, 11]] == 0).all()


def test_exponentials_rise(exp64):
    # neighbours in order: what is smaller does not come out larger by more than the two errors
    x = np.sort(np.random.default_rng(5).uniform(-60, 0, 400_000))
    y = exp64(x)
    assert (np.diff(y) >= -4 * np.spacing(y[1:])).all()
