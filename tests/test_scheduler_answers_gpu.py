"""Every role of a GEMM kernel agrees on the tiles it takes over from the scheduler (cluster launch control): many
launches back to back, bit for bit the same result, and none that runs into the wait limit."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg
from helpers import Operands, assert_within_tolerance, bf16_to_f64, run_gemm

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _short_waits():
    tkg.set_option(tkg.OPT_TIMEOUT_MS, 200)
    yield
    for o in (tkg.OPT_TIMEOUT_MS, tkg.OPT_CTA_GROUP):
        tkg.set_option(o, 0)


@pytest.mark.parametrize("cta_group", [1, 2])
@pytest.mark.parametrize("fmt", ["bf16", "mxfp8", "nvfp4"])
def test_no_tile_is_missed_by_a_dense_product(fmt, cta_group):
    # about ten tiles to each pair of SMs, of few stages each: many answers in a short launch
    m, n, k = 5000, 9608, 256
    tkg.set_option(tkg.OPT_CTA_GROUP, cta_group)
    ops = Operands(fmt, m, n, k, 71)
    dev = ops.upload()
    first = run_gemm(fmt, dev, m, n, k, 1.0)
    for _ in range(500):
        D = run_gemm(fmt, dev, m, n, k, 1.0)
    assert tkg.device_status() == tkg.OK
    assert torch.equal(D.view(torch.int16), first.view(torch.int16))
    ref, S = ops.reference(rows=(m - 128, 128))
    assert_within_tolerance(bf16_to_f64(D[m - 128:]), ref, S, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_no_tile_is_missed_by_a_list(fmt):
    entries = []
    for i in range(8):
        m, n, k = 700 + 131 * i, 4096 + 8 * i, 256
        ops = Operands(fmt, m, n, k, 80 + i)
        dev = ops.upload()
        D = torch.full((m, n), 3.0, dtype=torch.bfloat16, device="cuda")
        A, B, sfa, sfb, ta, tb = dev
        entries.append((ops, dev, D, tkg.gemm_desc(fmt, A, B, D, 1.0, sfa=sfa, sfb=sfb, ta=ta, tb=tb)))
    descs = [e[3] for e in entries]
    tkg.gemm_list(fmt, descs)
    first = [e[2].clone() for e in entries]
    for _ in range(500):
        tkg.gemm_list(fmt, descs)
    assert tkg.device_status() == tkg.OK
    for e, want in zip(entries, first):
        assert torch.equal(e[2].view(torch.int16), want.view(torch.int16))
    ops, _, D, _ = entries[-1]
    ref, S = ops.reference(rows=(0, 64))
    assert_within_tolerance(bf16_to_f64(D[:64]), ref, S, fmt)
