"""Sizes at the end of 32 bits are refused on the host by the training-side calls: they would leave 32 bits where tiles
are rounded up, or on the way into the library (no GPU needed; nothing of that size exists here)."""
import ctypes

import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_train_ops_abi import grad, loss

BF16 = torch.bfloat16
P = ctypes.c_void_p(4096)
FAR = [2 ** 31 - 2 ** 16 + 8, 2 ** 31 - 8]


@pytest.fixture(scope="module")
def lib():
    from dense_block_scaled_gb300 import build
    build.build()
    return tkg.load()


@pytest.mark.parametrize("far", FAR)
def test_sizes_near_the_end_of_32_bits(lib, far):
    for call in (loss, grad):
        for at in ("tokens", "vocab", "hidden"):
            assert call(lib, **{at: far}) == tkg.ERR_UNSUPPORTED, at
    assert lib.tkg_linear_ce_loss_workspace_bytes(far, 100) == lib.tkg_linear_ce_loss_workspace_bytes(3, far) == 0
    assert lib.tkg_linear_ce_grad_workspace_bytes(far, 100, 64, 0) == 0
    assert lib.tkg_linear_ce_grad_workspace_bytes(8, far, 64, 0) == lib.tkg_linear_ce_grad_workspace_bytes(8, 100, far, 0) == 0
    for sizes in ((far, 64, 64), (8, far, 64), (8, 64, far)):
        assert lib.tkg_gemm_grouped_dev_bf16_dgrad(2, P, *sizes, P, P, P, 1.0, None) == tkg.ERR_UNSUPPORTED
        assert lib.tkg_gemm_grouped_dev_bf16_wgrad(2, P, *sizes, P, P, P, 0, 1.0, None) == tkg.ERR_UNSUPPORTED


def meta(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("at", ["tokens", "vocab", "hidden"])
def test_sizes_past_32_bits(at):
    s = dict(tokens=8, vocab=100, hidden=64)
    s[at] = 2 ** 32 + 8
    t, v, h = s.values()
    X, W, y, f = meta(t, h), meta(v, h), meta(t, dtype=torch.int64), meta(t, dtype=torch.float32)
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg.linear_ce_loss(X, W, y, f, f)
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg.linear_ce_grad(X, W, y, f, f, X, W)


@pytest.mark.parametrize("at", [0, 1, 2])
def test_sizes_past_32_bits_of_groups(at):
    s = [8, 64, 64]
    s[at] = 2 ** 32 + 8
    cap, n, k = s
    sizes = meta(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg.gemm_grouped_dev_bf16_dgrad(sizes, meta(cap, n), meta(2, n, k), meta(cap, k))
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg.gemm_grouped_dev_bf16_wgrad(sizes, meta(cap, n), meta(cap, k), meta(2, n, k))


def test_row_pitches_past_32_bits():
    far = torch.empty_strided((8, 64), (2 ** 32 + 64, 1), dtype=BF16, device="meta")
    W, y, f = meta(100, 64), meta(8, dtype=torch.int64), meta(8, dtype=torch.float32)
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg.linear_ce_loss(far, W, y, f, f)
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg.linear_ce_grad(meta(8, 64), W, y, f, f, far, None)
