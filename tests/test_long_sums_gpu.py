"""FP32 weight gradients of many rows keep their precision: sums of products of one sign, whose error in one accumulator
would grow with their length.

An accumulator takes at most 2048 products, 128 steps of 16, at each of which it loses less than 2^-23 of itself; it is
half of its sum on average, so less than 2^-17 in all.  Adding up to 16 such sums, the scale and the addition to what
is there take at most 2^-24 each: together less than 2^-19."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64
BOUND = 2.0 ** -17 + 2.0 ** -19


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK
    tkg.set_option(tkg.OPT_BF16_TILE_N, 0)


def positive(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda").add_(0.5).to(BF16)


@pytest.mark.parametrize("tile_n", [0, 512])
@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("sizes,n,k", [([16384], 136, 264), ([30000], 512, 72), ([9000, 0, 2048, 2049, 64, 3001], 264, 520),
                                       ([1, 4097, 700], 8, 1000)])
def test_experts_of_many_rows(sizes, n, k, add, tile_n):
    tkg.set_option(tkg.OPT_BF16_TILE_N, tile_n)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(sum(sizes) + n)
    rows = sum(sizes)
    dD, A = positive(gen, rows + 5, n), positive(gen, rows + 5, k)
    dD[rows:], A[rows:] = float("nan"), float("nan")
    start = torch.rand(len(sizes), n, k, generator=gen, device="cuda") if add else None
    dB = start.clone() if add else torch.full((len(sizes), n, k), 7.0, device="cuda")
    dev = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    tkg.gemm_grouped_dev_bf16_wgrad(dev, dD, A, dB, alpha=0.75, accumulate=add)
    row = 0
    for g, m in enumerate(sizes):
        ref = 0.75 * (dD[row:row + m].to(F64).T @ A[row:row + m].to(F64))
        if add:
            ref += start[g].to(F64)
        assert ((dB[g].to(F64) - ref).abs() <= BOUND * ref).all(), (g, float(((dB[g].to(F64) - ref) / ref).abs().max()))
        row += m


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("tokens,hidden", [(2048, 72), (2056, 264), (16384, 136), (10000, 520)])
def test_head_of_many_tokens(tokens, hidden, add):
    # Equal logits over 256 entries: exp(z - lse) is 2^-8, every g and weight a BF16 number, all rounding in the sums
    gen = torch.Generator(device="cuda")
    gen.manual_seed(tokens)
    X, W = positive(gen, tokens, hidden), torch.zeros(256, hidden, device="cuda", dtype=BF16)
    y = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    lse = torch.full((tokens,), 8 * 0.6931471805599453, device="cuda")
    dloss = torch.full((tokens,), 2.0 ** -14, device="cuda")
    dW = torch.ones(256, hidden, device="cuda")
    tkg.linear_ce_grad(X, W, y, lse, dloss, None, dW, accumulate=add)
    ref = 2.0 ** -22 * X.to(F64).sum(dim=0)[None, :].expand(256, hidden).clone()
    ref[0] *= -255
    if add:   # (the first row may cancel: its bound is that of its terms)
        bound = BOUND * ref.abs() + 2.0 ** -24 * (1 + ref.abs())
        ref += 1
    else:
        bound = BOUND * ref.abs()
    assert ((dW.to(F64) - ref).abs() <= bound).all(), float(((dW.to(F64) - ref).abs() / bound).max())
