"""The training-side operators beside the library's plain product, and from two host threads on the default stream."""
import threading

import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_linear_ce_gpu import BF16, F32, F64, Head, run_grad, run_loss

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK


@pytest.mark.parametrize("rows,n,k", [(777, 512, 768), (1, 264, 72), (3001, 136, 520)])
def test_one_group_beside_the_plain_product(rows, n, k):
    """Both are within the library's bound for its products of the definition, 2^-7 |ref| + 1e-5 sum |a b|."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF16)
    dD, A, B = r(rows, n), r(rows, k), r(1, n, k)
    dev = torch.tensor([rows], dtype=torch.int32, device="cuda")
    dA, dB = torch.empty(rows, k, device="cuda", dtype=BF16), torch.empty(1, n, k, device="cuda", dtype=BF16)
    tkg.gemm_grouped_dev_bf16_dgrad(dev, dD, B, dA)
    tkg.gemm_grouped_dev_bf16_wgrad(dev, dD, A, dB)
    up = -rows % 8   # the plain product's contraction is a multiple of 8
    zeros = lambda t: torch.cat([t, torch.zeros(up, t.shape[1], device="cuda", dtype=BF16)]).T.contiguous()
    pA, pB = torch.empty_like(dA), torch.empty_like(dB[0])
    tkg.gemm_bf16(dD, B[0].T.contiguous(), pA, 1.0)
    tkg.gemm_bf16(zeros(dD), zeros(A), pB, 1.0)
    for got, plain, x, y in ((dA, pA, dD.to(F64), B[0].to(F64)), (dB[0], pB, dD.to(F64).T, A.to(F64))):
        ref, bound = x @ y, 2.0 ** -7 * (x @ y).abs() + 1e-5 * (x.abs() @ y.abs())
        assert ((got.to(F64) - ref).abs() <= bound).all() and ((plain.to(F64) - ref).abs() <= bound).all()
        # both round a sum that is within the bound's second part of the other's
        assert ((got.to(F64) - plain.to(F64)).abs() <= 2.0 ** -7 * ref.abs() + 2e-5 * (x.abs() @ y.abs())).all()


def test_two_threads_on_the_default_stream():
    # each thread keeps workspaces of its own for that stream; larger calls between smaller ones replace them
    heads = [[Head(t, v, h, seed=31 + i) for t, v, h in shapes] for i, shapes in enumerate(
        [[(1, 3000, 264), (200, 2500, 128), (17, 257, 64)], [(90, 4001, 136), (2, 1000, 512), (300, 700, 264)]])]
    want = [[(h, run_loss(h), run_grad(h, h.forward()[2].float())) for h in hs] for hs in heads]
    torch.cuda.synchronize()
    errors = []

    def work(cases):
        try:
            for _ in range(15):
                for h, (loss, lse), (dX, dW) in cases:
                    got = run_loss(h)
                    grads = run_grad(h, h.forward()[2].float())
                    if not (torch.equal(got[0], loss) and torch.equal(got[1], lse) and torch.equal(grads[0], dX)
                            and torch.equal(grads[1], dW)):
                        raise AssertionError(h.shape)
        except Exception as e:   # surfaced in the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(cases,)) for cases in want]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_infinities_in_rows_that_count_reach_the_gradients():
    """Where the definition's sums have terms that are not numbers, so do the results, and nowhere else."""
    for tokens, vocab, hidden in [(40, 700, 264), (3, 300, 64), (300, 900, 4104)]:
        h = Head(tokens, vocab, hidden, ignored=0.0, seed=33)
        clean = run_grad(h, h.forward()[2].float())
        h.X[1, 0] = float("inf")
        z = h.alpha * (h.X.to(F64) @ h.W.to(F64).T)
        lse = torch.logsumexp(z, dim=1)
        g = torch.exp(z - lse[:, None])
        g[torch.arange(tokens, device="cuda"), h.y] -= 1
        g = h.dloss.to(F64)[:, None] * h.alpha * g
        dX, dW = run_grad(h, lse.float(), dtype=F32)
        assert torch.equal(torch.isnan(dX), torch.isnan(g @ h.W.to(F64)))
        assert torch.equal(torch.isnan(dW), torch.isnan(g.T @ h.X.to(F64)))
        rest = torch.arange(tokens, device="cuda") != 1
        assert torch.equal(dX[rest], clean[0][rest])


def test_long_forms_time_out_and_recover():
    # sums in parts (logits, FP32 weight gradients), two blocks to an SM: every role's waits end
    wide, narrow = Head(200, 700, 4104, seed=34), Head(20, 20003, 4096, seed=35)
    lse = {h: h.forward()[2].float() for h in (wide, narrow)}
    dev = torch.tensor([2100, 0, 900], dtype=torch.int32, device="cuda")
    dD, A = (torch.randn(3000, w, device="cuda").to(BF16) for w in (264, 520))
    dB = torch.zeros(3, 264, 520, device="cuda")

    def calls():
        for h in (wide, narrow):
            yield lambda: run_loss(h)
            yield lambda: run_grad(h, lse[h])
        yield lambda: tkg.gemm_grouped_dev_bf16_wgrad(dev, dD, A, dB, accumulate=True)

    want = [f() for f in calls()]
    dB.zero_()
    try:
        tkg.set_option(tkg.OPT_TIMEOUT_MS, 100)
        tkg.set_option(tkg.OPT_INJECT_STALL, 1)
        for f in calls():
            f()
            assert tkg.device_status() == tkg.ERR_TIMEOUT
    finally:
        tkg.set_option(tkg.OPT_INJECT_STALL, 0)
        tkg.set_option(tkg.OPT_TIMEOUT_MS, 0)
    for f, w in zip(calls(), want):
        got = f()
        assert w is None or all(torch.equal(a, b) for a, b in zip(got, w))
