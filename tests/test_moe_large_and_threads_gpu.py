"""The mixture-of-experts operators past 2^31 elements (the last rows against their formulas), and from several host
threads at once, each on its own stream or all on the default one."""
import threading

import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_checkpoints_gpu import h_of, normal, rule, values

pytestmark = pytest.mark.gpu
BF16, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK
    torch.cuda.empty_cache()


def test_activation_past_32_bits():
    rows, inner = 132_000, 8192                     # 2.16 billion elements of [g | u]
    X = torch.zeros(rows, 2 * inner, device="cuda", dtype=BF16)
    X[-3:] = normal(3, 2 * inner)
    H = torch.empty(rows, inner, device="cuda", dtype=BF16)
    Q, sf = torch.empty(rows, 2 * inner, device="cuda", dtype=U8), torch.empty(rows, inner // 16, device="cuda", dtype=U8)
    tkg.swiglu(X, H, Q, sf)
    ref = h_of(X[-3:].to(F64))
    assert ((H[-3:].to(F64) - ref).abs() <= (2.0 ** -8 + 2.0 ** -18) * ref.abs()).all() and (H[:-3:1000] == 0).all()
    q, s = rule(X[-3:])
    assert torch.equal(Q[-3:], q) and torch.equal(sf[-3:], s)
    Q.zero_()
    tkg.checkpoint_mxfp8(X, Q, sf)
    assert torch.equal(Q[-3:], q) and torch.equal(sf[-3:], s)
    dH, dX = H, X
    dH[-3:] = normal(3, inner, seed=1)
    d = dH[-3:].to(F64)
    tkg.swiglu_grad(Q, sf, dH, dX)
    x = values(Q[-3:], sf[-3:]).requires_grad_(True)
    (h_of(x) * d).sum().backward()
    assert float((dX[-3:].to(F64) - x.grad).norm()) <= 2.0 ** -8 * float(x.grad.norm())


def test_weight_gradient_past_32_bits():
    cap, k, n = 270_000, 8192, 64                   # 2.2 billion elements of unpacked rows
    tokens, topk = 67_500, 4
    Q, sf = torch.zeros(tokens, k, device="cuda", dtype=U8), torch.full((tokens, k // 32), 127, device="cuda", dtype=U8)
    Q[-1] = 0x38                                    # 1.0
    slots = torch.arange(cap, device="cuda", dtype=I32)
    dD = torch.ones(cap, n, device="cuda", dtype=BF16)
    sizes = torch.tensor([100, cap - 100], device="cuda", dtype=I32)
    dB = torch.empty(2, n, k, device="cuda")
    tkg.gemm_grouped_dev_mxfp8_wgrad(sizes, dD, Q, sf, dB, slots=slots, topk=topk)
    assert (dB[0] == 0).all() and (dB[1] == topk).all()


@pytest.mark.parametrize("own_streams", [True, False])
def test_several_threads(own_streams):
    def work(seed, out):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        tokens, experts, k, hidden = 100 + 333 * seed, 64, 4, 256
        z = torch.randn(tokens, experts, generator=g, device="cuda").to(BF16)
        X = torch.randn(tokens, hidden, generator=g, device="cuda").to(BF16)
        bias = torch.randn(experts, generator=g, device="cuda") * 0.1
        for _ in range(15):
            e = lambda *s, dtype=I32: torch.full(s, 3, dtype=dtype, device="cuda")
            ids, w, sizes, rows, slots = e(tokens, k), e(tokens, k, dtype=F32), e(experts), e(tokens, k), e(tokens * k)
            tkg.moe_route(z, ids, w, sizes, rows, slots, bias=bias, scores="sigmoid")
            Xs, Y = e(tokens * k, hidden, dtype=BF16), e(tokens, hidden, dtype=BF16)
            tkg.moe_dispatch(X, rows, Xs)
            tkg.moe_combine(Xs, rows, Y, weights=w)
            dB = e(experts, 64, hidden, dtype=F32)
            Q, sf = e(tokens, hidden, dtype=U8), e(tokens, hidden // 32, dtype=U8)
            tkg.checkpoint_mxfp8(X, Q, sf)
            tkg.gemm_grouped_dev_mxfp8_wgrad(sizes, Xs[:, :64].contiguous(), Q, sf, dB, slots=slots, topk=k)
            out.append([x.clone() for x in (ids, w, sizes, rows, slots, Y, dB)])
        torch.cuda.current_stream().synchronize()

    alone = []
    for seed in range(4):
        out = []
        work(seed, out)
        alone.append(out)
    torch.cuda.synchronize()
    together, failed = [[] for _ in range(4)], []

    def thread(seed):
        try:
            if own_streams:
                with torch.cuda.stream(torch.cuda.Stream()):
                    work(seed, together[seed])
            else:
                work(seed, together[seed])
        except Exception as e:  # noqa: BLE001 - reported below
            failed.append(e)

    threads = [threading.Thread(target=thread, args=(s,)) for s in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for a, b in zip(alone, together):
        for x, y in zip(a, b):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
