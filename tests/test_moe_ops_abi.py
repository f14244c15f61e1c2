"""Host-side checks of the mixture-of-experts entry points: what is refused, and what is nothing to do, before any CUDA
call (no GPU needed).  The pointers are never dereferenced."""
import ctypes

import pytest
import torch

from dense_block_scaled_gb300 import tkg

P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4097)
BIG = 1 << 40
FAR = [2 ** 31 - 2 ** 16 + 8, 2 ** 31 - 8]
OK, INVALID, ALIGNMENT, UNSUPPORTED = tkg.OK, tkg.ERR_INVALID_ARG, tkg.ERR_ALIGNMENT, tkg.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from dense_block_scaled_gb300 import build
    build.build()
    return tkg.load()


def rule(scores=0, groups=1, stay=1, renormalise=1, scale=1.0):
    return ctypes.byref(tkg.RouteRule(scores, groups, stay, renormalise, scale))


def route(lib, tokens=8, experts=64, topk=4, logits=P, kind=0, ld=None, r=None, bias=P, keep=P, ids=P, weights=P, sizes=P,
          rows=P, slots=P, ws=P, nbytes=BIG):
    return lib.tkg_moe_route(tokens, experts, topk, logits, kind, experts if ld is None else ld, rule() if r is None else r,
                             bias, keep, ids, weights, sizes, rows, slots, ws, nbytes, None)


def route_grad(lib, tokens=8, experts=64, topk=4, logits=P, kind=0, ld=None, r=None, ids=P, dw=P, dz=P, lddz=None):
    return lib.tkg_moe_route_grad(tokens, experts, topk, logits, kind, experts if ld is None else ld,
                                  rule() if r is None else r, ids, dw, dz, experts if lddz is None else lddz, None)


def test_route(lib):
    for call in (route, route_grad):
        for bad in (dict(tokens=-1), dict(experts=0), dict(topk=0), dict(topk=65), dict(ld=63), dict(kind=2), dict(kind=-1),
                    dict(r=rule(scores=2)), dict(logits=None), dict(ids=None), dict(r=rule(renormalise=2))):
            assert call(lib, **bad) == INVALID, bad
        for bad in (dict(experts=513), dict(topk=33), dict(tokens=2 ** 30)):
            assert call(lib, **bad) == UNSUPPORTED, bad
        for bad in (dict(logits=ODD), dict(ids=ODD), dict(kind=1, logits=ctypes.c_void_p(4098))):
            assert call(lib, **bad) == ALIGNMENT, bad
    for bad in (dict(r=rule(groups=0)), dict(r=rule(groups=5)), dict(r=rule(groups=4, stay=5)), dict(r=rule(groups=4, stay=0)),
                dict(r=rule(groups=32, stay=1)), dict(weights=None), dict(sizes=None), dict(rows=None), dict(slots=None),
                dict(ws=None), dict(tokens=1000, nbytes=lib.tkg_moe_route_workspace_bytes(1000, 64) - 1)):
        assert route(lib, **bad) == INVALID, bad
    assert route(lib, r=rule(groups=64, stay=64)) == UNSUPPORTED
    for bad in ("bias", "weights", "sizes", "rows", "slots", "ws"):
        assert route(lib, **{bad: ODD}) == ALIGNMENT, bad
    for bad in (dict(dw=None), dict(dz=None), dict(lddz=63)):
        assert route_grad(lib, **bad) == INVALID, bad
    assert route_grad(lib, dw=ODD) == route_grad(lib, dz=ODD) == ALIGNMENT
    assert route_grad(lib, tokens=0, dz=None) == OK
    assert lib.tkg_moe_route(8, 64, 4, P, 0, 64, None, None, None, P, P, P, P, P, P, BIG, None) == INVALID
    assert lib.tkg_moe_route_workspace_bytes(-1, 64) == lib.tkg_moe_route_workspace_bytes(8, 0) == 0
    assert lib.tkg_moe_route_workspace_bytes(8, 513) == lib.tkg_moe_route_workspace_bytes(FAR[0], 8) == 0


def rows_call(lib, which, tokens=8, topk=2, hidden=64, a=P, lda=None, rows=P, cap=16, b=P, ldb=None, weights=P):
    lda, ldb = hidden if lda is None else lda, hidden if ldb is None else ldb
    if which == "dispatch":
        return lib.tkg_moe_dispatch(tokens, topk, hidden, a, lda, rows, cap, b, ldb, None)
    return lib.tkg_moe_combine(tokens, topk, hidden, a, lda, cap, rows, weights, b, ldb, None)


@pytest.mark.parametrize("which", ["dispatch", "combine"])
def test_rows(lib, which):
    for bad in (dict(tokens=-1), dict(topk=0), dict(hidden=-8), dict(cap=-1), dict(lda=56), dict(ldb=56), dict(a=None),
                dict(b=None), dict(rows=None)):
        assert rows_call(lib, which, **bad) == INVALID, bad
    for bad in (dict(topk=33), dict(tokens=2 ** 30 + 2 ** 29), dict(cap=FAR[0]), dict(hidden=FAR[0]), dict(hidden=FAR[1]),
                dict(tokens=2 ** 29, hidden=2 ** 24)):
        assert rows_call(lib, which, **bad) == UNSUPPORTED, bad
    for bad in (dict(hidden=60), dict(lda=68), dict(ldb=68), dict(a=ODD), dict(b=ODD), dict(rows=ODD)):
        assert rows_call(lib, which, **bad) == ALIGNMENT, bad
    assert rows_call(lib, which, tokens=0, a=None, rows=None, b=None) == OK
    assert rows_call(lib, which, hidden=0, lda=1, a=None, rows=None, b=None) == OK
    if which == "combine":
        assert rows_call(lib, which, weights=ODD) == ALIGNMENT
    else:
        assert rows_call(lib, which, cap=0, a=None, b=None) == OK


def test_checkpoint(lib):
    def call(rows=8, k=64, X=P, ldx=None, Q=P, sf=P):
        return lib.tkg_checkpoint_mxfp8(rows, k, X, k if ldx is None else ldx, Q, sf, None)

    for bad in (dict(rows=-1), dict(k=-32), dict(ldx=56), dict(X=None), dict(Q=None), dict(sf=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(k=48), dict(ldx=68), dict(X=ODD), dict(Q=ODD)):
        assert call(**bad) == ALIGNMENT, bad
    for bad in (dict(rows=FAR[0]), dict(k=2 ** 31 - 32)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(rows=0, X=None) == call(k=0, X=None) == OK


def test_activation(lib):
    def call(rows=8, inner=64, GU=P, ldgu=None, H=P, ldh=None, Q=P, sf=P):
        return lib.tkg_swiglu(rows, inner, GU, 2 * inner if ldgu is None else ldgu, H, inner if ldh is None else ldh, Q, sf, None)

    for bad in (dict(rows=-1), dict(inner=-8), dict(ldgu=120), dict(ldh=56), dict(Q=None), dict(sf=None), dict(GU=None),
                dict(H=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(inner=40), dict(inner=36, Q=None, sf=None), dict(ldgu=132), dict(ldh=68), dict(GU=ODD), dict(H=ODD),
                dict(Q=ODD)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(rows=FAR[0]) == call(inner=2 ** 30 - 32) == UNSUPPORTED
    assert call(rows=0, GU=None) == call(inner=0, GU=None, Q=None, sf=None) == OK


def test_activation_gradient(lib):
    def call(rows=8, inner=64, Q=P, sf=P, dH=P, lddh=None, slots=P, choices=8, w=P, dGU=P, lddgu=None, H=P, ldh=None, dw=P):
        d = lambda x, y: y if x is None else x
        return lib.tkg_swiglu_grad(rows, inner, Q, sf, dH, d(lddh, inner), slots, choices, w, dGU, d(lddgu, 2 * inner), H,
                                   d(ldh, inner), dw, None)

    for bad in (dict(rows=-1), dict(inner=-32), dict(choices=-1), dict(lddh=56), dict(lddgu=120), dict(ldh=56), dict(w=None),
                dict(Q=None), dict(sf=None), dict(dH=None), dict(dGU=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(inner=40), dict(lddh=68), dict(lddgu=132), dict(ldh=68), dict(Q=ODD), dict(dH=ODD), dict(dGU=ODD),
                dict(H=ODD), dict(slots=ODD), dict(w=ODD), dict(dw=ODD)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(rows=FAR[0]) == call(choices=FAR[1]) == UNSUPPORTED
    assert call(rows=0, Q=None) == call(inner=0, Q=None, dw=None) == OK


def test_weight_gradient(lib):
    need = lib.tkg_gemm_grouped_dev_mxfp8_wgrad_workspace_bytes(8, 64)

    def call(groups=2, sizes=P, cap=8, n=64, k=64, dD=P, tokens=8, Q=P, sf=P, slots=P, topk=1, dB=P, kind=0, ws=P, nbytes=need):
        return lib.tkg_gemm_grouped_dev_mxfp8_wgrad(groups, sizes, cap, n, k, dD, tokens, Q, sf, slots, topk, dB, kind, 1.0,
                                                    ws, nbytes, None)

    for bad in (dict(groups=0), dict(sizes=None), dict(cap=-1), dict(n=-8), dict(k=-32), dict(tokens=-1), dict(topk=0),
                dict(dD=None), dict(Q=None), dict(sf=None), dict(dB=None), dict(kind=3), dict(ws=None),
                dict(nbytes=need - 1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(groups=129), dict(cap=FAR[0]), dict(n=FAR[1]), dict(k=FAR[0]), dict(tokens=FAR[0])):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(n=60), dict(k=40), dict(sizes=ODD), dict(dD=ODD), dict(Q=ODD), dict(slots=ODD), dict(dB=ODD), dict(ws=ODD)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(n=0, dB=None) == call(k=0, dB=None, ws=None) == call(cap=0, kind=2, ws=None) == OK
    assert lib.tkg_gemm_grouped_dev_mxfp8_wgrad_workspace_bytes(-1, 64) == 0
    assert lib.tkg_gemm_grouped_dev_mxfp8_wgrad_workspace_bytes(FAR[0], 64) == 0


# ---------------------------------------------------------------- the tensors that the Python calls take

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def operands(device):
    e = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device=device)
    return {
        tkg.moe_route: dict(logits=e(8, 64), ids=e(8, 4, dtype=I32), weights=e(8, 4, dtype=F32), sizes=e(64, dtype=I32),
                            rows=e(8, 4, dtype=I32), slots=e(32, dtype=I32), bias=e(64, dtype=F32), keep=e(8, dtype=U8)),
        tkg.moe_route_grad: dict(logits=e(8, 64), ids=e(8, 4, dtype=I32), dweights=e(8, 4, dtype=F32), dlogits=e(8, 64)),
        tkg.moe_dispatch: dict(X=e(8, 64), rows=e(8, 4, dtype=I32), out=e(32, 64)),
        tkg.moe_combine: dict(O=e(32, 64), rows=e(8, 4, dtype=I32), Y=e(8, 64), weights=e(8, 4, dtype=F32)),
        tkg.checkpoint_mxfp8: dict(X=e(8, 64), Q=e(8, 64, dtype=U8), sf=e(8, 2, dtype=U8)),
        tkg.swiglu: dict(GU=e(8, 128), H=e(8, 64), Q=e(8, 128, dtype=U8), sf=e(8, 4, dtype=U8)),
        tkg.swiglu_grad: dict(Q=e(8, 128, dtype=U8), sf=e(8, 4, dtype=U8), dH=e(8, 64), dGU=e(8, 128), H=e(8, 64),
                              slots=e(8, dtype=I32), weights=e(4, 2, dtype=F32), dweights=e(4, 2, dtype=F32)),
        tkg.gemm_grouped_dev_mxfp8_wgrad: dict(sizes_dev=e(2, dtype=I32), dD=e(16, 64), Q=e(8, 96, dtype=U8),
                                               sf=e(8, 3, dtype=U8), dB=e(2, 64, 96), slots=e(16, dtype=I32)),
    }


CALLS = list(operands("cpu"))
NAMES = [(c, n) for c in CALLS for n in operands("cpu")[c]]
ids = lambda x: getattr(x, "__name__", x)  # noqa: E731


@pytest.mark.parametrize("call", CALLS, ids=ids)
def test_host_tensors_are_refused(call):
    with pytest.raises(ValueError, match="on the GPU is wanted"):
        call(**operands("cpu")[call])


@pytest.mark.parametrize("call,name", NAMES, ids=ids)
def test_wrong_types_shapes_and_strides_are_refused(call, name):
    t = operands("cpu")[call][name]
    longer = torch.zeros(*t.shape[:-1], t.shape[-1] + 1, dtype=t.dtype)
    wrong = [t.to(torch.float64), longer]
    if t.dim() == 1:
        wrong.append(torch.zeros(2 * t.shape[0], dtype=t.dtype)[::2])
    else:
        wrong.append(torch.zeros(*t.shape[::-1], dtype=t.dtype).permute(*range(t.dim())[::-1]))
    for w in wrong:
        args = operands("cpu")[call]
        args[name] = w
        with pytest.raises((ValueError, TypeError)):
            call(**args)


def test_other_refusals_of_the_python_calls():
    a = operands("cpu")
    with pytest.raises(ValueError, match="scores"):
        tkg._rule("tanh", 1, 1, True, 1.0)
    with pytest.raises(ValueError, match="both or neither"):
        tkg.swiglu(a[tkg.swiglu]["GU"], a[tkg.swiglu]["H"], Q=a[tkg.swiglu]["Q"])
    with pytest.raises(ValueError, match="together with weights"):
        tkg.swiglu_grad(**dict(a[tkg.swiglu_grad], weights=None))
    with pytest.raises(ValueError, match="can accumulate"):
        tkg.gemm_grouped_dev_mxfp8_wgrad(**a[tkg.gemm_grouped_dev_mxfp8_wgrad], accumulate=True)
    m = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="meta")
    far = 2 ** 32 + 8
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg.moe_dispatch(m(far, 64), m(far, 1, dtype=I32), m(far, 64))
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg.moe_route(m(far, 64), m(far, 1, dtype=I32), m(far, 1, dtype=F32), m(64, dtype=I32), m(far, 1, dtype=I32), m(far, dtype=I32))
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg.checkpoint_mxfp8(m(8, 2 ** 32), m(8, 2 ** 32, dtype=U8), m(8, 2 ** 27, dtype=U8))


@pytest.mark.gpu
@pytest.mark.parametrize("call,name", NAMES, ids=ids)
def test_one_host_tensor_is_refused(call, name):
    args = operands("cuda")[call]
    call(**args)
    args[name] = args[name].cpu()
    with pytest.raises(ValueError, match=f"{name}: a tensor on the GPU is wanted"):
        call(**args)
    assert tkg.device_status() == tkg.OK
