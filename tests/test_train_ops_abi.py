"""Host-side checks of the training-side entry points: what is refused, and what
is nothing to do, before any CUDA call (no GPU needed).  The pointers are never
dereferenced."""
import ctypes

import pytest

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from dense_block_scaled_gb300 import build, tkg
    build.build()
    return tkg.load()


def loss(lib, tokens=8, vocab=100, hidden=64, X=P, ldx=None, W=P, ldw=None, labels=P, alpha=1.0, loss=P, lse=P, ws=P,
         nbytes=BIG):
    return lib.tkg_linear_ce_loss(tokens, vocab, hidden, X, hidden if ldx is None else ldx, W,
                                  hidden if ldw is None else ldw, labels, alpha, loss, lse, ws, nbytes, None)


def grad(lib, tokens=8, vocab=100, hidden=64, X=P, ldx=None, W=P, ldw=None, labels=P, lse=P, dloss=P, dX=P, lddx=None,
         dW=P, lddw=None, kind=0, piece=0, ws=P, nbytes=BIG):
    d = lambda x: hidden if x is None else x
    return lib.tkg_linear_ce_grad(tokens, vocab, hidden, X, d(ldx), W, d(ldw), labels, 1.0, lse, dloss, dX, d(lddx), dW,
                                  d(lddw), kind, piece, ws, nbytes, None)


@pytest.mark.parametrize("call", [loss, grad])
def test_head_arguments(lib, call):
    from dense_block_scaled_gb300 import tkg
    for bad in (dict(tokens=-1), dict(vocab=-1), dict(hidden=-8), dict(X=None), dict(W=None), dict(labels=None),
                dict(ldx=56), dict(ldw=56), dict(ws=None), dict(nbytes=0)):
        assert call(lib, **bad) == tkg.ERR_INVALID_ARG, bad
    for bad in (dict(vocab=0), dict(hidden=0)):
        assert call(lib, **bad) == tkg.ERR_UNSUPPORTED, bad
    for bad in (dict(hidden=60), dict(ldx=68), dict(ldw=68), dict(X=ODD), dict(W=ODD), dict(labels=ODD), dict(ws=ODD),
                dict(lse=ODD)):
        assert call(lib, **bad) == tkg.ERR_ALIGNMENT, bad


def test_loss_arguments(lib):
    from dense_block_scaled_gb300 import tkg
    assert loss(lib, loss=None) == tkg.ERR_INVALID_ARG
    assert loss(lib, lse=None) == tkg.ERR_INVALID_ARG
    assert loss(lib, loss=ODD) == tkg.ERR_ALIGNMENT
    need = lib.tkg_linear_ce_loss_workspace_bytes(8, 100)
    assert need > 0 and loss(lib, nbytes=need - 1) == tkg.ERR_INVALID_ARG
    assert loss(lib, tokens=0, X=None, labels=None, ws=None, nbytes=0) == tkg.OK
    assert lib.tkg_linear_ce_loss_workspace_bytes(-1, 100) == 0


def test_grad_arguments(lib):
    from dense_block_scaled_gb300 import tkg
    for bad in (dict(lse=None), dict(dloss=None), dict(lddx=56), dict(lddw=56), dict(kind=3), dict(kind=-1),
                dict(piece=-1)):
        assert grad(lib, **bad) == tkg.ERR_INVALID_ARG, bad
    for bad in (dict(dX=ODD), dict(dW=ODD), dict(lddx=68), dict(lddw=68), dict(kind=1, lddw=66), dict(dloss=ODD)):
        assert grad(lib, **bad) == tkg.ERR_ALIGNMENT, bad
    for piece in (0, 16, 64, 1000):
        need = lib.tkg_linear_ce_grad_workspace_bytes(8, 100, 64, piece)
        assert need > 0 and grad(lib, piece=piece, nbytes=need - 1) == tkg.ERR_INVALID_ARG
    assert grad(lib, dX=None, dW=None) == tkg.OK
    assert grad(lib, tokens=0, dW=None, ws=None, nbytes=0) == tkg.OK
    assert grad(lib, tokens=0, kind=2, ws=None, nbytes=0) == tkg.OK
    assert lib.tkg_linear_ce_grad_workspace_bytes(8, 100, 64, -1) == 0


def test_workspaces_do_not_grow_with_the_vocabulary_alone(lib):
    # g is kept for one piece: past it the gradient's workspace stays the same
    one = lib.tkg_linear_ce_grad_workspace_bytes(8192, 65536, 4096, 8192)
    assert lib.tkg_linear_ce_grad_workspace_bytes(8192, 262144, 4096, 8192) == one
    auto = lib.tkg_linear_ce_grad_workspace_bytes(8192, 262144, 4096, 0)
    assert auto < 8192 * 262144 * 2 / 2


def test_grouped_arguments(lib):
    from dense_block_scaled_gb300 import tkg

    def dgrad(groups=2, sizes=P, cap=8, n=64, k=64, dD=P, B=P, dA=P):
        return lib.tkg_gemm_grouped_dev_bf16_dgrad(groups, sizes, cap, n, k, dD, B, dA, 1.0, None)

    def wgrad(groups=2, sizes=P, cap=8, n=64, k=64, dD=P, A=P, dB=P, kind=0):
        return lib.tkg_gemm_grouped_dev_bf16_wgrad(groups, sizes, cap, n, k, dD, A, dB, kind, 1.0, None)

    for call in (dgrad, wgrad):
        for bad in (dict(groups=0), dict(sizes=None), dict(cap=-1), dict(n=-8), dict(k=-8), dict(dD=None)):
            assert call(**bad) == tkg.ERR_INVALID_ARG, bad
        assert call(groups=129) == tkg.ERR_UNSUPPORTED
        for bad in (dict(sizes=ODD), dict(n=60), dict(k=60), dict(dD=ODD)):
            assert call(**bad) == tkg.ERR_ALIGNMENT, bad
    assert dgrad(B=None) == dgrad(dA=None) == tkg.ERR_INVALID_ARG
    assert dgrad(B=ODD) == dgrad(dA=ODD) == tkg.ERR_ALIGNMENT
    assert dgrad(n=0) == tkg.ERR_UNSUPPORTED
    assert dgrad(cap=0, dD=None) == dgrad(k=0, dA=None) == tkg.OK
    assert wgrad(A=None) == wgrad(dB=None) == wgrad(kind=3) == tkg.ERR_INVALID_ARG
    assert wgrad(A=ODD) == wgrad(dB=ODD) == tkg.ERR_ALIGNMENT
    assert wgrad(n=0, dB=None) == wgrad(k=0, dB=None) == wgrad(cap=0, kind=2) == tkg.OK
