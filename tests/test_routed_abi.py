"""Argument checks of the row-routed products: they answer before any CUDA call."""
import pytest

import dense_gemm_03_gb300 as g

DIM, LD, NULL, ARG = -2, -3, -1, -7


@pytest.fixture(scope="module")
def L():
    from dense_gemm_03_gb300 import build
    build.build()
    return g.lib()


def lora(L, X=16, W=16, C=16, A=16, B=16, ids=16, scales=None, M=4, N=4, K=4, R=2, n=2, ldx=4,
         ldw=4, ldc=4, lda=2, ldb=4, alpha=1.0, beta=0.0):
    return L.gemm_f16_lora(X, W, C, A, B, ids, scales, M, N, K, R, n, ldx, ldw, ldc, lda, ldb,
                           alpha, beta, None)


def grad(L, G=16, X=16, W=16, A=16, B=16, ids=16, scales=None, dX=16, dA=16, dB=16, M=4, N=4, K=4,
         R=2, n=2, ldg=4, ldx=4, ldw=4, lda=2, ldb=4, lddx=4, alpha=1.0, beta=0.0):
    return L.gemm_f16_lora_grad(G, X, W, A, B, ids, scales, dX, dA, dB, M, N, K, R, n, ldg, ldx,
                                ldw, lda, ldb, lddx, alpha, beta, None)


def moe(L, X=16, Wr=16, W1=16, W2=16, Y=16, ids=None, probs=None, T=2, H=4, I=4, E=3, topk=2,
        renorm=1, ldx=4, ldy=4, beta=0.0):
    return L.gemm_f16_moe(X, Wr, W1, W2, Y, ids, probs, T, H, I, E, topk, renorm, ldx, ldy, beta,
                          None)


@pytest.mark.parametrize("code,kw", [
    (DIM, dict(M=-1)), (DIM, dict(N=-1)), (DIM, dict(K=-1)), (DIM, dict(R=-1)), (DIM, dict(n=-1)),
    (ARG, dict(R=129, lda=129)),
    (LD, dict(ldx=3)), (LD, dict(ldw=3)), (LD, dict(ldc=3)), (LD, dict(lda=1)), (LD, dict(ldb=3)),
    (NULL, dict(X=None)), (NULL, dict(W=None)), (NULL, dict(C=None)), (NULL, dict(A=None)),
    (NULL, dict(B=None)), (NULL, dict(ids=None)),
    (ARG, dict(X=17)), (ARG, dict(C=33)), (ARG, dict(B=17)), (ARG, dict(ids=18)),
    (ARG, dict(scales=18)),
    (0, dict(M=0)), (0, dict(N=0)),
    (LD, dict(R=0, ldx=3)), (NULL, dict(n=0, W=None)),
])
def test_lora_refusals(L, code, kw):
    assert lora(L, **kw) == code


@pytest.mark.parametrize("code,kw", [
    (DIM, dict(M=-1)), (DIM, dict(R=-2)), (ARG, dict(R=129, lda=129)),
    (LD, dict(ldg=3)), (LD, dict(ldx=3)), (LD, dict(ldw=3)), (LD, dict(lda=1)), (LD, dict(ldb=3)),
    (LD, dict(lddx=3)),
    (NULL, dict(G=None)), (NULL, dict(X=None)), (NULL, dict(W=None)), (NULL, dict(A=None)),
    (NULL, dict(B=None)), (NULL, dict(ids=None)),
    (ARG, dict(dX=17)), (ARG, dict(dA=18)), (ARG, dict(dB=18)), (ARG, dict(G=17)),
    (0, dict(dX=None, dA=None, dB=None)), (0, dict(dA=None, dB=None, M=0)),
    (NULL, dict(dX=None, X=None)), (NULL, dict(dB=None, B=None)),
])
def test_grad_refusals(L, code, kw):
    assert grad(L, **kw) == code


@pytest.mark.parametrize("code,kw", [
    (DIM, dict(T=-1)), (DIM, dict(H=-1)), (DIM, dict(I=-1)), (DIM, dict(E=-1)),
    (ARG, dict(topk=0)), (ARG, dict(topk=4)), (ARG, dict(E=1025)), (ARG, dict(E=64, topk=33)),
    (ARG, dict(E=0, topk=0)),
    (LD, dict(ldx=3)), (LD, dict(ldy=3)),
    (NULL, dict(X=None)), (NULL, dict(Wr=None)), (NULL, dict(W1=None)), (NULL, dict(W2=None)),
    (NULL, dict(Y=None)),
    (ARG, dict(X=17)), (ARG, dict(Y=17)), (ARG, dict(ids=18)), (ARG, dict(probs=18)),
    (0, dict(T=0)), (0, dict(H=0)),
])
def test_moe_refusals(L, code, kw):
    assert moe(L, **kw) == code


def test_binding_raises():
    with pytest.raises(g.GemmError):
        g.gemm_f16_lora(16, 16, 16, 16, 16, 16, M=4, N=4, K=4, R=200, adapters=2)
    with pytest.raises(g.GemmError):
        g.gemm_f16_moe(16, 16, 16, 16, 16, 9, T=1, H=8, I=8, E=8)
    with pytest.raises(g.GemmError):
        g.gemm_f16_lora_grad(16, 16, 16, 16, 16, 16, dX=17, M=4, N=4, K=4, R=2, adapters=2)
