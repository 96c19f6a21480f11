"""What the binding refuses before the row-routed products are called: index
operands of another type or too short, views that are not dense where no leading
dimension says so, shapes that disagree."""
import numpy as np
import pytest

import dense_gemm_03_gb300 as g
from helpers import torch

M, N, K, R, n = 6, 16, 8, 4, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


def lora(**kw):
    t = torch()
    h = dict(dtype=t.float16)
    o = dict(X=t.zeros(M, K, **h), W=t.zeros(K, N, **h), C=t.zeros(M, N, **h),
             A=t.zeros(n, K, R, **h), B=t.zeros(n, R, N, **h), ids=t.zeros(M, dtype=t.int32),
             scales=t.ones(n), G=t.zeros(M, N, **h), dX=t.zeros(M, K, **h),
             dA=t.zeros(n, K, R), dB=t.zeros(n, R, N))
    o.update(kw)
    return o


def forward(o, **kw):
    g.gemm_f16_lora(o["X"], o["W"], o["C"], o["A"], o["B"], o["ids"], o["scales"], **kw)


def grad(o, **kw):
    g.gemm_f16_lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"], o["dX"],
                         o["dA"], o["dB"], **kw)


def moe(topk=2, **kw):
    t = torch()
    T, H, I, E = 5, 16, 8, 4
    h = dict(dtype=t.float16)
    o = dict(X=t.zeros(T, H, **h), Wr=t.zeros(H, E, **h), W1=t.zeros(E, H, 2 * I, **h),
             W2=t.zeros(E, I, H, **h), Y=t.zeros(T, H, **h), ids=t.zeros(T, topk, dtype=t.int32),
             probs=t.zeros(T, topk))
    o.update(kw)
    g.gemm_f16_moe(o["X"], o["Wr"], o["W1"], o["W2"], o["Y"], topk, ids=o["ids"], probs=o["probs"])


@pytest.mark.parametrize("call", [forward, grad])
def test_types_of_index_operands(call):
    t = torch()
    with pytest.raises(TypeError, match="ids is int64, not int32"):
        call(lora(ids=t.zeros(M, dtype=t.int64)))
    with pytest.raises(TypeError, match="ids is int64"):
        call(lora(ids=np.zeros(M, np.int64)))
    with pytest.raises(TypeError, match="scales is float16"):
        call(lora(scales=t.ones(n, dtype=t.float16)))
    with pytest.raises(TypeError, match="scales is float64"):
        call(lora(scales=np.ones(n)))


@pytest.mark.parametrize("call", [forward, grad])
def test_views_and_lengths(call):
    t = torch()
    with pytest.raises(ValueError, match="ids"):
        call(lora(ids=t.zeros(M - 1, dtype=t.int32)))
    with pytest.raises(ValueError, match="ids"):
        call(lora(ids=t.zeros(2 * M, dtype=t.int32)[::2]))
    with pytest.raises(ValueError, match="scales"):
        call(lora(scales=t.ones(n - 1)))
    with pytest.raises(ValueError, match="A is not dense"):
        call(lora(A=t.zeros(n, R, K, dtype=t.float16).transpose(1, 2)))
    with pytest.raises(ValueError, match="B is not dense"):
        call(lora(B=np.zeros((R, n, N), np.float16).transpose(1, 0, 2)))
    with pytest.raises(ValueError, match="K of A"):
        call(lora(A=t.zeros(n, K + 8, R, dtype=t.float16)))


def test_forward_shapes():
    t = torch()
    with pytest.raises(ValueError, match="K of W"):
        forward(lora(W=t.zeros(N, K + 1, dtype=t.float16)))


def test_gradients_outputs():
    t = torch()
    with pytest.raises(TypeError, match="dA is float16"):
        grad(lora(dA=t.zeros(n, K, R, dtype=t.float16)))
    with pytest.raises(ValueError, match="dB"):
        grad(lora(dB=t.zeros(n, R, N - 1)))
    with pytest.raises(ValueError, match="dA"):
        grad(lora(dA=t.zeros(n, R, K).transpose(1, 2)))


def test_experts():
    t = torch()
    with pytest.raises(TypeError, match="ids is int64"):
        moe(ids=t.zeros(5, 2, dtype=t.int64))
    with pytest.raises(TypeError, match="probs is float16"):
        moe(probs=t.zeros(5, 2, dtype=t.float16))
    with pytest.raises(ValueError, match="ids"):
        moe(ids=t.zeros(5, 1, dtype=t.int32))
    with pytest.raises(ValueError, match="W1 is not dense"):
        moe(W1=t.zeros(4, 16, 16, dtype=t.float16).transpose(1, 2))
    with pytest.raises(ValueError, match="Wr is not dense"):
        moe(Wr=t.zeros(4, 16, dtype=t.float16).t())
    with pytest.raises(ValueError, match="H of W2"):
        moe(W2=t.zeros(4, 8, 24, dtype=t.float16))


def test_what_is_right_passes_the_checks():
    """(empty calls, which need no device)"""
    t = torch()
    o = lora()
    forward(o, M=0)
    forward(lora(ids=np.zeros(M, np.int32), scales=None), M=0)
    o["dX"] = o["dA"] = o["dB"] = None
    grad(o)
    # views of wider buffers with their leading dimensions
    wide = t.zeros(n, K, R + 4, dtype=t.float16)
    forward(lora(A=wide[:, :, :R]), M=0, N=N, K=K, R=R, adapters=n, lda=R + 4)
    g.gemm_f16_moe(16, 16, 16, 16, 16, 2, T=0, H=8, I=8, E=4)
