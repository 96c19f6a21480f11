"""Streamed products of a transposed left operand whose rows make several blocks: of widths
that are no multiple of 256, each block starts where the one before it ends."""
import numpy as np
import pytest

import block_ref as ref
from helpers import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


def sync(t):
    import dense_gemm_03_gb300 as g
    t.cuda.synchronize()
    assert g.debug_status() == 0


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("M,N,K", [
    (320, 512, 2048), (320, 1000, 8192), (320, 64, 1024), (448, 128, 1175), (448, 130, 1536),
    (640, 512, 2048), (640, 1536, 1536), (704, 512, 2048), (832, 100, 1024), (896, 896, 1536),
    (896, 128, 2048), (960, 512, 2048), (1152, 64, 2048), (1600, 96, 1024), (2880, 128, 1024),
    (330, 512, 2048), (1151, 96, 1024),
    (256, 512, 2048), (512, 512, 1536), (1024, 128, 1024)])
def test_transposed_left_operand(M, N, K, tb):
    """Entries of -1, 0 and 1: sums are exact, and small enough for halves."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator().manual_seed(M + 3 * N + K)
    A = t.randint(-1, 2, (K, M), generator=gen).half().cuda()
    B = t.randint(-1, 2, (K, N), generator=gen).half().cuda()
    want = A.double().t() @ B.double()
    assert float(want.abs().max()) <= 2048
    C, H = t.empty(M, N, device="cuda"), t.empty(M, N, dtype=t.float16, device="cuda")
    b = B.t().contiguous() if tb else B
    for call, out in ((g.gemm_f16_trans_f32out, C), (g.gemm_f16_trans, H)):
        call(A, b, out, True, tb)
        assert g.last_path().startswith("trans.stream")
        sync(t)
        assert t.equal(out.double(), want)


@pytest.mark.parametrize("T,K,N", [(2048, 320, 256), (2048, 896, 500), (1600, 448, 1024)])
@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_weight_gradient(T, K, N, beta):
    """dW of a gate whose input is K wide, over T tokens."""
    import dense_gemm_03_gb300 as g
    t = torch()
    rng = np.random.default_rng(T + K)
    new = lambda *s, std=1.0: t.from_numpy(rng.normal(0, std, s).astype(np.float16))
    X, W, dC, W0 = new(T, K), new(K, 2 * N, std=K ** -0.5), new(T, N, std=0.5), new(K, 2 * N)
    gu, dX, dW = (t.empty(*s, dtype=t.float16, device="cuda") for s in ((T, 2 * N), (T, K), (K, 2 * N)))
    dW.copy_(W0)
    g.gemm_f16_glu_grad(dC.cuda(), X.cuda(), W.cuda(), gu, dX, dW, beta=beta)
    sync(t)
    held = gu.cpu()
    ref.check(held, *ref.glu_grad(dC, X, W, "silu"), "dGU")
    ref.check(dX.cpu(), *ref.product(held, W.t()), "dX")
    ref.check(dW.cpu(), *ref.product(X.t(), held, 1.0, beta, W0), "dW")
