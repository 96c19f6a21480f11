"""Sums of 8-bit products past 2^24, where they are no longer exact."""
import pytest

import block_ref as ref
from helpers import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


@pytest.mark.parametrize("M,N,K", [(1, 256, 8192), (40, 300, 8192), (130, 512, 16384), (700, 2600, 8192)])
@pytest.mark.parametrize("act", [None, "silu"])
def test_tokens_of_one_sign(M, N, K, act):
    """Tokens that were relu'd and weights of one sign: sums of 5e7 and more.  In any order, and
    truncating, K additions leave at most K x 2^-23 of such a sum (the definition's own bound,
    2 parts in a thousand); as the tensor core adds, 16 at a time, K / 16 of them."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator().manual_seed(M + K)
    cols = 2 * N if act else N
    X = t.randint(0, 128, (M, K), generator=gen).to(t.int8)
    W = t.randint(60, 128, (K, cols), generator=gen).to(t.int8)
    sx, sw = (t.rand(n, generator=gen) * 2e-4 + 1e-4 for n in (M, cols))
    sw[:N] /= K / 1024
    sw[N:] /= K / 1024
    C = t.empty(M, N, dtype=t.float16, device="cuda")
    g.gemm_i8(X.cuda(), W.cuda(), C, sx.cuda(), sw.cuda(), act)
    t.cuda.synchronize()
    assert g.debug_status() == 0
    S, e = ref.i8_sums(X, W)
    assert float(S.min()) > 2 ** 24
    ref.check(C.cpu(), *ref.i8(X, W, sx, sw, act), g.last_path())
    if act is None:
        want = S * sx.double()[:, None] * sw.double()[None, :]
        off = (C.cpu().double() - want).abs()
        assert bool((off <= ref.half_round(want) + (K / 16 + 8) * 2.0 ** -23 * want).all())
