"""Long sums are added up in parts, rounded to nearest: how far they are off, where a
result shows it, and that it takes no scratch to speak of.

The tensor core truncates as it adds, 16 products at a time: a step is off by a fraction of the
last place of the sum so far, 0.36 x 2^-23 of it on the average (uniform over the place, the place
2^-24 to 2^-23 of the value), and always toward the same side of zero.  For a sum of n products of
standard normals, |sum so far| is on the average 2/3 x 0.8 x sqrt(n), so n / 16 steps are off by
n / 16 x 0.36 x 2^-23 x 0.53 sqrt(n), with a root mean square 1.25 times that (as |normal|'s).
Parts of 512: 2.1e-5 each; of 1024: 5.8e-5; sums of 4096 in one go: 4.7e-4.  Parts' errors have
their sums' signs and add up like independent ones; rounding to nearest adds less than 2^-24
of a sum for each part, which counts for little."""
import pytest

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


def rms(t, x):
    return float(x.double().pow(2).mean().sqrt())


def there_and_back(t, M, N, K, seed):
    """X and W = [Wg Wu] whose sums climb to sqrt(K / 2) and return to 2^-6, exactly."""
    gen = t.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: t.randn(s, generator=gen, device="cuda").half()
    n = K // 2
    X, W = normal(M, K), normal(K, 2 * N)
    order = t.randperm(n - 1, generator=gen, device="cuda") + 1
    X[:, 0], X[:, n] = 1, 0
    W[0], W[n] = 2.0 ** -6, 0
    X[:, n + 1:2 * n] = X[:, order]
    W[n + 1:2 * n] = -W[order]
    if K % 2:
        X[:, -1] = 0
    return X, W


@pytest.mark.parametrize("M,N,K,path", [
    (700, 1368, 4096, "gate_grad.fold"), (1500, 1111, 4096, "glu_grad.copied"),
    (2000, 2048, 4097, "glu_grad.copied"), (64, 1000, 4096, "glu.stream"),
    (2048, 4096, 4096, "gate_grad.fold"), (8192, 8192, 4096, "gate_grad.fold")])
def test_relu_gradient(M, N, K, path):
    """G and U are 2^-6, and so are dU and dG for dC = 1, but for the sums' errors and a
    rounding to 2^-17 at most: eight parts of 512, off by 2.1e-5 x sqrt(8) = 5.9e-5; twice that is
    allowed.  Sums of 4096 in one go, to 45 and back, are off by 3.3e-4."""
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W = there_and_back(t, M, N, K, M + N)
    dC = t.ones(M, N, dtype=t.float16, device="cuda")
    gu = t.empty(M, 2 * N, dtype=t.float16, device="cuda")
    g.gemm_f16_glu_grad(dC, X, W, gu, act="relu")
    assert path in g.last_path()
    sync(t)
    assert rms(t, gu[:, :N].float() - 2.0 ** -6) <= 1.2e-4      # dG = U
    assert rms(t, gu[:, N:].float() - 2.0 ** -6) <= 1.2e-4      # dU = G


def test_relu_gradient_takes_little_scratch():
    """Nothing but the partial sums of a last wave of tiles: 76 of 256 x 256 floats, twice."""
    import dense_gemm_03_gb300 as g
    t = torch()
    M, K, N = 4096, 2048, 4096
    X, W = there_and_back(t, M, N, K, 1)
    dC = t.ones(M, N, dtype=t.float16, device="cuda")
    gu = t.empty(M, 2 * N, dtype=t.float16, device="cuda")
    g.gemm_f16_glu_grad(dC, X, W, gu, act="relu")     # (its code is loaded)
    sync(t)
    stream = t.cuda.Stream()
    before = t.cuda.mem_get_info()[0]
    g.gemm_f16_glu_grad(dC, X, W, gu, act="relu", stream=stream)
    sync(t)
    assert before - t.cuda.mem_get_info()[0] <= 76 * 2 * 256 * 256 * 4 + (8 << 20)


@pytest.mark.parametrize("ta,tb", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,N,K,path", [
    (1024, 2048, 8192, "pair"), (4096, 4096, 4096, "ktail"), (1000, 2050, 8192, "pair"),
    (128, 512, 8192, "trans.stream"), (96, 4096, 4096, "trans.stream")])
def test_float_results(M, N, K, path, ta, tb):
    """Parts of 1024 products at most: off by 5.8e-5 x sqrt(K / 1024), 1.8e-6 of the sums' size;
    2.5e-6 is allowed.  In one go they are off by 7e-6 (4096) and more."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(M + N + K)
    A = t.randn((K, M) if ta else (M, K), generator=gen, device="cuda").half()
    B = t.randn((N, K) if tb else (K, N), generator=gen, device="cuda").half()
    C = t.empty(M, N, device="cuda")
    g.gemm_f16_trans_f32out(A, B, C, ta, tb)
    assert path in g.last_path()
    sync(t)
    want = (A.t() if ta else A).double() @ (B.t() if tb else B).double()
    assert rms(t, C - want) <= 2.5e-6 * rms(t, want)


@pytest.mark.parametrize("M,N,K", [(192, 16384, 16384), (128, 16384, 16384)])
def test_long_float_sums_over_few_rows(M, N, K):
    """Their parts are added up on the chip too: as exact, and with the scratch of a last wave."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(M)
    A, B = (t.randn(K, n, generator=gen, device="cuda").half() for n in (M, N))
    C = t.empty(M, N, device="cuda")
    g.gemm_f16_trans_f32out(A, B, C, True)            # (its code is loaded)
    sync(t)
    stream = t.cuda.Stream()
    before = t.cuda.mem_get_info()[0]
    g.gemm_f16_trans_f32out(A, B, C, True, stream=stream)
    sync(t)
    assert before - t.cuda.mem_get_info()[0] <= 76 * 2 * 256 * 256 * 4 + (8 << 20)
    rows = [0, M // 2, M - 1]
    want = A[:, rows].double().t() @ B.double()
    assert rms(t, C[rows] - want) <= 2.5e-6 * rms(t, want)
