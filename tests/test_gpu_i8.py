"""Products in 8-bit integers with scales by token and channel, and tokens rounded
to 8 bits, through the public binding, against the 64-bit definitions."""
import numpy as np
import pytest

import block_ref as ref
from helpers import torch
from test_gpu_block import Padded, normal, sync

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


SHAPES = [
    # M, N, K, pads of X, W, C, shift of X, W
    (1, 1, 1, 0, 0, 0, 0),
    (1, 128, 128, 0, 0, 0, 0),
    (1, 1000, 500, 0, 0, 0, 0),
    (3, 256, 1024, 16, 16, 8, 0),
    (16, 130, 90, 3, 1, 5, 1),
    (33, 640, 4096, 0, 0, 0, 0),
    (128, 516, 300, 0, 4, 1, 4),
    (129, 64, 128, 0, 0, 0, 0),
    (200, 300, 1000, 8, 4, 0, 0),
    (640, 5000, 100, 0, 0, 0, 0),
    (1025, 2504, 130, 1, 3, 1, 5),
    (777, 5001, 64, 0, 0, 0, 0),
    (2048, 2560, 1040, 0, 0, 0, 0),
]


def operands(t, M, cols, K):
    rng = np.random.default_rng(100 * M + 10 * cols + K)
    X = t.from_numpy(rng.integers(-128, 128, (M, K)).astype(np.int8))
    W = t.from_numpy(rng.integers(-128, 128, (K, cols)).astype(np.int8))
    # products of scales that bring results to about 1
    sx = t.from_numpy(rng.uniform(0.5, 2, M).astype(np.float32) / (74 * K ** 0.5))
    sw = t.from_numpy(rng.uniform(0.5, 2, cols).astype(np.float32) / 74)
    return X, W, sx, sw, rng


@pytest.mark.parametrize("act", (None,) + ref.ACTS)
@pytest.mark.parametrize("M,N,K,px,pw,pc,shift", SHAPES)
def test_i8(M, N, K, px, pw, pc, shift, act):
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W, sx, sw, rng = operands(t, M, N if act is None else 2 * N, K)
    C0 = normal(t, rng, (M, N))
    x, w = Padded(t, X, px, shift), Padded(t, W, pw, shift)
    for beta in (0.0, 0.5) if act is None else (0.0,):
        c = Padded(t, C0 if beta else t.full((M, N), float("nan"), dtype=t.float16), pc, 0)
        g.gemm_i8(x.ptr, w.ptr, c.ptr, sx.cuda(), sw.cuda(), act, beta, M=M, N=N, K=K, ldx=x.ld,
                  ldw=w.ld, ldc=c.ld)
        sync(t)
        ref.check(c.view.cpu(), *ref.i8(X, W, sx, sw, act, beta, C0), g.last_path())
        assert c.untouched(t)


@pytest.mark.parametrize("M,N,K", [(5, 300, 700), (700, 2600, 200)])
def test_i8_without_scales(M, N, K):
    """Ones in the place of a missing scale; sums past the half range are infinite."""
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W, sx, sw, _ = operands(t, M, N, K)
    C = t.empty(M, N, dtype=t.float16, device="cuda")
    for a, b in ((None, sw), (sx, None), (None, None)):
        g.gemm_i8(X.cuda(), W.cuda(), C, None if a is None else a.cuda(), None if b is None else b.cuda())
        sync(t)
        want, tol = ref.i8(X, W, a, b)
        got = C.cpu().double()
        big = want.abs() > 65520 + 64
        assert bool((got[big] == want[big].sign() * float("inf")).all())
        ok = want.abs() < 65504
        ref.check(got[ok], want[ok], tol[ok])


@pytest.mark.parametrize("M,N,K", [(2, 128, 1024), (130, 128, 1024), (600, 2600, 1024)])
@pytest.mark.parametrize("x,w", [(-128, -128), (127, -128), (-128, 127)])
def test_i8_largest_magnitudes(M, N, K, x, w):
    """The largest sums of 1024 products are exact (2^24)."""
    import dense_gemm_03_gb300 as g
    t = torch()
    C = t.empty(M, N, dtype=t.float16, device="cuda")
    X = t.full((M, K), x, dtype=t.int8, device="cuda")
    W = t.full((K, N), w, dtype=t.int8, device="cuda")
    sx = t.full((M,), 2.0 ** -10, device="cuda")
    g.gemm_i8(X, W, C, sx)
    sync(t)
    assert t.equal(C.double(), t.full_like(C, x * w * K * 2.0 ** -10).double())


def test_i8_every_integer():
    """Each of the 256 values times each of a few: the conversion to halves."""
    import dense_gemm_03_gb300 as g
    t = torch()
    every = t.arange(-128, 128).to(t.int8)
    some = t.tensor([-128, -127, -1, 0, 1, 2, 127, 5], dtype=t.int8)
    for M, N in ((256, 8), (8, 256)):
        X, W = (every if M == 256 else some)[:, None], (some if M == 256 else every)[None, :]
        C = t.empty(M, N, dtype=t.float16, device="cuda")
        g.gemm_i8(X.contiguous().cuda(), W.contiguous().cuda(), C)
        sync(t)
        assert t.equal(C.cpu(), (X.double() @ W.double()).half())


def test_i8_rows_of_other_tokens_do_not_matter():
    """A token whose scale is not finite is NaN or infinite, the others as ever."""
    import dense_gemm_03_gb300 as g
    t = torch()
    for M, N, K in ((7, 256, 256), (600, 2600, 128)):
        X, W, sx, sw, _ = operands(t, M, N, K)
        C, D = (t.empty(M, N, dtype=t.float16, device="cuda") for _ in range(2))
        g.gemm_i8(X.cuda(), W.cuda(), C, sx.cuda(), sw.cuda())
        bad = sx.clone()
        bad[3], bad[5] = float("nan"), float("inf")
        g.gemm_i8(X.cuda(), W.cuda(), D, bad.cuda(), sw.cuda())
        sync(t)
        keep = [i for i in range(M) if i not in (3, 5)]
        assert t.equal(C[keep], D[keep])
        assert bool(D[3].isnan().all()) and not bool(D[5].isfinite().any())


def test_i8_blank():
    import dense_gemm_03_gb300 as g
    t = torch()
    C = t.full((3, 5), 2.0, dtype=t.float16, device="cuda")
    g.gemm_i8(0, 0, C, beta=0.5, M=3, N=5, K=0)
    sync(t)
    assert bool((C == 1).all())
    g.gemm_i8(0, 0, C, act="silu", M=3, N=5, K=0)
    g.gemm_i8(0, 0, 0, M=0, N=5, K=2)
    sync(t)
    assert not bool(C.any())


# ------------------------------------------------------------------- tokens
@pytest.mark.parametrize("M,K,px,pq,sx,sq", [
    (1, 1, 0, 0, 0, 0), (3, 7, 0, 0, 1, 1), (9, 8, 0, 0, 0, 0), (5, 255, 1, 0, 0, 3), (2, 256, 0, 0, 0, 0),
    (17, 500, 4, 4, 0, 0), (4, 1000, 0, 1, 3, 0), (24, 4099, 0, 0, 0, 0), (3, 8192, 8, 8, 0, 0),
    (2, 8191, 1, 1, 1, 7), (2, 20000, 0, 0, 0, 0), (2, 32773, 0, 0, 0, 1), (2, 40000, 0, 0, 0, 0),
    (1000, 64, 0, 0, 0, 0)])
def test_to_i8(M, K, px, pq, sx, sq):
    import dense_gemm_03_gb300 as g
    t = torch()
    rng = np.random.default_rng(M + K)
    X = normal(t, rng, (M, K)) * t.from_numpy(2.0 ** rng.integers(-9, 9, (M, 1))).half()
    x = Padded(t, X, px, sx)
    q = Padded(t, t.zeros(M, K, dtype=t.int8), pq, sq)
    scales = t.full((M + 1,), -1.0, device="cuda")
    g.f16_to_i8(x.ptr, q.ptr, scales, M=M, K=K, ldx=x.ld, ldq=q.ld)
    sync(t)
    want, s = ref.to_i8(X)
    assert t.equal(q.view.cpu(), want) and t.equal(scales[:M].cpu(), s) and float(scales[M]) == -1.0
    assert q.untouched(t) and x.untouched(t)


def test_to_i8_ties_and_every_half():
    """All finite halves beside several maxima, among them ones that make exact ties
    (127 x / a = k + 1/2), subnormal ones and the largest."""
    import dense_gemm_03_gb300 as g
    t = torch()
    every = t.arange(0, 0x7C00, dtype=t.int32).to(t.int16).view(t.float16)
    rows = []
    for a in (254.0, 127.0, 63.5, 1.0, 65504.0, 2.0 ** -24, 2.0 ** -14, 3 * 2.0 ** -24, 8128.0, 0.9922):
        row = every[every <= a]
        row = t.cat([row, -row, t.zeros(2 * every.numel() - 2 * row.numel(), dtype=t.float16)])
        rows.append(row)
    X = t.stack(rows)
    Q = t.empty(X.shape, dtype=t.int8, device="cuda")
    scales = t.empty(len(rows), device="cuda")
    g.f16_to_i8(X.cuda(), Q, scales)
    sync(t)
    # rne(127 x / a) by 64-bit division: 127 x exact, and a quotient that is no tie is at
    # least 2^-12 |quotient| from one, far more than 64 bits round
    x = X.double()
    want = t.round(127 * x / x.abs().amax(1, keepdim=True))
    assert t.equal(Q.cpu().double(), want)
    assert bool((want.abs() == 127).any(1).all())


@pytest.mark.parametrize("M,K,pad", [(25000, 512, 0), (26011, 496, 16), (13000, 1008, 0),
                                     (7001, 1824, 0), (3200, 4096, 32), (1601, 8000, 0),
                                     (803, 16384, 0), (1500, 16400, 0)])
def test_to_i8_many_rows(M, K, pad):
    """Rows by way of the ring (and, past its longest, not), with special rows among them.
    rne(127 x / a) by 64-bit division, as in the test above."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(K)
    X = t.randn(M, K + pad, generator=gen, device="cuda").half()
    X *= t.exp2(t.randint(-9, 9, (M, 1), generator=gen, device="cuda").float()).half()
    X[7], X[11, 5], X[13, K - 1] = 0.0, float("inf"), float("nan")
    X[17, :K] = 254.0
    X[17, :100] = t.arange(100, device="cuda").half()      # ties: 127 x / 254 = x / 2
    Q = t.full((M, K + pad), 9, dtype=t.int8, device="cuda")
    scales = t.empty(M, device="cuda")
    g.f16_to_i8(X, Q, scales, M=M, K=K, ldx=K + pad, ldq=K + pad)
    sync(t)
    assert g.last_path() == ("to_i8" if K > 16384 else "to_i8.ring")
    x = X[:, :K].double()
    a = x.abs().amax(1, keepdim=True)
    want = t.round(127 * x / a)
    want[[7, 11, 13]] = 0
    assert t.equal(Q[:, :K].double(), want) and bool((Q[:, K:] == 9).all())
    s = a[:, 0].float() / t.full_like(scales, 127.0)
    fine = s.isfinite()
    assert t.equal(scales[fine], s[fine]) and scales[11] == float("inf") and bool(scales[13].isnan())


@pytest.mark.parametrize("K", [40, 3000, 50000])
def test_to_i8_special_rows(K):
    """Zeros, infinities and NaNs, each in a row by itself."""
    import dense_gemm_03_gb300 as g
    t = torch()
    X = t.ones(6, K, dtype=t.float16)
    X[1] = 0.0
    X[2, K - 1] = float("inf")
    X[3, 0] = float("nan")
    X[4, 5], X[4, 6] = float("nan"), -float("inf")
    Q = t.full((6, K), 9, dtype=t.int8, device="cuda")
    scales = t.empty(6, device="cuda")
    g.f16_to_i8(X.cuda(), Q, scales)
    sync(t)
    s = scales.cpu()
    assert s[0] == s[5] and s[1] == 0 and s[2] == float("inf") and bool(s[3].isnan()) and bool(s[4].isnan())
    assert bool((Q[[0, 5]] == 127).all()) and not bool(Q[1:5].any())
    W = t.ones(K, 16, dtype=t.int8, device="cuda")
    C = t.empty(6, 16, dtype=t.float16, device="cuda")
    g.gemm_i8(Q, W, C, scales)
    sync(t)
    assert bool(C[2:5].isnan().all()) and not bool(C[1].any()) and bool(C[0].isfinite().all() or K > 40000)


def test_to_i8_blank():
    import dense_gemm_03_gb300 as g
    t = torch()
    scales = t.ones(300, device="cuda")
    g.f16_to_i8(0, 0, scales, M=300, K=0)
    g.f16_to_i8(0, 0, 0, M=0, K=4)
    sync(t)
    assert not bool(scales.any())
