"""Gated projections, their gradients and products with transposed operands through
the public binding, against the 64-bit definitions."""
import itertools

import numpy as np
import pytest

import block_ref as ref
from helpers import torch

pytestmark = pytest.mark.gpu
SENTINEL = 0x7E55   # a NaN: padding that must stay as it was


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


def sync(t):
    import dense_gemm_03_gb300 as g
    t.cuda.synchronize()
    assert g.debug_status() == 0


class Padded:
    """A (rows, cols) matrix on the GPU with `pad` more columns a row and `shift`
    elements before it, all of them sentinels."""

    def __init__(self, t, x, pad=0, shift=0):
        rows, cols = x.shape
        self.ld, self.shift = cols + pad, shift
        kind = {t.float16: t.int16, t.float32: t.int32, t.int8: t.int8}[x.dtype]
        self.fill = {t.float16: SENTINEL, t.float32: 0x7FC0DEAD, t.int8: 0x55}[x.dtype]
        flat = t.full((shift + max(rows, 1) * self.ld + 8,), self.fill, dtype=kind).view(x.dtype)
        self.buf = flat.cuda()
        self.view = self.buf[shift:shift + rows * self.ld].view(rows, self.ld)[:, :cols]
        self.view.copy_(x.cuda())

    @property
    def ptr(self):
        return self.buf.data_ptr() + self.shift * self.buf.element_size()

    def untouched(self, t):
        """Every element outside the matrix still holds the sentinel."""
        rows, cols = self.view.shape
        mask = t.ones(self.buf.shape, dtype=t.bool, device="cuda")
        mask[self.shift:self.shift + rows * self.ld].view(rows, self.ld)[:, :cols] = False
        kind = {2: t.int16, 4: t.int32, 1: t.int8}[self.buf.element_size()]
        return bool((self.buf.view(kind)[mask] == self.fill).all())


def normal(t, rng, shape, std=1.0, dtype=np.float16):
    return t.from_numpy(rng.normal(0, std, shape).astype(dtype))


# ---------------------------------------------------------------- transposed
TRANS = [
    # M, N, K, pads of A, B, C, shift of every pointer
    (1, 1, 1, 0, 0, 0, 0),
    (1, 300, 513, 7, 0, 0, 0),
    (5, 64, 64, 0, 0, 0, 0),
    (127, 129, 65, 1, 3, 5, 1),
    (130, 640, 96, 0, 0, 8, 0),
    (333, 2056, 200, 8, 8, 8, 0),
    (512, 5120, 72, 0, 0, 0, 0),
    (1031, 2051, 77, 1, 0, 3, 0),
    (2049, 1992, 1, 0, 0, 0, 0),
    (700, 96, 1500, 0, 0, 0, 0),
]


@pytest.mark.parametrize("ta,tb", [(True, False), (False, True), (True, True), (False, False)])
@pytest.mark.parametrize("M,N,K,pa,pb,pc,shift", TRANS)
def test_trans(M, N, K, pa, pb, pc, shift, ta, tb):
    import dense_gemm_03_gb300 as g
    t = torch()
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    A, B = normal(t, rng, (M, K)), normal(t, rng, (K, N), K ** -0.5)
    C0 = normal(t, rng, (M, N))
    a = Padded(t, A.t().contiguous() if ta else A, pa, shift)
    b = Padded(t, B.t().contiguous() if tb else B, pb, shift)
    for f32, (alpha, beta) in itertools.product((False, True), ((1.0, 0.0), (-1.5, 0.5))):
        c = Padded(t, C0.float() if f32 else C0, pc, shift)
        if beta == 0.0:
            c.view.fill_(float("nan"))     # not read
        call = g.gemm_f16_trans_f32out if f32 else g.gemm_f16_trans
        call(a.ptr, b.ptr, c.ptr, ta, tb, alpha, beta, M=M, N=N, K=K, lda=a.ld, ldb=b.ld, ldc=c.ld)
        sync(t)
        want, tol = ref.product(A, B, alpha, beta, C0, f32)
        ref.check(c.view.cpu(), want, tol, "%s f32=%s" % (g.last_path(), f32))
        assert c.untouched(t)


@pytest.mark.parametrize("ta,tb", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,N,K", [(96, 200, 640), (1024, 5000, 320), (2304, 4864, 3200)])
def test_trans_integers_exact(M, N, K, ta, tb):
    """Small integers: every sum is exact in fp32 and as a float result."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator().manual_seed(M + N)
    A = t.randint(-3, 4, (M, K), generator=gen).half()
    B = t.randint(-3, 4, (K, N), generator=gen).half()
    C = t.empty(M, N, device="cuda")
    g.gemm_f16_trans_f32out((A.t().contiguous() if ta else A).cuda(),
                            (B.t().contiguous() if tb else B).cuda(), C, ta, tb)
    sync(t)
    assert t.equal(C, (A.cuda().double() @ B.cuda().double()).float())


def test_trans_empty_and_blank():
    import dense_gemm_03_gb300 as g
    t = torch()
    C = t.full((4, 6), 2.0, dtype=t.float16, device="cuda")
    F = t.full((4, 6), 2.0, device="cuda")
    nan = t.full((6, 8), float("nan"), dtype=t.float16, device="cuda")
    g.gemm_f16_trans(nan[:, :4].t(), nan, C, False, True, beta=0.5, M=4, N=6, K=0, lda=8, ldb=8)
    g.gemm_f16_trans_f32out(nan, nan, F, True, False, alpha=0.0, beta=0.5, M=4, N=6, K=6, lda=8, ldb=8)
    g.gemm_f16_trans(0, 0, 0, True, True, M=0, N=6, K=3)
    sync(t)
    assert bool((C == 1).all()) and bool((F == 1).all())


# ------------------------------------------------------------------- gated
GLU = [
    # M, N, K, pads of X, W, C (and dC, dGU), shift
    (1, 1, 1, 0, 0, 0, 0),
    (1, 8, 64, 0, 0, 0, 0),
    (1, 1001, 500, 0, 0, 0, 0),
    (3, 256, 1024, 8, 16, 8, 0),
    (17, 130, 90, 3, 1, 5, 1),
    (64, 520, 2048, 0, 0, 0, 0),
    (129, 64, 128, 0, 0, 0, 0),
    (300, 2504, 72, 0, 8, 8, 0),
    (777, 1501, 100, 0, 0, 0, 0),
    (640, 1500, 136, 0, 0, 0, 0),
    (1025, 1432, 64, 1, 1, 1, 1),
    (2048, 2560, 40, 0, 0, 0, 0),
]


def operands(t, M, N, K, spread=2.0):
    """Gates with a standard deviation of `spread` (both tails of f), U about 1."""
    rng = np.random.default_rng(1000 * M + 10 * N + K)
    X = normal(t, rng, (M, K))
    W = normal(t, rng, (K, 2 * N), K ** -0.5)
    W[:, :N] *= spread
    return X, W, normal(t, rng, (M, N), 0.5)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M,N,K,px,pw,pc,shift", GLU)
def test_glu(M, N, K, px, pw, pc, shift, act):
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W, _ = operands(t, M, N, K)
    x, w = Padded(t, X, px, shift), Padded(t, W, pw, shift)
    c = Padded(t, t.full((M, N), float("nan"), dtype=t.float16), pc, shift)
    g.gemm_f16_glu(x.ptr, w.ptr, c.ptr, act, M=M, N=N, K=K, ldx=x.ld, ldw=w.ld, ldc=c.ld)
    sync(t)
    ref.check(c.view.cpu(), *ref.glu(X, W, act), g.last_path())
    assert c.untouched(t)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M,N,K,px,pw,pc,shift", GLU)
def test_glu_grad(M, N, K, px, pw, pc, shift, act):
    """dGU against the formula; dX and dW against the products of what dGU holds."""
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W, dC = operands(t, M, N, K)
    x, w, dc = Padded(t, X, px, shift), Padded(t, W, pw, shift), Padded(t, dC, pc, shift)
    nan = lambda *s: t.full(s, float("nan"), dtype=t.float16)
    W0 = normal(t, np.random.default_rng(3), (K, 2 * N))
    for beta in (0.0, 0.5):
        gu = Padded(t, nan(M, 2 * N), pc, shift)
        dx = Padded(t, nan(M, K), px, shift)
        dw = Padded(t, W0 if beta else nan(K, 2 * N), pw, shift)
        g.gemm_f16_glu_grad(dc.ptr, x.ptr, w.ptr, gu.ptr, dx.ptr, dw.ptr, act, beta, M=M, N=N, K=K,
                            lddc=dc.ld, ldx=x.ld, ldw=w.ld, lddgu=gu.ld, lddx=dx.ld, lddw=dw.ld)
        sync(t)
        ref.check(gu.view.cpu(), *ref.glu_grad(dC, X, W, act), "dGU")
        held = gu.view.cpu()
        ref.check(dx.view.cpu(), *ref.product(held, W.t()), "dX")
        ref.check(dw.view.cpu(), *ref.product(X.t(), held, 1.0, beta, W0), "dW")
        assert gu.untouched(t) and dx.untouched(t) and dw.untouched(t)


@pytest.mark.parametrize("M,N,K", [(9, 48, 40), (400, 2504, 24)])
def test_glu_grad_parts(M, N, K):
    """dX and dW are the same whether asked for alone or together; dGU always comes."""
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W, dC = (v.cuda() for v in operands(t, M, N, K))
    new = lambda *s: t.full(s, float("nan"), dtype=t.float16, device="cuda")
    gu, dX, dW = new(M, 2 * N), new(M, K), new(K, 2 * N)
    g.gemm_f16_glu_grad(dC, X, W, gu, dX, dW)
    for want_x, want_w in ((True, False), (False, True), (False, False)):
        gu2, dX2, dW2 = new(M, 2 * N), new(M, K), new(K, 2 * N)
        g.gemm_f16_glu_grad(dC, X, W, gu2, dX2 if want_x else None, dW2 if want_w else None)
        sync(t)
        assert t.equal(gu, gu2)
        assert t.equal(dX, dX2) if want_x else bool(dX2.isnan().all())
        assert t.equal(dW, dW2) if want_w else bool(dW2.isnan().all())


@pytest.mark.parametrize("act", ref.ACTS)
def test_glu_grad_by_differences(act):
    """The gradients against central differences of the 64-bit forward formula: the
    step's own error, h^2 / 6 of a third derivative of order one, is far below 1e-6."""
    import dense_gemm_03_gb300 as g
    t = torch()
    M, N, K = 6, 10, 12
    X, W, dC = operands(t, M, N, K, 1.0)
    out = [t.empty(s, dtype=t.float16, device="cuda") for s in ((M, 2 * N), (M, K), (K, 2 * N))]
    g.gemm_f16_glu_grad(dC.cuda(), X.cuda(), W.cuda(), *out, act)
    sync(t)

    def loss(x, w):
        S = x @ w
        return float((ref.act_both(act, S[:, :N])[0] * S[:, N:] * dC.double()).sum())

    h = 1e-5
    assert float((X.double() @ W.double())[:, :N].abs().min()) > 10 * h   # off relu's corner
    held = out[0].cpu().double().abs()
    terms = (held @ W.double().abs().t(), X.double().abs().t() @ held)
    rng = np.random.default_rng(11)
    for base, got, which in ((X, out[1], 0), (W, out[2], 1)):
        for _ in range(12):
            i, j = (int(rng.integers(n)) for n in base.shape)
            vals = []
            for s in (h, -h):
                x, w = X.double(), W.double()
                (x if which == 0 else w)[i, j] += s
                vals.append(loss(x, w))
            want = (vals[0] - vals[1]) / (2 * h)
            # the rounding of dGU's entries to half, and of the result
            tol = ref.HALF * (float(terms[which][i, j]) + abs(want)) + 1e-6
            assert abs(float(got[i, j]) - want) <= tol


@pytest.mark.parametrize("M,N", [(4, 40), (600, 2504)])
def test_glu_extremes(M, N):
    """Gates far out on both sides, infinite and NaN rows: each row by itself."""
    import dense_gemm_03_gb300 as g
    t = torch()
    K = 16
    X = t.zeros(M, K, dtype=t.float16)
    W = t.zeros(K, 2 * N, dtype=t.float16)
    W[0, :N], W[1, N:] = 1.0, 1.0       # G = X[:, 0], U = X[:, 1]
    gates = [0.0, -0.0, 1.0, -1.0, 9.0, -9.0, 30.0, -30.0, 90.0, -90.0, 6e4, -6e4, 2.0 ** -24]
    for i in range(M):
        X[i, 0], X[i, 1] = gates[i % len(gates)], (-1) ** i * 1.0
    bad = M - 2
    X[bad, 0] = float("nan")
    X[bad + 1, 1] = float("inf")        # U infinite (0 * inf makes G NaN)
    for act in ref.ACTS:
        C = t.empty(M, N, dtype=t.float16, device="cuda")
        gu = t.empty(M, 2 * N, dtype=t.float16, device="cuda")
        one = t.ones(M, N, dtype=t.float16)
        g.gemm_f16_glu(X.cuda(), W.cuda(), C, act)
        g.gemm_f16_glu_grad(one.cuda(), X.cuda(), W.cuda(), gu, act=act)
        sync(t)
        good = slice(0, bad)
        ref.check(C[good].cpu(), *ref.glu(X[good], W, act), act)
        ref.check(gu[good].cpu(), *ref.glu_grad(one[good], X[good], W, act), act)
        assert bool(C[bad:].isnan().all()) and not bool(gu[bad:, :N].isfinite().any())


@pytest.mark.parametrize("M", [5, 700])
def test_glu_past_the_half_range(M):
    """C past 65504 is infinite, with the sign of the product; f(0) U is 0."""
    import dense_gemm_03_gb300 as g
    t = torch()
    N, K = 1504, 32
    X = t.full((M, K), 100.0, dtype=t.float16)
    W = t.full((K, 2 * N), 1.0, dtype=t.float16)
    W[:, N + 1::2] = -1.0
    W[:, 4] = 0.0
    C = t.empty(M, N, dtype=t.float16, device="cuda")
    g.gemm_f16_glu(X.cuda(), W.cuda(), C)
    sync(t)
    want = t.full((M, N), float("inf"))
    want[:, 1::2] = -float("inf")
    want[:, 4] = 0.0
    assert t.equal(C.float().cpu(), want)


def test_glu_blank():
    import dense_gemm_03_gb300 as g
    t = torch()
    new = lambda *s: t.full(s, 2.0, dtype=t.float16, device="cuda")
    C, gu, dX, dW = new(3, 5), new(3, 10), new(3, 4), new(4, 10)
    g.gemm_f16_glu(0, 0, C, M=3, N=5, K=0)
    g.gemm_f16_glu_grad(0, 0, 0, gu, M=3, N=5, K=0)
    g.gemm_f16_glu_grad(0, 0, 0, 0, dX, None, M=3, N=0, K=4)
    g.gemm_f16_glu_grad(0, 0, 0, 0, None, dW, beta=0.5, M=0, N=5, K=4)
    g.gemm_f16_glu(0, 0, 0, M=0, N=5, K=4)
    sync(t)
    assert not bool(C.any()) and not bool(gu.any()) and not bool(dX.any()) and bool((dW == 1).all())


@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (40, 512, 512), (1500, 1368, 400), (4096, 1664, 3200)])
def test_repeats_are_bitwise_equal(M, N, K):
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W, dC = (v.cuda() for v in operands(t, M, N, K))
    def once():
        out = [t.empty(s, dtype=t.float16, device="cuda") for s in ((M, N), (M, 2 * N), (M, K), (K, 2 * N))]
        g.gemm_f16_glu(X, W, out[0])
        g.gemm_f16_glu_grad(dC, X, W, *out[1:])
        return out
    first = once()
    for _ in range(3):
        assert all(t.equal(a, b) for a, b in zip(first, once()))
    sync(t)


@pytest.mark.parametrize("M,N,K", [(4096, 640, 3200), (2304, 1280, 3200)])
def test_long_k_tail(M, N, K):
    """Shapes whose last wave of tiles is cut into K slices (gated, its gradient, dX, dW):
    small integers, compared with the GPU's own 64-bit products."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(5)
    draw = lambda *s: t.randint(-1, 2, s, generator=gen, device="cuda").half()
    X, W, dC = draw(M, K), draw(K, 2 * N), draw(M, N)
    S = X.double() @ W.double()
    G, U = S[:, :N], S[:, N:]
    C, gu = t.empty(M, N, dtype=t.float16, device="cuda"), t.empty(M, 2 * N, dtype=t.float16, device="cuda")
    dX, dW = t.empty(M, K, dtype=t.float16, device="cuda"), t.empty(K, 2 * N, dtype=t.float16, device="cuda")
    g.gemm_f16_glu(X, W, C, "relu")
    assert ".ktail" in g.last_path()
    g.gemm_f16_glu_grad(dC, X, W, gu, dX, dW, "relu")
    sync(t)
    assert t.equal(C, (G.clamp(min=0) * U).half())
    assert t.equal(gu, t.cat([dC.double() * U * (G > 0), dC.double() * G.clamp(min=0)], 1).half())
    # integers: exact in fp32 as long as every partial sum stays below 2^24
    assert float((gu.double().abs() @ W.double().abs().t()).max()) < 2 ** 24
    assert t.equal(dX, (gu.double() @ W.double().t()).half())
    assert t.equal(dW, (X.double().t() @ gu.double()).half())


@pytest.mark.parametrize("f32", [True, False])
def test_sums_over_millions_of_tokens(f32):
    """So many short chunks of K that their count times K's steps passes 32 bits.  Of -1, 0
    and 1 every partial sum is an integer below 2^24: a float result is exact."""
    import dense_gemm_03_gb300 as g
    t = torch()
    K, M, N = 13_000_007, 64, 56
    gen = t.Generator(device="cuda").manual_seed(7)
    A = t.randint(-1, 2, (K, M), generator=gen, device="cuda", dtype=t.int8).half()
    B = t.randint(-1, 2, (K, N), generator=gen, device="cuda", dtype=t.int8).half()
    want = t.zeros(M, N, dtype=t.float64, device="cuda")
    for k in range(0, K, 1 << 20):
        want += (A[k:k + (1 << 20)].double().t() @ B[k:k + (1 << 20)].double())
    C = t.full((M, N), float("nan"), dtype=t.float32 if f32 else t.float16, device="cuda")
    (g.gemm_f16_trans_f32out if f32 else g.gemm_f16_trans)(A, B, C, True, False)
    sync(t)
    # half results: |sums| stay below 2^24, exact in fp32 too, and are rounded once
    assert t.equal(C, want.to(C.dtype))


@pytest.mark.parametrize("off", ["none", "x", "w", "dc", "gu", "dx", "dw", "all"])
@pytest.mark.parametrize("M,N,K", [(300, 1504, 264), (700, 1111, 331)])
def test_glu_grad_with_single_matrices_off_the_grid(M, N, K, off):
    """Every matrix by itself at an odd address and pitch, the others on the 16-byte grid
    (odd widths in rows padded to it); a row with an infinity leaves the others alone."""
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W, dC = operands(t, M, N, K)
    bad = M - 3
    X[bad, 5] = float("inf")
    good = [i for i in range(M) if i != bad]
    nan = lambda *s: t.full(s, float("nan"), dtype=t.float16)
    W0 = normal(t, np.random.default_rng(3), (K, 2 * N))

    def put(name, v):
        if off in (name, "all"):
            return Padded(t, v, 1 + v.shape[1] % 2 * 2, 3)      # odd pitches, odd address
        return Padded(t, v, -v.shape[1] % 8, 0)
    x, w, dc = put("x", X), put("w", W), put("dc", dC)
    gu, dx, dw = put("gu", nan(M, 2 * N)), put("dx", nan(M, K)), put("dw", W0)
    for rows, beta in ((good, 0.0), (None, 0.5)):
        if rows is None:                 # dW of finite rows, added onto what is there
            X[bad, 5] = 1.0
            x.view.copy_(X.cuda())
            rows = range(M)
            dw.view.copy_(W0.cuda())
        g.gemm_f16_glu_grad(dc.ptr, x.ptr, w.ptr, gu.ptr, dx.ptr, dw.ptr, "silu", beta, M=M, N=N, K=K,
                            lddc=dc.ld, ldx=x.ld, ldw=w.ld, lddgu=gu.ld, lddx=dx.ld, lddw=dw.ld)
        sync(t)
        rows = list(rows)
        held = gu.view.cpu()
        ref.check(held[rows], *ref.glu_grad(dC[rows], X[rows], W, "silu"), "dGU")
        ref.check(dx.view.cpu()[rows], *ref.product(held[rows], W.t()), "dX")
        if len(rows) == M:
            ref.check(dw.view.cpu(), *ref.product(X.t(), held, 1.0, beta, W0), "dW")
        else:
            assert not bool(held[bad].isfinite().all()) and not bool(dx.view[bad].isfinite().any())
        assert all(m.untouched(t) for m in (gu, dx, dw))


@pytest.mark.parametrize("M,N", [(8192, 1056), (6000, 1312), (16384, 296)])
@pytest.mark.parametrize("K", [24, 72])
def test_short_sums_and_a_narrow_last_tile(M, N, K):
    """Tiles that follow one another at once, the last of a row of tiles only 32 or 40
    columns wide: what a tile leaves on its way out is not overwritten by the next.
    Small integers, exact throughout."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(9)
    draw = lambda *s: t.randint(-2, 3, s, generator=gen, device="cuda").half()
    A, B, B2, dC = draw(M, K), draw(K, N), draw(K, 2 * N), draw(M, N)
    AT, C, H = A.t().contiguous(), *(t.empty(M, N, dtype=t.float16, device="cuda") for _ in "ch")
    F, gu = t.empty(M, N, device="cuda"), t.empty(M, 2 * N, dtype=t.float16, device="cuda")
    P, S = A.float() @ B.float(), A.float() @ B2.float()
    G, U = S[:, :N], S[:, N:]
    for _ in range(5):
        for o in (C, H, F, gu):
            o.fill_(float("nan"))
        g.gemm_f16(A, B, C)
        assert t.equal(C.float(), P)
        C.fill_(float("nan"))
        g.gemm_f16_trans(AT, B, C, True, False)
        g.gemm_f16_trans_f32out(AT, B, F, True, False)
        g.gemm_f16_glu(A, B2, H, "relu")
        g.gemm_f16_glu_grad(dC, A, B2, gu, act="relu")
        sync(t)
        assert t.equal(C.float(), P) and t.equal(F, P)
        assert t.equal(H, (G.clamp(min=0) * U).half())
        assert t.equal(gu, t.cat([dC.float() * U * (G > 0), dC.float() * G.clamp(min=0)], 1).half())


@pytest.mark.parametrize("M,N,K", [(700, 1368, 4096), (300, 1111, 2049), (64, 1000, 3000)])
def test_relu_gradient_of_long_sums(M, N, K):
    """relu's derivative jumps where G is 0: sums of G as near as sums in fp32 get.  Rounded
    to nearest in runs of 512, G's error is below 2e-6 of its size here (one in 2^24 for
    each of the runs' additions, and the truncation within them), so at most 2 sqrt(2/pi) 2e-6
    of the entries (a normal density about 0) can be on the wrong side: 4 in a million,
    and as many again for the unlucky."""
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W, dC = operands(t, M, N, K)
    gu = t.empty(M, 2 * N, dtype=t.float16, device="cuda")
    g.gemm_f16_glu_grad(dC.cuda(), X.cuda(), W.cuda(), gu, act="relu")
    sync(t)
    want, tol = ref.glu_grad(dC, X, W, "relu")
    off = ((gu.cpu().double() - want).abs() > tol + 1e-5).double().mean()
    assert float(off) <= 8e-6 + 2.0 / (M * N)
