"""Argument checks of the dense block's entry points: no GPU is touched."""
import pytest

import dense_gemm_03_gb300 as g

BIG = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    from dense_gemm_03_gb300 import build
    build.build()
    return g.lib()


@pytest.mark.parametrize("name", ["gemm_f16_trans", "gemm_f16_trans_f32out"])
def test_trans_refusals(L, name):
    f = getattr(L, name)
    def call(ta, tb, M, N, K, lda, ldb, ldc, A=16, B=16, C=16):
        return f(ta, tb, A, B, C, M, N, K, lda, ldb, ldc, 1.0, 0.0, None)
    assert call(1, 0, -1, 4, 4, 4, 4, 4) == -2
    assert call(1, 0, 4, 4, -1, 4, 4, 4) == -2
    assert call(2, 0, 4, 4, 4, 4, 4, 4) == -7
    assert call(0, -1, 4, 4, 4, 4, 4, 4) == -7
    assert call(1, 0, 8, 4, 4, 7, 4, 4) == -3      # A is K x M
    assert call(0, 1, 4, 4, 8, 8, 7, 4) == -3      # B is N x K
    assert call(1, 1, 4, 4, 8, 4, 7, 4) == -3
    assert call(1, 0, 4, 4, 4, 4, 4, 3) == -3
    assert call(0, 0, 4, 4, 4, 3, 4, 4) == -3      # as gemm_f16_ld
    assert call(1, 0, 4, 4, 4, 4, 4, 4, A=None) == -1
    assert call(1, 0, 4, 4, 4, 4, 4, 4, C=None) == -1
    assert call(1, 0, 4, 4, 4, 4, 4, 4, A=17) == -7
    assert call(1, 0, 4, 4, 4, 4, 4, 4, C=17) == -7
    assert call(1, 0, 0, 4, 4, 0, 4, 4, A=None, B=None, C=None) == 0
    assert call(1, 0, 4, 0, 4, 4, 0, 0, A=None, B=None, C=None) == 0


def test_glu_refusals(L):
    def call(M, N, K, act=0, ldx=8, ldw=16, ldc=8, X=16, W=16, C=16):
        return L.gemm_f16_glu(X, W, C, M, N, K, act, ldx, ldw, ldc, None)
    assert call(-1, 8, 8) == -2 and call(8, -8, 8) == -2 and call(8, 8, -8) == -2
    assert call(8, 8, 8, act=-1) == -7 and call(8, 8, 8, act=4) == -7
    assert call(8, (1 << 29) + 1, 8, ldw=BIG, ldc=BIG) == -7
    assert call(8, 8, 8, ldx=7) == -3 and call(8, 8, 8, ldw=15) == -3 and call(8, 8, 8, ldc=7) == -3
    for missing in ("X", "W", "C"):
        assert call(8, 8, 8, **{missing: None}) == -1
        assert call(8, 8, 8, **{missing: 17}) == -7
    assert call(8, 8, 0, C=None) == -1
    assert call(0, 8, 8, X=None, W=None, C=None) == 0


def test_glu_grad_refusals(L):
    ok = dict(dC=16, X=16, W=16, dGU=16, dX=16, dW=16, M=8, N=8, K=8, act=0, lddc=8, ldx=8, ldw=16,
              lddgu=16, lddx=8, lddw=16, beta=0.0)
    def call(**k):
        return L.gemm_f16_glu_grad(*{**ok, **k}.values(), None)
    for name in ("M", "N", "K"):
        assert call(**{name: -1}) == -2
    assert call(act=-1) == -7 and call(act=4) == -7 and call(N=(1 << 29) + 1) == -7
    for name in ("lddc", "ldx", "ldw", "lddgu", "lddx", "lddw"):
        assert call(**{name: ok[name] - 1}) == -3
    for name in ("dC", "X", "W", "dGU"):
        assert call(**{name: None}) == -1
    for name in ("dC", "X", "W", "dGU", "dX", "dW"):
        assert call(**{name: 17}) == -7
    assert call(dGU=None, dX=None, dW=None) == -1
    # not wanted: their leading dimensions are not looked at
    assert call(dX=None, dW=None, lddx=0, lddw=0, dC=17) == -7
    assert call(M=0, dC=None, X=None, W=None, dGU=None, dX=None, dW=None) == 0
    assert call(M=0, dW=None, dC=None, X=None, W=None, dGU=None) == 0


def test_binding_shapes(L):
    torch = pytest.importorskip("torch")
    z = lambda *s: torch.zeros(*s, dtype=torch.float16)
    with pytest.raises(ValueError, match="K of W and X"):
        g.gemm_f16_glu(z(2, 8), z(9, 8), z(2, 4))
    with pytest.raises(ValueError, match="columns"):
        g.gemm_f16_glu(z(2, 8), z(8, 7), z(2, 4))
    with pytest.raises(ValueError, match="activation"):
        g.gemm_f16_glu(z(2, 8), z(8, 8), z(2, 4), "tanh")
    with pytest.raises(ValueError, match="K of W and X"):
        g.gemm_f16_glu_grad(z(2, 4), z(2, 8), z(9, 8), z(2, 8))
    with pytest.raises(ValueError, match="K of B and A"):
        g.gemm_f16_trans(z(8, 2), z(9, 4), z(2, 4), True)
    with pytest.raises(g.GemmError):
        g.gemm_f16_glu(16, 16, 16, M=-1, N=1, K=1)


def test_i8_refusals(L):
    def call(M, N, K, act=-1, ldx=8, ldw=16, ldc=8, beta=0.0, X=1, W=1, C=16, sx=None, sw=None):
        return L.gemm_i8(X, W, C, sx, sw, M, N, K, act, ldx, ldw, ldc, beta, None)
    assert call(-1, 8, 8) == -2 and call(8, -8, 8) == -2 and call(8, 8, -8) == -2
    assert call(8, 8, 8, act=-2) == -7 and call(8, 8, 8, act=4) == -7
    assert call(8, 8, 8, act=0, beta=0.5) == -7
    assert call(8, (1 << 29) + 1, 8, act=0, ldw=BIG, ldc=BIG) == -7
    assert call(8, 8, 8, ldx=7) == -3 and call(8, 8, 8, ldw=7) == -3 and call(8, 8, 8, ldc=7) == -3
    assert call(8, 8, 8, act=0, ldw=15) == -3
    for missing in ("X", "W", "C"):
        assert call(8, 8, 8, **{missing: None}) == -1
    assert call(8, 8, 8, C=17) == -7 and call(8, 8, 8, sx=6) == -7 and call(8, 8, 8, sw=6) == -7
    assert call(0, 8, 8, X=None, W=None, C=None) == 0


def test_to_i8_refusals(L):
    def call(M, K, ldx=8, ldq=8, X=16, Q=1, scales=16):
        return L.gemm_f16_to_i8(X, Q, scales, M, K, ldx, ldq, None)
    assert call(-1, 8) == -2 and call(8, -1) == -2
    assert call(8, 8, ldx=7) == -3 and call(8, 8, ldq=7) == -3
    for missing in ("X", "Q", "scales"):
        assert call(8, 8, **{missing: None}) == -1
    assert call(8, 0, scales=None) == -1
    assert call(8, 8, X=17) == -7 and call(8, 8, scales=18) == -7
    assert call(0, 8, X=None, Q=None, scales=None) == 0


def test_matrix_of_the_binding():
    """Addresses and leading dimensions of what the calls are given.  (A tensor that says
    it is in device memory; nothing is launched.)"""
    torch = pytest.importorskip("torch")

    class OnDevice:
        is_cuda = True

        def __init__(self, t):
            self.t = t

        def __getattr__(self, name):
            return getattr(self.t, name)

    t = torch.zeros(8, 12, dtype=torch.float16)
    m = lambda x, rows, cols, ld=None: g._matrix(OnDevice(x), rows, cols, ld, "float16", "X")
    assert m(t, 8, 12) == (t.data_ptr(), 12)
    assert m(t[2:6, 4:], 4, 8) == (t[2:, 4:].data_ptr(), 12)      # rows of a larger matrix
    assert m(t[:, :5], 3, 5, 24) == (t.data_ptr(), 24)            # a given one counts
    assert m(t[3:4, :7], 1, 7) == (t[3:].data_ptr(), 7)
    assert g._matrix(4096, 8, 12, None, "float16", "X") == (4096, 12)
    assert g._matrix(None, 8, 12, None, "float16", "X") == (None, 12)
    for bad in (t.t(), t[:, ::2], t[::2].t()):
        with pytest.raises(ValueError, match="not dense"):
            m(bad, *bad.shape)
    seen = g._devices
    try:
        g._devices = 2          # as if there were another: get_device() of a CPU tensor is -1
        with pytest.MonkeyPatch.context() as patch:
            patch.setattr(torch.cuda, "current_device", lambda: 0)
            for x in (t, t[:, :5]):
                with pytest.raises(ValueError, match="on device -1"):
                    m(x, 2, 5)
    finally:
        g._devices = seen
    with pytest.raises(ValueError, match="not 9 x 12"):
        m(t, 9, 12)
    with pytest.raises(ValueError, match="not 8 x 13"):
        m(t, 8, 13)
    with pytest.raises(TypeError, match="X is bfloat16"):
        m(t.bfloat16(), 8, 12)
    with pytest.raises(ValueError, match="device memory"):
        g._matrix(t, 8, 12, None, "float16", "X")
    with pytest.raises(ValueError, match="device memory"):
        g._matrix(t.numpy(), 8, 12, None, "float16", "X")


def test_i8_binding(L):
    torch = pytest.importorskip("torch")
    q = lambda *s: torch.zeros(*s, dtype=torch.int8)
    c = torch.zeros(2, 4, dtype=torch.float16)
    with pytest.raises(TypeError, match="X is float16"):
        g.gemm_i8(c, q(4, 4), c)
    with pytest.raises(ValueError, match="X is not in device memory"):
        g.gemm_i8(q(2, 4), q(4, 4), c)
    with pytest.raises(TypeError, match="W is uint8"):
        g.gemm_i8(16, torch.zeros(4, 4, dtype=torch.uint8), 16, M=2, K=4)
    with pytest.raises(TypeError, match="sx is float16"):
        g.gemm_i8(16, 16, 16, torch.zeros(2, dtype=torch.float16), M=2, N=4, K=4)
    with pytest.raises(ValueError, match="sw is not in device memory"):
        g.gemm_i8(16, 16, 16, None, torch.zeros(8), "silu", M=2, N=4, K=4)
    with pytest.raises(ValueError, match="K of W and X"):
        g.gemm_i8(q(2, 4), q(5, 4), c)
    with pytest.raises(ValueError, match="columns"):
        g.gemm_i8(q(2, 4), q(4, 7), c, act="relu")
    with pytest.raises(TypeError, match="Q is float16"):
        g.f16_to_i8(16, c, 16, M=2, K=4)
    with pytest.raises(ValueError, match="scales is not in device memory"):
        g.f16_to_i8(16, 16, torch.zeros(1), M=2, K=4)


def test_sizes_near_the_largest_int(L):
    for M, N, K in ((BIG, 8, 8), (8, BIG, 8), (8, 8, BIG)):
        assert L.gemm_f16_trans(1, 0, 16, 16, 16, M, N, K, BIG, BIG, BIG, 1.0, 0.0, None) == -7
        assert L.gemm_f16_glu(16, 16, 16, M, N, K, 0, BIG, BIG, BIG, None) == -7
        assert L.gemm_f16_glu_grad(16, 16, 16, 16, 16, 16, M, N, K, 0, BIG, BIG, BIG, BIG, BIG, BIG,
                                   0.0, None) == -7
        assert L.gemm_i8(16, 16, 16, None, None, M, N, K, -1, BIG, BIG, BIG, 0.0, None) == -7
    assert L.gemm_f16_to_i8(16, 16, 16, BIG, 8, BIG, BIG, None) == -7
    assert L.gemm_f16_to_i8(16, 16, 16, 8, BIG, BIG, BIG, None) == -7
