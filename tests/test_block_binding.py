"""What the dense block's calls make of the tensors that they are given.  (Tensors that say
they are in device memory; nothing is launched.)"""
import pytest

import dense_gemm_03_gb300 as g

torch = pytest.importorskip("torch")


class OnDevice:
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)


def matrix(x, rows, cols, ld=None, dtype="float16"):
    return g._matrix(OnDevice(x), rows, cols, ld, dtype, "X")


def test_a_contiguous_tensor_wider_than_its_matrix():
    """The distance of the tensor's rows counts, not the matrix's width."""
    t = torch.zeros(8, 12, dtype=torch.float16)
    wide = torch.zeros(8, 16, dtype=torch.float16)[:, :12]
    for _ in range(2):                                      # (types are looked up, then known)
        assert matrix(t, 8, 12) == (t.data_ptr(), 12)
        assert matrix(t, 8, 10) == (t.data_ptr(), 12)
        assert matrix(t, 8, 5) == (t.data_ptr(), 12)
        assert matrix(t, 5, 12) == (t.data_ptr(), 12)       # its first rows
        assert matrix(t, 1, 5) == (t.data_ptr(), 5)
        assert matrix(wide, 8, 12) == (wide.data_ptr(), 16)


@pytest.mark.parametrize("shape,rows,cols", [
    ((12, 8), 8, 12), ((16, 8), 8, 16), ((4, 24), 8, 12), ((96, 1), 8, 12), ((1, 96), 8, 12),
    ((2, 4, 24), 8, 12), ((2, 3, 12), 8, 12), ((95,), 8, 12), ((), 1, 1)])
def test_tensors_of_another_shape_are_refused(shape, rows, cols):
    with pytest.raises(ValueError, match="not %d x %d" % (rows, cols)):
        matrix(torch.zeros(shape, dtype=torch.float16), rows, cols)


def test_batches_and_flat_buffers():
    for shape in ((2, 4, 12), (8, 1, 12), (96,), (100,)):
        x = torch.zeros(shape, dtype=torch.float16)
        assert matrix(x, 8, 12) == (x.data_ptr(), 12)
    x = torch.zeros(2, 4, 16, dtype=torch.float16)[:, :, :12]
    with pytest.raises(ValueError, match="not 8 x 12"):
        matrix(x, 8, 12)


@pytest.mark.parametrize("given,K,N", [((5, 9), 6, 8), ((6, 9), 6, 9)])
def test_a_weight_of_other_sizes(given, K, N):
    """K or N that the caller gives does not excuse a weight without them."""
    z = lambda *s: torch.zeros(s, dtype=torch.int8)
    with pytest.raises(ValueError):
        g.gemm_i8(16, OnDevice(z(*given)), 16, M=2, N=N + 1, K=K)


def test_results_with_padding_or_transposed(monkeypatch):
    """Every call's result goes with the distance of its rows; transposed ones are refused."""
    seen = {}

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.update({name: a}) or 0

    monkeypatch.setattr(g, "_lib", Lib())
    monkeypatch.setattr(g, "_devices", 1)
    h = lambda *s: OnDevice(torch.zeros(s, dtype=torch.float16))
    q = lambda *s: OnDevice(torch.zeros(s, dtype=torch.int8))
    f = lambda *s: OnDevice(torch.zeros(s))
    g.gemm_f16_glu(h(4, 8), h(8, 12), h(4, 10), stream=0)
    assert seen["gemm_f16_glu"][3:10] == (4, 6, 8, 0, 8, 12, 10)
    g.gemm_f16_glu_grad(h(4, 7), h(4, 8), h(8, 12), h(4, 14), h(4, 9), h(8, 20), stream=0)
    assert seen["gemm_f16_glu_grad"][6:16] == (4, 6, 8, 0, 7, 8, 12, 14, 9, 20)
    g.gemm_f16_trans_f32out(h(8, 4), h(8, 6), f(4, 9), True, stream=0)
    assert seen["gemm_f16_trans_f32out"][5:11] == (4, 6, 8, 4, 6, 9)
    g.gemm_i8(q(4, 8), q(8, 6), h(4, 7), stream=0)
    assert seen["gemm_i8"][5:12] == (4, 6, 8, -1, 8, 6, 7)
    g.f16_to_i8(h(4, 8), q(4, 16), f(4), stream=0)
    assert seen["gemm_f16_to_i8"][3:7] == (4, 8, 8, 16)
    with pytest.raises(ValueError, match="dW is"):
        g.gemm_f16_glu_grad(h(4, 6), h(4, 8), h(8, 12), h(4, 12), None, h(12, 8), stream=0)
    with pytest.raises(ValueError, match="C is"):
        g.gemm_f16_trans(h(8, 4), h(8, 6), h(6, 4), True, stream=0)


def test_scales_of_another_device(monkeypatch):
    """Scales are read on the current device, as the matrices are."""
    monkeypatch.setattr(g, "_devices", 2)       # (get_device() of a CPU tensor is -1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = OnDevice(torch.zeros(8))
    for _ in range(2):
        with pytest.raises(ValueError, match="sx is on device -1"):
            g._scales(x, 8, "sx")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    assert g._scales(x, 8, "sx") == x.data_ptr()


@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32 + 5, -2 ** 32 + 5])
def test_sizes_past_32_bits(monkeypatch, size):
    """They are refused, not cut to their low 32 bits."""
    class Lib:                              # (none of the calls)
        def gemm_strerror(self, code):
            return b""

    monkeypatch.setattr(g, "_lib", Lib())
    for sizes in (dict(M=size, N=8, K=8), dict(M=8, N=size, K=8), dict(M=8, N=8, K=size),
                  dict(M=8, N=8, K=8, ldc=size)):
        for call in (g.gemm_f16_trans, g.gemm_f16_trans_f32out, g.gemm_f16_glu, g.gemm_i8):
            with pytest.raises(g.GemmError) as e:
                call(16, 16, 16, **sizes)
            assert e.value.code == -7
        sizes["lddx"] = sizes.pop("ldc", None)
        with pytest.raises(g.GemmError):
            g.gemm_f16_glu_grad(16, 16, 16, 16, 16, 16, **sizes)
    for sizes in (dict(M=size, K=8), dict(M=8, K=size), dict(M=8, K=8, ldq=size)):
        with pytest.raises(g.GemmError):
            g.f16_to_i8(16, 16, 16, **sizes)


def test_tensors_past_32_bits():
    """(Expanded, so that they take no memory.)"""
    long = torch.zeros(1, 8, dtype=torch.float16).expand(2 ** 32 + 5, 8)
    long.is_contiguous = lambda: True
    with pytest.raises(g.GemmError):
        matrix(long, *long.shape)
    far = torch.zeros(1, dtype=torch.float16).as_strided((1, 8), (2 ** 31, 0))
    assert matrix(far, 1, 1) == (far.data_ptr(), 1)
    far = far.expand(1, 8)

    class Rows(OnDevice):
        shape = (2, 8)

        def stride(self, i):
            return (2 ** 31, 1)[i]

    with pytest.raises(g.GemmError, match="apart"):
        g._matrix(Rows(far), 2, 8, None, "float16", "X")
