"""The adapter products whose result is large enough for CTA pairs (more than a
quarter as many 256 x 256 tiles as SMs), against the 64-bit definition: lists of
more adapters than a warp, several chunks of ranks, odd widths, weights that are
not finite; and gradients over more adapters than one launch has places for."""
import pytest

import routed_ref as ref
from helpers import torch
from test_gpu_lora import dev, operands, sync

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


def forward(o, C, alpha=1.0, beta=0.0, scales=True, **kw):
    import dense_gemm_03_gb300 as g
    g.gemm_f16_lora(o["X"], o["W"], C, o["A"], o["B"], o["ids"], o["scales"] if scales else None,
                    alpha, beta, **kw)
    assert g.last_path().startswith("lora.tiles"), g.last_path()


def gradients(o, dX, dA=None, dB=None, alpha=1.0, beta=0.0, scales=True, **kw):
    import dense_gemm_03_gb300 as g
    g.gemm_f16_lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"],
                         o["scales"] if scales else None, dX, dA, dB, alpha, beta, **kw)
    assert g.last_path().startswith("lora_grad.tiles"), g.last_path()


SHAPES = [
    # M, N, K, R, adapters, ids: C and dX both have at least 45 tiles
    (2300, 1290, 1100, 8, 40, "mixed"),       # N off the 16-byte grid
    (2305, 1296, 1101, 33, 5, "mixed"),       # K and R off it
    (2560, 1152, 1280, 128, 3, "runs"),
    (2300, 1280, 1152, 16, 300, "mixed"),     # over 32 adapters to every block of rows
    (2400, 1288, 1096, 6, 7, "outside"),
    (2304, 1536, 1280, 64, 1, "one"),
    (4100, 648, 776, 24, 9, "runs"),
]


@pytest.mark.parametrize("M,N,K,R,n,order", SHAPES)
def test_forward(M, N, K, R, n, order):
    t = torch()
    o = operands(t, M + N + K, M, N, K, R, n, order)
    v = dev(o)
    for alpha, beta, scales in ((1.0, 0.0, True), (1.5, -0.5, False)):
        C = t.full_like(v["C0"], float("nan")) if beta == 0.0 else v["C0"].clone()
        forward(v, C, alpha, beta, scales)
        sync(t)
        r, tol = ref.lora(o["X"], o["W"], o["C0"], o["A"], o["B"], o["ids"],
                          o["scales"] if scales else None, alpha, beta)
        ref.check(C.cpu(), r, tol)


@pytest.mark.parametrize("M,N,K,R,n,order", SHAPES)
def test_gradients(M, N, K, R, n, order):
    t = torch()
    o = operands(t, M + N + K + 1, M, N, K, R, n, order)
    v = dev(o)
    dX = t.full_like(v["X"], float("nan"))
    dA, dB = v["dA0"].clone(), v["dB0"].clone()
    gradients(v, dX, dA, dB, 0.5, 1.0)
    alone = t.full_like(v["X"], float("nan"))
    gradients(v, alone, alpha=0.5)
    sync(t)
    r = ref.lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"], 0.5, 1.0,
                      o["dA0"], o["dB0"])
    for name, got in (("dX", dX), ("dA", dA), ("dB", dB)):
        ref.check(got.cpu(), *r[name], what=name)
    assert t.equal(dX, alone)


@pytest.mark.parametrize("M,N,K,R,n,order", SHAPES)
def test_integers_exact(M, N, K, R, n, order):
    """Small integers: every sum before the result's rounding is exact."""
    t = torch()
    o = operands(t, M * N + K, M, N, K, R, n, order, integers=True)
    o["G"] = o["C0"]
    v = dev(o)
    C, dX = v["C0"].clone(), t.empty_like(v["X"])
    dA, dB = v["dA0"].clone(), v["dB0"].clone()
    forward(v, C, 2.0, -1.0)
    gradients(v, dX, dA, dB, 2.0, 1.0)
    sync(t)
    r, _ = ref.lora(o["X"], o["W"], o["C0"], o["A"], o["B"], o["ids"], o["scales"], 2.0, -1.0)
    assert t.equal(C.cpu(), r.half())
    r = ref.lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"], 2.0, 1.0,
                      o["dA0"], o["dB0"])
    assert t.equal(dX.cpu(), r["dX"][0].half())
    assert t.equal(dA.cpu(), r["dA"][0].float()) and t.equal(dB.cpu(), r["dB"][0].float())


@pytest.mark.parametrize("R,n", [(16, 6), (40, 45)])
def test_what_is_not_finite_stays_with_its_rows(R, n):
    """Adapters holding Inf and NaN (in a first, a middle and a last rank), and
    rows of X and dC that do: every other row keeps its bits."""
    t = torch()
    M, N, K = 2300, 1296, 1104
    o = operands(t, 61, M, N, K, R, n, "mixed")
    o["ids"][o["ids"] == 5] = 0
    o["ids"][77], o["ids"][78] = 0, 4
    clean = dev({k: x.clone() for k, x in o.items()})
    o["A"][2, 3, R - 1] = float("inf")
    o["A"][1, K - 1, 0] = float("nan")
    o["B"][3, R // 2, N - 1] = float("nan")
    o["B"][1, 0, 0] = float("-inf")
    o["A"][5], o["B"][5] = float("nan"), float("inf")    # of no row
    o["X"][77, 5] = float("inf")
    o["G"][78, 9] = float("nan")
    dirty = dev(o)
    outs = []
    for x in (clean, dirty):
        C, dX = t.empty_like(x["C0"]), t.empty_like(x["X"])
        forward(x, C)
        gradients(x, dX)
        sync(t)
        outs.append((C.cpu(), dX.cpu()))
    (C, dX), (C2, dX2) = outs
    good = (o["ids"] != 1) & (o["ids"] != 2) & (o["ids"] != 3)
    good[77] = good[78] = False
    assert t.equal(C[good], C2[good]) and t.equal(dX[good], dX2[good])
    assert not t.isfinite(C2[77]).any() and not t.isfinite(dX2[78]).any()
    # the adapters' own rows: finite where the formula is
    r, tol = ref.lora(o["X"], o["W"], None, o["A"], o["B"], o["ids"], o["scales"], 1.0, 0.0)
    for a in (1, 2, 3):
        rows = o["ids"] == a
        fin = r[rows].isfinite()
        assert t.equal(C2[rows].isfinite(), fin)
        ref.check(C2[rows][fin], r[rows][fin], tol[rows][fin])
    assert (C2[o["ids"] == 3][:, : N - 1]).isfinite().all()


@pytest.mark.parametrize("pad", [8, 3])
def test_leading_dimensions_and_beta(pad):
    t = torch()
    M, N, K, R, n = 2300, 1288, 1104, 12, 4
    o = operands(t, 62 + pad, M, N, K, R, n, "mixed")

    def wide(x):
        w = t.full(x.shape[:-1] + (x.shape[-1] + pad,), float("nan"), dtype=x.dtype, device="cuda")
        w[..., :x.shape[-1]] = x.cuda()
        return w

    v = {k: wide(o[k]) for k in ("X", "W", "A", "B", "G")}
    v["ids"], v["scales"] = o["ids"].cuda(), o["scales"].cuda()
    C = wide(o["C0"])
    dX = t.full((M, K + pad), float("nan"), dtype=t.float16, device="cuda")
    size = dict(M=M, N=N, K=K, R=R, adapters=n, ldx=K + pad, ldw=N + pad, lda=R + pad, ldb=N + pad)
    forward(v, C, 1.0, 0.5, ldc=N + pad, **size)
    gradients(v, dX, lddc=N + pad, lddx=K + pad, **size)
    sync(t)
    assert C[:, N:].isnan().all() and dX[:, K:].isnan().all()
    ref.check(C[:, :N].cpu(), *ref.lora(o["X"], o["W"], o["C0"], o["A"], o["B"], o["ids"],
                                        o["scales"], 1.0, 0.5))
    r = ref.lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"], 1.0, 0.0, None,
                      None)
    ref.check(dX[:, :K].cpu(), *r["dX"])


def test_repeats_streams_and_graphs():
    t = torch()
    o = dev(operands(t, 63, 2500, 1290, 1032, 24, 70, "mixed"))
    t.cuda.synchronize()

    def outs():
        return [t.full_like(o[k], float("nan")) for k in ("C0", "X", "dA0", "dB0")]

    def call(x):
        forward(o, x[0])
        gradients(o, *x[1:])

    first, second, third = outs(), outs(), outs()
    call(first)
    t.cuda.synchronize()
    s = t.cuda.Stream()
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(s):
        call(second)
        call(third)
        s.synchronize()
        with t.cuda.graph(graph, stream=s):
            call(third)
    for _ in range(3):
        for x in third:
            x.fill_(float("nan"))
        graph.replay()
    sync(t)
    for a, b, c in zip(first, second, third):
        assert t.equal(a, b) and t.equal(a, c)


@pytest.mark.parametrize("M,N,K,R,n", [(2100, 72, 64, 4, 5000), (1600, 64, 136, 16, 8000)])
def test_gradients_of_more_adapters_than_a_launch_has_places_for(M, N, K, R, n):
    """Several launches over the rows, each adding to the one before."""
    import dense_gemm_03_gb300 as g
    t = torch()
    o = operands(t, 64 + n, M, N, K, R, n, "mixed")
    o["ids"][::3] = n // 2                       # an adapter with rows in every launch
    v = dev(o)
    dA, dB = v["dA0"].clone(), v["dB0"].clone()
    g.gemm_f16_lora_grad(v["G"], v["X"], v["W"], v["A"], v["B"], v["ids"], v["scales"], None, dA, dB,
                         0.5, -1.0)
    sync(t)
    r = ref.lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"], 0.5, -1.0,
                      o["dA0"], o["dB0"])
    ref.check(dA.cpu(), *r["dA"])
    ref.check(dB.cpu(), *r["dB"])


@pytest.mark.parametrize("M,N,K,R,n", [(100, 256, 4096, 128, 3), (128, 520, 2056, 64, 128)])
def test_few_rows_of_a_large_rank(M, N, K, R, n):
    import dense_gemm_03_gb300 as g
    t = torch()
    o = operands(t, M + R, M, N, K, R, n, "mixed")
    v = dev(o)
    C = t.full_like(v["C0"], float("nan"))
    g.gemm_f16_lora(v["X"], v["W"], C, v["A"], v["B"], v["ids"], v["scales"])
    sync(t)
    ref.check(C.cpu(), *ref.lora(o["X"], o["W"], None, o["A"], o["B"], o["ids"], o["scales"], 1.0,
                                 0.0), what=g.last_path())
