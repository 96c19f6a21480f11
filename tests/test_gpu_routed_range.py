"""The range of the row-routed products' intermediates: V, U and the gated rows
past the half range and far below it, adapters of very different magnitude side
by side, and infinities, which come out as the formula gives them.

u = 2^-24 as in routed_ref.  V and U on CTA pairs are kept to 2^-22 of themselves
or 2^-25 where that is below the result's own rounding, else to 2^-14 of the
largest entry of their row; in the sums of dA and dB, and the gated rows of the
experts, to 2^-22 of themselves or 2^-37 of the largest entry that shares their
scale (two halves whose sum is scaled so that the largest lies in [2^13, 2^14):
steps of 2^-24)."""
import pytest

import routed_ref as ref
from helpers import torch
from test_gpu_lora import dev, operands, sync
from test_gpu_moe import operands as moe_operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


def same_where_not_finite(got, want, what=""):
    """got has want's infinities and NaN, and is finite elsewhere."""
    t = torch()
    got, want = got.double(), want.double()
    fin = want.isfinite()
    assert t.equal(got.isfinite(), fin), "%s: finite in other places" % what
    assert t.equal(got[~fin].nan_to_num(0.0, 1.0, -1.0), want[~fin].nan_to_num(0.0, 1.0, -1.0)), what


# tiles, chunks with V by the shrink, chunks with V by rows
LORA_SIZES = [(2300, 1288, 1100, "tiles"), (1300, 264, 320, "stream"), (300, 264, 320, "stream"),
              (40, 264, 320, "stream")]


@pytest.mark.parametrize("M,N,K,path", LORA_SIZES)
@pytest.mark.parametrize("R", [6, 33, 64])
def test_ranks_past_the_last_stay_zero(M, N, K, path, R):
    """A row of X with an infinity, all weights positive: every output of the row
    is +Inf, whatever the rank is padded to."""
    import dense_gemm_03_gb300 as g
    t = torch()
    o = operands(t, M + R, M, N, K, R, 3, "mixed")
    o["ids"][[3, 17]] = 1
    for k in "WAB":
        o[k] = o[k].abs() + 2.0 ** -10
    o["X"][3, 7], o["G"][17, 5] = float("inf"), float("inf")
    v = dev(o)
    C, dX = t.empty_like(v["C0"]), t.empty_like(v["X"])
    g.gemm_f16_lora(v["X"], v["W"], C, v["A"], v["B"], v["ids"], v["scales"])
    assert path in g.last_path()
    g.gemm_f16_lora_grad(v["G"], v["X"], v["W"], v["A"], v["B"], v["ids"], v["scales"], dX)
    assert path in g.last_path()
    sync(t)
    assert (C[3] == float("inf")).all() and (dX[17] == float("inf")).all()
    C[3], dX[17] = 0.0, 0.0
    assert C.isfinite().all() and dX.isfinite().all()


@pytest.mark.parametrize("M,N,K,n", [(2300, 1288, 1096, 4), (300, 264, 320, 4), (49, 333, 777, 29)])
def test_infinite_entries_in_gradients(M, N, K, n):
    """An infinity in a row of X or of dC: dA and dB are infinite or NaN where
    the formula is (a part of U or V that is zero must not make it NaN)."""
    import dense_gemm_03_gb300 as g
    t = torch()
    o = operands(t, M + N, M, N, K, 16, n, "mixed")
    o["ids"][[3, 17]] = t.tensor([1, 2], dtype=t.int32)
    o["X"][3, 7], o["G"][17, 5] = float("inf"), float("-inf")
    v = dev(o)
    dA, dB = t.empty_like(v["dA0"]), t.empty_like(v["dB0"])
    g.gemm_f16_lora_grad(v["G"], v["X"], v["W"], v["A"], v["B"], v["ids"], v["scales"], None, dA, dB)
    sync(t)
    r = ref.lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"], 1.0, 0.0,
                      o["dA0"], o["dB0"])
    for name, got in (("dA", dA), ("dB", dB)):
        want, tol = r[name]
        same_where_not_finite(got.cpu(), want, name)
        fin = want.isfinite()
        ref.check(got.cpu()[fin], want[fin], tol[fin], name)


@pytest.mark.parametrize("M,N,K,n", [(2300, 1288, 1096, 4), (1100, 264, 320, 6), (300, 264, 320, 4),
                                     (49, 333, 777, 29)])
def test_adapters_of_different_magnitude(M, N, K, n):
    """Neighbouring rows whose adapters' scales are 2^-60 to 2^60: each adapter's
    gradients within its own bound."""
    import dense_gemm_03_gb300 as g
    t = torch()
    o = operands(t, M + 3 * N, M, N, K, 16, n, "mixed")
    o["scales"] = t.tensor([2.0 ** (-60 + 120 * i / (n - 1)) for i in range(n)])
    v = dev(o)
    dA, dB = t.empty_like(v["dA0"]), t.empty_like(v["dB0"])
    g.gemm_f16_lora_grad(v["G"], v["X"], v["W"], v["A"], v["B"], v["ids"], v["scales"], None, dA, dB)
    sync(t)
    r = ref.lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"], 1.0, 0.0,
                      o["dA0"], o["dB0"])
    ref.check(dA.cpu(), *r["dA"], what="dA")
    ref.check(dB.cpu(), *r["dB"], what="dB")


@pytest.mark.parametrize("exponent", [-120, -40, 100])
def test_gradients_of_any_magnitude(exponent):
    """U and V from 2^-120 to 2^100 (fp32's range, not half's)."""
    import dense_gemm_03_gb300 as g
    t = torch()
    o = operands(t, 300 + exponent, 300, 264, 320, 16, 4, "mixed")
    o["scales"] = t.full((4,), 2.0 ** exponent)
    v = dev(o)
    dA, dB = t.empty_like(v["dA0"]), t.empty_like(v["dB0"])
    g.gemm_f16_lora_grad(v["G"], v["X"], v["W"], v["A"], v["B"], v["ids"], v["scales"], None, dA, dB)
    sync(t)
    r = ref.lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"], 1.0, 0.0,
                      o["dA0"], o["dB0"])
    # (below 2^-126 the results are denormal: one of their steps more)
    ref.check(dA.cpu(), r["dA"][0], r["dA"][1] + 2.0 ** -149)
    ref.check(dB.cpu(), r["dB"][0], r["dB"][1] + 2.0 ** -149)


def kept(V, F):
    """The bound on V F of V's representation: 2^-22 of itself, or 2^-14 of its
    row's largest entry below the half's normal steps (2^-25)."""
    top = V.abs().amax(1, keepdim=True)
    return (2.0 ** -22 * V.abs() + (2.0 ** -14 * top).clamp(max=2.0 ** -25)) @ F.abs()


@pytest.mark.parametrize("M,N,K,path", LORA_SIZES)
@pytest.mark.parametrize("up", [20, 9, 0, -8, -12, -16, -20])
def test_forward_range(M, N, K, path, up):
    """V about 2^up, B about 2^-up, so that V B is about 1; every other column has
    nothing else."""
    import dense_gemm_03_gb300 as g
    t = torch()
    R, n = 12, 3
    o = operands(t, M + up, M, N, K, R, n, "mixed")
    o["W"][:, ::2] = 0
    o["scales"] = t.full((n,), 2.0 ** up)
    o["B"] = (o["B"].float() * 2.0 ** min(-up, 14)).half()
    v = dev(o)
    C = t.empty_like(v["C0"])
    g.gemm_f16_lora(v["X"], v["W"], C, v["A"], v["B"], v["ids"], v["scales"])
    assert path in g.last_path()
    sync(t)
    r, tol = ref.lora(o["X"], o["W"], None, o["A"], o["B"], o["ids"], o["scales"], 1.0, 0.0)
    for a in range(n):
        rows = o["ids"] == a
        tol[rows] += kept(2.0 ** up * o["X"][rows].double() @ o["A"][a].double(), o["B"][a].double())
    ref.check(C.cpu(), r, tol)


@pytest.mark.parametrize("M,N,K,path", LORA_SIZES)
@pytest.mark.parametrize("up,down", [(14, -13), (12, -12), (0, 0), (-13, 13), (-18, 18)])
def test_dx_range(M, N, K, path, up, down):
    """dC about 2^up with alpha 2^down: loss scaling, and its contrary; every other
    column of dX has the adapters' part alone."""
    import dense_gemm_03_gb300 as g
    t = torch()
    R, n = 16, 3
    o = operands(t, M + up, M, N, K, R, n, "mixed")
    o["W"][::2] = 0
    o["G"] = (o["G"].float().clamp(-0.35, 0.35) * 10 * 2.0 ** up).half()   # below 65504
    o["B"] = o["B"] * 4
    v = dev(o)
    dX = t.empty_like(v["X"])
    g.gemm_f16_lora_grad(v["G"], v["X"], v["W"], v["A"], v["B"], v["ids"], v["scales"], dX,
                         alpha=2.0 ** down)
    assert path in g.last_path()
    sync(t)
    r, tol = ref.lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"],
                           2.0 ** down, 0.0, None, None)["dX"]
    for a in range(n):
        rows = o["ids"] == a
        U = float(o["scales"][a]) * o["G"][rows].double() @ o["B"][a].double().t()
        tol[rows] += 2.0 ** down * kept(U, o["A"][a].double().t())
    ref.check(dX.cpu(), r, tol)


@pytest.mark.parametrize("M,N,K,path", LORA_SIZES)
@pytest.mark.parametrize("up", [-11, -16, -22])
def test_small_gradients_without_scaling(M, N, K, path, up):
    """dC about 2^up with alpha 1 and weights of the usual size: what U is kept to,
    2^-25, is below the result's own rounding (2^-25 as well, where it is small)."""
    import dense_gemm_03_gb300 as g
    t = torch()
    R, n = 16, 3
    o = operands(t, M - up, M, N, K, R, n, "mixed")
    o["G"] = (o["G"].float() * 10 * 2.0 ** up).half()
    o["G"][5, 3] = float("inf")                       # in a row of small entries
    o["W"][::2] = 0
    v = dev(o)
    dX = t.empty_like(v["X"])
    g.gemm_f16_lora_grad(v["G"], v["X"], v["W"], v["A"], v["B"], v["ids"], v["scales"], dX)
    assert path in g.last_path()
    sync(t)
    r, tol = ref.lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"], o["scales"], 1.0, 0.0,
                           None, None)["dX"]
    for a in range(n):
        rows = o["ids"] == a
        tol[rows] += 2.0 ** -25 * o["A"][a].double().abs().sum(1)
    rows = t.arange(M) != 5
    ref.check(dX.cpu()[rows], r[rows], tol[rows])
    assert not dX[5].isfinite().any() or int(o["ids"][5]) < 0


def test_rows_of_either_range_side_by_side():
    """In one tile: rows past the half range, far below it and between, with an
    adapter that is not finite among them."""
    import dense_gemm_03_gb300 as g
    t = torch()
    M, N, K, R, n = 2300, 1288, 1096, 40, 5
    o = operands(t, 71, M, N, K, R, n, "mixed")
    up = [18, 0, -12, -20, 0]
    o["scales"] = t.tensor([2.0 ** e for e in up])
    for a in range(n):
        o["B"][a] = (o["B"][a].float() * 2.0 ** min(-up[a], 14)).half()
    o["B"][4, 3, 5] = float("inf")
    v = dev(o)
    C, dX = t.empty_like(v["C0"]), t.empty_like(v["X"])
    g.gemm_f16_lora(v["X"], v["W"], C, v["A"], v["B"], v["ids"], v["scales"], 1.0, 0.0)
    sync(t)
    r, tol = ref.lora(o["X"], o["W"], None, o["A"], o["B"], o["ids"], o["scales"], 1.0, 0.0)
    for a in range(n):
        rows = o["ids"] == a
        tol[rows] += kept(2.0 ** up[a] * o["X"][rows].double() @ o["A"][a].double(),
                          o["B"][a].double()).nan_to_num(0.0)
    same_where_not_finite(C.cpu(), r)
    fin = r.isfinite()
    ref.check(C.cpu()[fin], r[fin], tol[fin])


def moe_exact(o, topk):
    """(Y, tol) of the renormalised layer with the gated rows kept to 2^-22 of
    themselves or 2^-37 of a row's largest."""
    t = torch()
    X, Wr = o["X"].double(), o["Wr"].double()
    T, H = X.shape
    I = o["W2"].shape[1]
    l = X @ Wr
    dl = ((H + 8) * ref.U2 * (X.abs() @ Wr.abs())).amax(1)
    ids = t.sort(l, dim=1, descending=True, stable=True).indices[:, :topk]
    p = t.gather(t.softmax(l, dim=1), 1, ids)
    p = p / p.sum(1, keepdim=True)
    Y, tol = t.zeros(T, H, dtype=t.float64), t.zeros(T, H, dtype=t.float64)
    for i in range(T):
        for k in range(topk):
            w1, w2 = o["W1"][ids[i, k]].double(), o["W2"][ids[i, k]].double()
            gu, terms = X[i] @ w1, X[i].abs() @ w1.abs()
            g, u = gu[:I], gu[I:]
            e = (H + 8) * ref.U2 * terms
            s = g * t.sigmoid(g)
            h = s * u
            eh = 1.1 * e[:I] * (u.abs() + e[I:]) + s.abs() * e[I:] + 2.0 ** -20 * h.abs()
            eh = eh + 2.0 ** -22 * h.abs() + 2.0 ** -37 * h.abs().max()
            ep = p[i, k] * (4 * dl[i] + 2.0 ** -20 + Wr.shape[1] * ref.U2)
            Y[i] += p[i, k] * (h @ w2)
            th = h.abs() @ w2.abs()
            tol[i] += p[i, k] * (eh @ w2.abs() + (I + topk + 8) * ref.U2 * th) + ep * th
    return ids, Y, tol + ref.HALF * Y.abs() + ref.TINY


@pytest.mark.parametrize("T,H,I,E,topk", [(1, 512, 256, 16, 4), (5, 512, 256, 8, 2),
                                          (40, 264, 712, 3, 2), (64, 256, 192, 1, 1),
                                          (6, 257, 129, 8, 2)])
@pytest.mark.parametrize("up", [9, 4, 0, -7, -12])
def test_moe_range(T, H, I, E, topk, up):
    """Gate and up of about 2^up: gated rows from 2^-25 to 2^18, tokens of
    different magnitude side by side; W2 makes the result about 1."""
    import dense_gemm_03_gb300 as g
    t = torch()
    o = moe_operands(t, T + H + up, T, H, I, E)
    o["Wr"] = t.zeros_like(o["Wr"])
    o["Wr"][0] = t.arange(E, 0, -1).half()            # a choice no rounding changes
    o["X"] = (o["X"].float() * t.tensor([1.0, 0.25, 1.0, 0.0625])[t.arange(T) % 4, None]).half()
    o["X"][:, 0] = 1.0
    o["W1"][:, 0] = 0
    o["W1"] = (o["W1"].float() * 2.0 ** up).half()
    o["W2"] = (o["W2"].float() * 2.0 ** max(min(-2 * up, 14), -10)).half()
    v = {k: x.cuda() for k, x in o.items()}
    Y, ids = t.empty_like(v["Y0"]), t.empty((T, topk), dtype=t.int32, device="cuda")
    g.gemm_f16_moe(v["X"], v["Wr"], v["W1"], v["W2"], Y, topk, ids=ids)
    sync(t)
    want_ids, want, tol = moe_exact(o, topk)
    assert t.equal(ids.cpu().long(), want_ids)
    ref.check(Y.cpu(), want, tol, g.last_path())


@pytest.mark.parametrize("H,I", [(256, 192), (257, 129)])
def test_moe_infinite_weights(H, I):
    """Infinities in W2: the tokens of that expert are infinite or NaN where the
    formula is."""
    import dense_gemm_03_gb300 as g
    t = torch()
    T, E, topk = 9, 4, 2
    o = moe_operands(t, 81, T, H, I, E)
    o["W2"][1, 5, 7], o["W2"][2, I - 1, H - 1] = float("inf"), float("-inf")
    v = {k: x.cuda() for k, x in o.items()}
    Y = t.empty_like(v["Y0"])
    g.gemm_f16_moe(v["X"], v["Wr"], v["W1"], v["W2"], Y, topk)
    sync(t)
    _, want, tol = moe_exact(o, topk)
    same_where_not_finite(Y.cpu(), want)
    fin = want.isfinite()
    ref.check(Y.cpu()[fin], want[fin], tol[fin])


@pytest.mark.parametrize("T,H,I,E", [(24, 2560, 1408, 16), (40, 2816, 640, 64)])
def test_moe_tokens_do_not_mix_in_units_of_many_chunks(T, H, I, E):
    """Tokens of Inf and NaN beside others, in experts whose matrices are cut into
    many chunks: the others stay within the bound they have alone (what they
    choose leaves other chunks, so bits may differ)."""
    import dense_gemm_03_gb300 as g
    t = torch()
    o = moe_operands(t, 91 + T, T, H, I, E)
    o["Wr"] = (o["Wr"].float() * 4).half()
    o["X"][5, 3], o["X"][9] = float("inf"), float("nan")
    v = {k: x.cuda() for k, x in o.items()}
    Y, ids = t.empty_like(v["Y0"]), t.empty((T, 2), dtype=t.int32, device="cuda")
    g.gemm_f16_moe(v["X"], v["Wr"], v["W1"], v["W2"], Y, 2, ids=ids)
    sync(t)
    rows = [i for i in range(T) if i not in (5, 9)]
    o["X"] = o["X"][rows]
    want_ids, want, tol = moe_exact(o, 2)
    same = (ids.cpu()[rows].long() == want_ids).all(1)
    assert int(same.sum()) >= len(rows) - 1           # a near tie may go either way
    ref.check(Y.cpu()[rows][same], want[same], tol[same])
    assert Y[9].isnan().all()


@pytest.mark.parametrize("T,H,I,E", [(1, 128, 96, 4), (5, 2560, 640, 3), (33, 264, 200, 2),
                                     (64, 1024, 1024, 1), (5, 130, 97, 3)])
def test_moe_integers_exact(T, H, I, E):
    """Gated rows of 15 to 17 bits whose differences are the result: every sum is
    exact, and the half that their upper 11 bits leave out is needed."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator().manual_seed(T + H)

    def ints(lo, hi, *shape):
        return t.randint(lo, hi + 1, shape, generator=gen).double()

    X = ints(-1, 1, T, H)
    X[:, 0] = 1
    Wr = t.zeros(H, E, dtype=t.float64)
    Wr[1] = t.arange(E, dtype=t.float64)
    W1 = t.zeros(E, H, 2 * I, dtype=t.float64)
    W1[:, 0, :I], W1[:, 0, I:] = 210, 190             # silu(x) = x in fp32 from about 20 on
    for k in range(2, min(H, 34)):
        W1[:, k] = ints(-1, 1, E, 2 * I)
    W1[:, H - 1] = ints(-2, 2, E, 2 * I)
    W2 = t.zeros(E, I, H, dtype=t.float64)
    for e in range(E):
        a, b = (t.randint(0, I, (H,), generator=gen) for _ in range(2))
        W2[e, a, t.arange(H)] += 1
        W2[e, b, t.arange(H)] -= 1
    e = (X @ Wr).argmax(1)
    gu = (X[:, None] @ W1[e])[:, 0]
    assert gu.min() > 100
    want = ((gu[:, :I] * gu[:, I:])[:, None] @ W2[e])[:, 0]
    v = [x.half().cuda() for x in (X, Wr, W1, W2)]
    Y = t.empty((T, H), dtype=t.float16, device="cuda")
    ids = t.empty((T, 1), dtype=t.int32, device="cuda")
    g.gemm_f16_moe(*v, Y, 1, ids=ids)
    sync(t)
    assert t.equal(ids.cpu()[:, 0].long(), e)
    assert t.equal(Y.cpu(), want.half()), g.last_path()
