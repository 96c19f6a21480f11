"""A whole mixture-of-experts layer for a few tokens, through the public
binding, against the 64-bit definition."""
import numpy as np
import pytest

import routed_ref as ref
from helpers import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


def operands(t, seed, T, H, I, E):
    rng = np.random.default_rng(seed)
    def draw(*shape, std=1.0):
        return t.from_numpy(rng.normal(0, std, shape).astype(np.float16))
    return dict(X=draw(T, H), Wr=draw(H, E, std=2 * H ** -0.5), W1=draw(E, H, 2 * I, std=H ** -0.5),
                W2=draw(E, I, H, std=I ** -0.5), Y0=draw(T, H))


def call(o, topk, renorm, beta, Y=None):
    import dense_gemm_03_gb300 as g
    t = torch()
    v = {k: x.cuda() for k, x in o.items()}
    T = v["X"].shape[0]
    if Y is None:
        Y = v["Y0"].clone() if beta else t.full_like(v["Y0"], float("nan"))
    ids = t.full((T, topk), -9, dtype=t.int32, device="cuda")
    probs = t.full((T, topk), float("nan"), device="cuda")
    g.gemm_f16_moe(v["X"], v["Wr"], v["W1"], v["W2"], Y, topk, ids=ids, probs=probs,
                   renormalize=renorm, beta=beta)
    t.cuda.synchronize()
    assert g.debug_status() == 0
    return Y.cpu(), ids.cpu(), probs.cpu()


SHAPES = [
    # T, H, I, E, topk
    (1, 1, 1, 1, 1),
    (1, 64, 32, 4, 2),
    (1, 512, 256, 16, 8),
    (1, 1024, 704, 8, 1),
    (2, 200, 72, 5, 5),            # every expert chosen
    (3, 136, 1000, 7, 3),
    (4, 65, 33, 6, 2),             # nothing aligned
    (5, 256, 7, 9, 4),             # odd I
    (8, 520, 264, 32, 4),
    (16, 256, 128, 3, 2),          # many tokens to an expert
    (17, 384, 320, 64, 6),
    (33, 128, 136, 130, 8),
    (40, 264, 200, 1, 1),          # one expert for all
    (64, 512, 256, 16, 2),
    (100, 192, 64, 4, 3),
    (129, 128, 72, 8, 2),          # more tokens than one block takes
    (300, 72, 64, 5, 2),
    (3, 64, 40, 1000, 20),
]


@pytest.mark.parametrize("T,H,I,E,topk", SHAPES)
@pytest.mark.parametrize("renorm,beta", [(True, 0.0), (False, -0.5)])
def test_layer(T, H, I, E, topk, renorm, beta):
    import dense_gemm_03_gb300 as g
    t = torch()
    seed = T + H + I
    while True:   # inputs whose choice the logits' own error cannot change
        o = operands(t, seed, T, H, I, E)
        ids, p, ptol, Y, tol, margin = ref.moe(o["X"], o["Wr"], o["W1"], o["W2"], o["Y0"], topk,
                                               renorm, beta)
        if margin > 1:
            break
        seed += 1000003
    got, gids, gp = call(o, topk, renorm, beta)
    assert t.equal(gids.long(), ids), g.last_path()
    ref.check(gp, p, ptol, "probs " + g.last_path())
    ref.check(got, Y, tol, "Y " + g.last_path())


def test_ties_go_to_the_lowest_index():
    t = torch()
    T, H, I, E, k = 6, 64, 64, 12, 5
    o = operands(t, 3, T, H, I, E)
    o["Wr"].zero_()
    o["Wr"][0] = t.tensor([1, 3, 3, 2, 3, 0, 2, 3, 1, 2, -1, 0], dtype=t.float16)
    o["X"][:, 0] = t.tensor([1, 2, 0.5, 0, -1, -0.0], dtype=t.float16)
    _, ids, probs = call(o, k, True, 0.0)
    assert ids[0].tolist() == ids[1].tolist() == ids[2].tolist() == [1, 2, 4, 7, 3]
    assert ids[3].tolist() == ids[5].tolist() == [0, 1, 2, 3, 4]      # all logits equal
    assert ids[4].tolist() == [10, 5, 11, 0, 8]
    assert t.allclose(probs[3], t.full((k,), 1.0 / k), rtol=1e-6, atol=0)


def test_tokens_and_experts_do_not_mix():
    """A token of Inf, one of NaN, and experts holding NaN and Inf: every other
    token that did not choose those experts keeps its bits."""
    t = torch()
    T, H, I, E, k = 24, 128, 96, 16, 2
    o = operands(t, 8, T, H, I, E)
    Y, ids, probs = call(o, k, True, 0.0)
    b = {n: x.clone() for n, x in o.items()}
    b["X"][5, 3] = float("inf")
    b["X"][9] = float("nan")
    e1, e2 = int(ids[0, 0]), int(ids[1, 1])
    b["W1"][e1] = float("nan")
    b["W2"][e2] = float("inf")
    Y2, ids2, probs2 = call(b, k, True, 0.0)
    assert ((ids2 >= 0) & (ids2 < E)).all()
    rows = [i for i in range(T) if i not in (5, 9)]
    assert t.equal(ids[rows], ids2[rows]) and t.equal(probs[rows], probs2[rows])
    keep = [i for i in rows if e1 not in ids[i].tolist() and e2 not in ids[i].tolist()]
    assert keep and t.equal(Y[keep], Y2[keep])
    assert Y2[9].isnan().all() and Y2[0].isnan().all() and not t.isfinite(Y2[1]).any()


def test_unchosen_experts_are_not_read_for_one_token():
    t = torch()
    o = operands(t, 4, 1, 256, 128, 32)
    Y, ids, _ = call(o, 4, True, 0.0)
    for e in range(32):
        if e not in ids[0].tolist():
            o["W1"][e] = float("nan")
            o["W2"][e] = float("nan")
    assert t.equal(Y, call(o, 4, True, 0.0)[0])


@pytest.mark.parametrize("T,H,I", [(7, 128, 64), (7, 130, 64), (65, 136, 72)])
def test_leading_dimensions(T, H, I):
    import dense_gemm_03_gb300 as g
    t = torch()
    E, k = 6, 2
    o = operands(t, T + H, T, H, I, E)
    want, _, _ = call(o, k, True, 0.5)
    X = t.full((T, H + 8), float("nan"), dtype=t.float16, device="cuda")
    Y = t.full((T, H + 5), float("nan"), dtype=t.float16, device="cuda")
    X[:, :H], Y[:, :H] = o["X"].cuda(), o["Y0"].cuda()
    g.gemm_f16_moe(X, o["Wr"].cuda(), o["W1"].cuda(), o["W2"].cuda(), Y, k, beta=0.5, H=H,
                   ldx=H + 8, ldy=H + 5)
    t.cuda.synchronize()
    assert g.debug_status() == 0
    assert t.equal(Y[:, :H].cpu(), want) and Y[:, H:].isnan().all()


def test_empty_calls():
    import dense_gemm_03_gb300 as g
    t = torch()
    o = operands(t, 2, 4, 32, 16, 3)
    v = {n: x.cuda() for n, x in o.items()}
    Y = v["Y0"].clone()
    g.gemm_f16_moe(v["X"], v["Wr"], v["W1"], v["W2"], Y, 2, T=0)
    t.cuda.synchronize()
    assert t.equal(Y, v["Y0"])
    g.gemm_f16_moe(v["X"], v["Wr"], None, v["W2"], Y, 2, I=0, beta=0.5)   # nothing but beta Y
    t.cuda.synchronize()
    assert t.equal(Y, (v["Y0"].float() * 0.5).half())


@pytest.mark.parametrize("T", [1, 20, 140])
def test_streams_graphs_and_repeats(T):
    import dense_gemm_03_gb300 as g
    t = torch()
    k = 4
    v = {n: x.cuda() for n, x in operands(t, 5, T, 256, 192, 16).items()}
    t.cuda.synchronize()
    def run(Y):
        g.gemm_f16_moe(v["X"], v["Wr"], v["W1"], v["W2"], Y, k)
    a, b, c = (t.full_like(v["Y0"], float("nan")) for _ in range(3))
    run(a)
    t.cuda.synchronize()
    s = t.cuda.Stream()
    with t.cuda.stream(s):
        run(b)
        run(c)
    s.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(s):
        with t.cuda.graph(graph, stream=s):
            run(c)
    for _ in range(3):
        c.fill_(float("nan"))
        graph.replay()
    t.cuda.synchronize()
    assert g.debug_status() == 0
    assert t.equal(a, b) and t.equal(a, c)
