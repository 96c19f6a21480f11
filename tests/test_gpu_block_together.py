"""The dense block's operators as a program uses them together (a feed-forward block
trained in half and served in 8 bits), and under what programs do around them: streams,
host threads, captured graphs, larger calls in between, matrices past 2^31 elements."""
import threading

import numpy as np
import pytest

import block_ref as ref
from helpers import torch
from test_gpu_block import normal, operands, sync
from test_gpu_i8 import operands as i8_operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T,H,I", [(1, 256, 512), (37, 384, 1000), (700, 512, 1368)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_block_trained(T, H, I, act):
    """Forward and backward of Y = (f(X W1g) * (X W1u)) W2, every step against its
    definition on what the step before it left."""
    import dense_gemm_03_gb300 as g
    t = torch()
    X, W1, _ = operands(t, T, I, H, 1.0)
    rng = np.random.default_rng(T)
    W2, dY = normal(t, rng, (I, H), I ** -0.5), normal(t, rng, (T, H), 0.1)
    x, w1, w2, dy = (v.cuda() for v in (X, W1, W2, dY))
    new = lambda *s, dtype=t.float16: t.full(s, float("nan"), dtype=dtype, device="cuda")
    h, y, dh, dgu, dx, dw1 = (new(*s) for s in ((T, I), (T, H), (T, I), (T, 2 * I), (T, H), (H, 2 * I)))
    dw2 = new(I, H, dtype=t.float32)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        g.gemm_f16_glu(x, w1, h, act)
        g.gemm_f16(h, w2, y)
        g.gemm_f16_trans(dy, w2, dh, False, True)            # dH = dY W2^T
        g.gemm_f16_trans_f32out(h, dy, dw2, True, False)     # dW2 = H^T dY, in float
        g.gemm_f16_trans_f32out(h, dy, dw2, True, False, beta=1.0)   # a second micro-batch
        g.gemm_f16_glu_grad(dh, x, w1, dgu, dx, dw1, act)
    s.synchronize()
    sync(t)
    H_, dH_, dGU_ = h.cpu(), dh.cpu(), dgu.cpu()
    ref.check(H_, *ref.glu(X, W1, act), "H")
    ref.check(y.cpu(), *ref.product(H_, W2), "Y")
    ref.check(dH_, *ref.product(dY, W2.t()), "dH")
    want, tol = ref.product(H_.t(), dY, f32=True)
    ref.check(dw2.cpu(), 2 * want, 2 * tol + 2 * ref.U2 * want.abs(), "dW2")
    ref.check(dGU_, *ref.glu_grad(dH_, X, W1, act), "dGU")
    ref.check(dx.cpu(), *ref.product(dGU_, W1.t()), "dX")
    ref.check(dw1.cpu(), *ref.product(X.t(), dGU_), "dW1")


@pytest.mark.parametrize("T,H,I", [(1, 256, 512), (19, 384, 1000), (600, 512, 1408)])
def test_block_served(T, H, I):
    """The same block in 8 bits: tokens rounded, gated product, tokens rounded, product;
    the result added onto its residual."""
    import dense_gemm_03_gb300 as g
    t = torch()
    rng = np.random.default_rng(T + H)
    X, R = normal(t, rng, (T, H)), normal(t, rng, (T, H))
    def weights(k, n):
        w = rng.normal(0, k ** -0.5, (k, n))
        s = (np.abs(w).max(0) / 127).astype(np.float32)
        return t.from_numpy(np.rint(w / s).astype(np.int8)), t.from_numpy(s)
    (W1, s1), (W2, s2) = weights(H, 2 * I), weights(I, H)
    c = lambda v: v.cuda()
    q1, q2 = (t.empty(s, dtype=t.int8, device="cuda") for s in ((T, H), (T, I)))
    a1, a2 = (t.empty(T, device="cuda") for _ in range(2))
    h, y = t.empty(T, I, dtype=t.float16, device="cuda"), R.cuda().clone()
    g.f16_to_i8(c(X), q1, a1)
    g.gemm_i8(q1, c(W1), h, a1, c(s1), "silu")
    g.f16_to_i8(h, q2, a2)
    g.gemm_i8(q2, c(W2), y, a2, c(s2), beta=1.0)
    sync(t)
    want, scales = ref.to_i8(X)
    assert t.equal(q1.cpu(), want) and t.equal(a1.cpu(), scales)
    ref.check(h.cpu(), *ref.i8(q1.cpu(), W1, a1.cpu(), s1, "silu"), "H")
    want, scales = ref.to_i8(h.cpu())
    assert t.equal(q2.cpu(), want) and t.equal(a2.cpu(), scales)
    ref.check(y.cpu(), *ref.i8(q2.cpu(), W2, a2.cpu(), s2, None, 1.0, R), "Y")


# ------------------------------------------------------------------ programs
def make(t, kind, big, seed):
    """(run(**stream), outputs) of a call; `big`: one that takes other kernels and more
    scratch than the small one."""
    import dense_gemm_03_gb300 as g
    gen = t.Generator(device="cuda").manual_seed(seed)
    h = lambda *s: t.randn(s, generator=gen, device="cuda").half()
    new = lambda *s, dtype=t.float16: t.zeros(s, dtype=dtype, device="cuda")
    q = lambda *s: t.randint(-127, 128, s, generator=gen, device="cuda").to(t.int8)
    if kind == "glu":
        M, K, N = (1500, 500, 1501) if big else (9, 1000, 2501)
        X, W, C = h(M, K), h(K, 2 * N) * K ** -0.5, new(M, N)
        return (lambda **k: g.gemm_f16_glu(X, W, C, **k)), [C]
    if kind == "grad":
        M, K, N = (2304, 3200, 1283) if big else (30, 512, 701)
        X, W, dC = h(M, K), h(K, 2 * N) * K ** -0.5, h(M, N)
        out = [new(M, 2 * N), new(M, K), new(K, 2 * N)]
        return (lambda **k: g.gemm_f16_glu_grad(dC, X, W, *out, "gelu", **k)), out
    if kind == "trans":
        M, K, N = (4096, 3200, 1291) if big else (300, 3001, 130)
        A, B, C = h(K, M), h(N, K), new(M, N, dtype=t.float32)
        return (lambda **k: g.gemm_f16_trans_f32out(A, B, C, True, True, **k)), [C]
    if kind == "i8":
        M, K, N = (1100, 1000, 2605) if big else (5, 2000, 12001)
        X, W, C = q(M, K), q(K, N), new(M, N)
        sx = t.rand(M, generator=gen, device="cuda") / 5000
        return (lambda **k: g.gemm_i8(X, W, C, sx, **k)), [C]
    M, K = (6000, 4096) if big else (40, 3001)
    X, Q, S = h(M, K), new(M, K, dtype=t.int8), new(M, dtype=t.float32)
    return (lambda **k: g.f16_to_i8(X, Q, S, **k)), [Q, S]


KINDS = ("glu", "grad", "trans", "i8", "to_i8")


def fresh(t, run, outs, **k):
    for o in outs:
        o.zero_()
    t.cuda.synchronize()
    run(**k)
    t.cuda.synchronize()
    return [o.clone() for o in outs]


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_graph_replays(kind, big):
    """A captured call gives the direct call's bits at every replay."""
    import dense_gemm_03_gb300 as g
    t = torch()
    run, outs = make(t, kind, big, 7)
    want = fresh(t, run, outs)
    s = t.cuda.Stream()
    with t.cuda.stream(s):
        run()
    s.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=s):
        run()
        run()
    for _ in range(3):
        for o in outs:
            o.zero_()
        t.cuda.synchronize()
        graph.replay()
        sync(t)
        assert all(t.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.parametrize("kind,larger", [(a, b) for a in KINDS for b in ("grad", "i8") if a != "to_i8"])
def test_a_graph_outlives_larger_calls_on_its_stream(kind, larger):
    import dense_gemm_03_gb300 as g
    t = torch()
    g.release()
    (run, outs), (more, _) = make(t, kind, False, 11), make(t, larger, True, 12)
    s = t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.stream(s):
        run()
        s.synchronize()
        want = [o.clone() for o in outs]
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, stream=s):
            run()
        more()
        s.synchronize()
        for o in outs:
            o.zero_()
        graph.replay()
        s.synchronize()
    sync(t)
    assert all(t.equal(a, b) for a, b in zip(want, outs))
    del graph
    g.release()


def test_calls_of_all_kinds_on_two_streams_at_once():
    import dense_gemm_03_gb300 as g
    t = torch()
    calls = [make(t, kind, big, 20 + i) for i, kind in enumerate(KINDS) for big in (False, True)]
    want = [fresh(t, run, outs) for run, outs in calls]
    twins = [make(t, kind, big, 20 + i) for i, kind in enumerate(KINDS) for big in (False, True)]
    a, b = t.cuda.Stream(), t.cuda.Stream()
    for turn in range(4):
        for _, outs in calls + twins:
            for o in outs:
                o.zero_()
        t.cuda.synchronize()
        for i in range(len(calls)):     # in different orders
            with t.cuda.stream(a):
                calls[i][0]()
            with t.cuda.stream(b):
                twins[(i * 3 + turn) % len(twins)][0]()
        sync(t)
        for (_, x), (_, y), w in zip(calls, twins, want):
            assert all(t.equal(p, r) and t.equal(q, r) for p, q, r in zip(x, y, w))


def test_host_threads_on_one_stream():
    """Calls whose kernels share a stream's scratch stay together there."""
    import dense_gemm_03_gb300 as g
    t = torch()
    calls = [make(t, kind, False, 30 + i) for i, kind in enumerate(KINDS)]
    want = [fresh(t, run, outs) for run, outs in calls]
    s = t.cuda.Stream()
    failed = []

    def work(run):
        try:
            for _ in range(40):
                run(stream=s)
        except Exception as e:          # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(run,)) for run, _ in calls]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    sync(t)
    assert not failed
    for (_, outs), w in zip(calls, want):
        assert all(t.equal(a, b) for a, b in zip(outs, w))


def test_per_thread_stream_and_explicit_handles():
    import dense_gemm_03_gb300 as g
    t = torch()
    for kind in KINDS:
        run, outs = make(t, kind, False, 40)
        want = fresh(t, run, outs)
        for handle in (0, 1, 2):        # legacy (two names) and per-thread default streams
            got = fresh(t, run, outs, stream=handle)
            assert all(t.equal(a, b) for a, b in zip(want, got)), (kind, handle)


# ------------------------------------------------------------------ large
@pytest.mark.parametrize("op", ["glu", "grad", "trans", "i8", "to_i8", "i8_weights"])
def test_past_32_bit_offsets(op):
    """Matrices of more than 2^31 elements: the first and last rows and some between."""
    import dense_gemm_03_gb300 as g
    t = torch()
    gen = t.Generator(device="cuda").manual_seed(1)
    h = lambda *s: t.randn(s, generator=gen, device="cuda").half()
    rows = lambda M: t.tensor([0, 1, M // 3, M - 129, M - 1])
    if op in ("glu", "grad", "trans"):
        M, N, K = 70000, 32768, 64
        X, W = h(M, K), h(K, N if op != "glu" else 2 * N) * 0.125
        if op == "glu":
            C = t.empty(M, N, dtype=t.float16, device="cuda")
            g.gemm_f16_glu(X, W, C)
            sync(t)
            i = rows(M)
            ref.check(C[i].cpu(), *ref.glu(X[i].cpu(), W.cpu(), "silu"), op)
        elif op == "trans":
            C = t.empty(M, N, dtype=t.float16, device="cuda")
            g.gemm_f16_trans(X.t().contiguous(), W, C, True, False)
            sync(t)
            i = rows(M)
            ref.check(C[i].cpu(), *ref.product(X[i].cpu(), W.cpu()), op)
        else:
            N //= 2                      # dGU has more than 2^31 elements
            dC, gu, dX = h(M, N), t.empty(M, 2 * N, dtype=t.float16, device="cuda"), t.empty_like(X)
            g.gemm_f16_glu_grad(dC, X, W, gu, dX)
            sync(t)
            i = rows(M)
            ref.check(gu[i].cpu(), *ref.glu_grad(dC[i].cpu(), X[i].cpu(), W.cpu(), "silu"), op)
            ref.check(dX[i].cpu(), *ref.product(gu[i].cpu(), W.t().cpu()), "dX")
    elif op == "to_i8":
        M, K = 300001, 7168
        X = h(M, K)
        Q, s = t.empty(M, K, dtype=t.int8, device="cuda"), t.empty(M, device="cuda")
        g.f16_to_i8(X, Q, s)
        sync(t)
        i = rows(M)
        want, scales = ref.to_i8(X[i].cpu())
        assert t.equal(Q[i].cpu(), want) and t.equal(s[i].cpu(), scales)
    else:
        # many tokens, or weights of more than 2^31 bytes for a few
        M, N, K = (70000, 32768, 64) if op == "i8" else (3, 40000, 65536)
        q = lambda *s: t.randint(-127, 128, s, generator=gen, device="cuda", dtype=t.int8)
        X, W = q(M, K), q(K, N)
        C = t.empty(M, N, dtype=t.float16, device="cuda")
        sx = t.full((M,), 1.0 / (5400 * K ** 0.5), device="cuda")
        g.gemm_i8(X, W, C, sx)
        sync(t)
        i = rows(M) if op == "i8" else t.arange(M)
        cols = t.tensor([0, 77, N // 2, N - 1])
        ref.check(C[i][:, cols].cpu(), *ref.i8(X[i].cpu(), W[:, cols].cpu(), sx[i].cpu(), None), op)


def test_example():
    """It runs, and its gradients are the definition's: those of the mean squared
    distance, by 64-bit autograd on the same rows."""
    import importlib.util
    import os
    t = torch()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "dense_block.py")
    spec = importlib.util.spec_from_file_location("dense_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    out = ex.main(H=64, I=96, T=40, steps=2)
    assert len(out["losses"]) == 2 and all(np.isfinite(out["losses"]))
    # 8 bits: two roundings to 1/254 of a row's or channel's largest entry on each side
    assert 0 < out["off"] < 0.1
    gen = t.Generator(device="cuda").manual_seed(8)
    x, dy = (t.randn(s, generator=gen, device="cuda").half() for s in ((40, 64), (40, 64)))
    w1, w2 = out["weights"]
    dw1, dw2 = (t.full(w.shape, float("nan"), device="cuda") for w in (w1, w2))
    h, _ = ex.forward(x, w1, w2)
    ex.backward(x, w1, w2, h, dy, dw1, dw2, True)
    a, b = (w.double().requires_grad_(True) for w in (w1, w2))
    s = x.double() @ a
    y = (t.nn.functional.silu(s[:, :96]) * s[:, 96:]) @ b
    y.backward(dy.double())
    # h, dh and dgu are halves: each rounding is at most 2^-11 of every term
    terms = lambda p, q: p.double().abs().t() @ q.double().abs()
    assert bool(((dw2.double() - b.grad).abs() <= 1.01 * ref.HALF * terms(h, dy) + 1e-6).all())
    dh_terms = dy.double().abs() @ w2.double().abs().t()
    g_, u_ = s[:, :96].detach(), s[:, 96:].detach()
    f, df = ref.act_both("silu", g_)
    each = t.cat([dh_terms * u_.abs() * df.abs(), dh_terms * f.abs()], 1)
    assert bool(((dw1.double() - a.grad).abs() <= 2.02 * ref.HALF * (x.double().abs().t() @ each) + 1e-6).all())


# ------------------------------------------- calls that start as others end
def chain(t, seed, T, H, I):
    """Calls that each read what the one before wrote, or write what it reads, between a
    framework's own kernels, copies and fills."""
    import dense_gemm_03_gb300 as g
    rng = np.random.default_rng(seed)
    x, dy = (normal(t, rng, (T, H), 1.0).cuda() for _ in "xd")
    w = normal(t, rng, (H, 2 * I), H ** -0.5).cuda()
    wd = normal(t, rng, (I, H), I ** -0.5).cuda()
    q = t.zeros((T, H), dtype=t.int8, device="cuda")
    wq = t.randint(-127, 128, (H, H), dtype=t.int8, device="cuda",
                   generator=t.Generator(device="cuda").manual_seed(seed))
    sq, sw = t.zeros(T, device="cuda"), t.full((H,), 1.0 / 73 / H ** 0.5, device="cuda")
    new = lambda *s, dtype=t.float16: t.zeros(s, dtype=dtype, device="cuda")
    h, y, z, dgu, dx = new(T, I), new(T, H), new(T, H), new(T, 2 * I), new(T, H)
    dw, dh = new(H, 2 * I), new(T, I)
    dwd = new(I, H, dtype=t.float32)
    first = x.clone()
    def steps():
        yield lambda: x.copy_(first)
        for turn in range(3):
            yield lambda: g.gemm_f16_glu(x, w, h, "silu")
            yield lambda: g.gemm_f16(h, wd, y)
            yield lambda: g.f16_to_i8(y, q, sq)
            yield lambda: g.gemm_i8(q, wq, z, sq, sw)
            yield lambda: y.zero_()
            yield lambda: g.gemm_f16_trans(z, wd, dh, False, True)
            yield lambda: g.gemm_f16_trans_f32out(h, z, dwd, True, False, beta=0.5 if turn else 0.0)
            yield lambda: h.mul_(0.5)
            yield lambda: g.gemm_f16_glu_grad(dh, x, w, dgu, dx, dw, "gelu", beta=0.5 if turn else 0.0)
            yield lambda: x.copy_(dx)
            yield lambda: x.add_(first)
            yield lambda: g.f16_to_i8(x, q, sq)
            yield lambda: g.gemm_i8(q, wq, z, sq, sw)
            yield lambda: x.add_(z)
    return steps, [x, y, z, h, q, sq, dgu, dx, dw, dh, dwd]


@pytest.mark.parametrize("T,H,I", [(1, 256, 512), (24, 515, 1001), (300, 512, 1024), (700, 777, 1201),
                                   (2048, 768, 1024)])
def test_calls_in_a_row_wait_for_the_ones_before(T, H, I):
    t = torch()
    steps, outs = chain(t, 5, T, H, I)
    for step in steps():     # one at a time
        step()
        t.cuda.synchronize()
    want = [o.clone() for o in outs]
    # (values grow from turn to turn: entries of the last dW pass the half range)
    assert not any(bool(t.isnan(o.float()).any()) for o in outs)
    for stream in (t.cuda.current_stream(), t.cuda.Stream()):
        with t.cuda.stream(stream):
            for _ in range(20):
                for step in steps():
                    step()
        sync(t)
        assert all(t.equal(a, b) for a, b in zip(want, outs))
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=stream):
        for step in steps():
            step()
    for _ in range(3):
        graph.replay()
    sync(t)
    assert all(t.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.parametrize("big", [False, True])
def test_a_captured_call_after_a_join(big):
    """Calls captured first on a forked stream, and behind two streams at once."""
    import dense_gemm_03_gb300 as g
    t = torch()
    T, H, I = (600, 512, 1024) if big else (24, 512, 1024)
    rng = np.random.default_rng(3)
    x, w = normal(t, rng, (T, H), 1.0).cuda(), normal(t, rng, (H, 2 * I), H ** -0.5).cuda()
    h, v = (t.zeros((T, I), dtype=t.float16, device="cuda") for _ in "hv")
    dw = t.zeros((I, I), dtype=t.float32, device="cuda")
    q, sq = t.zeros((T, I), dtype=t.int8, device="cuda"), t.zeros(T, device="cuda")
    a, b = t.cuda.Stream(), t.cuda.Stream()

    def run():
        x2 = x * 0.5
        b.wait_stream(a)
        g.gemm_f16_glu(x, w, h, "silu", stream=a)
        with t.cuda.stream(b):
            g.gemm_f16_glu(x2, w, v, "gelu", stream=b)
        a.wait_stream(b)
        g.gemm_f16_trans_f32out(h, v, dw, True, False, stream=a)   # behind both
        b.wait_stream(a)
        with t.cuda.stream(b):
            g.f16_to_i8(h, q, sq, stream=b)
            g.f16_to_i8(v, q, sq, stream=b)
        a.wait_stream(b)
    with t.cuda.stream(a):
        run()
    sync(t)
    want = [o.clone() for o in (h, v, dw, q, sq)]
    ref.check(dw.cpu(), *ref.product(h.cpu().t(), v.cpu(), f32=True), "dW")
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph, stream=a):
        run()
    for _ in range(3):
        for o in (h, v, dw, q, sq):
            o.zero_()
        t.cuda.synchronize()
        graph.replay()
        sync(t)
        assert all(t.equal(p, r) for p, r in zip((h, v, dw, q, sq), want))
