"""The library's scratch under programs that share it: graphs captured on a
stream beside larger calls on it, and host threads on one stream."""
import threading

import pytest

from helpers import torch
from test_gpu_lora import operands as lora_operands
from test_gpu_moe import operands as moe_operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


def lora_call(t, M, N, K, R, n, seed, grad=False):
    """A call on `M` rows: (run(), its outputs)."""
    import dense_gemm_03_gb300 as g
    o = {k: v.cuda() for k, v in lora_operands(t, seed, M, N, K, R, n, "mixed").items()}
    if not grad:
        C = t.full_like(o["C0"], float("nan"))
        return (lambda **k: g.gemm_f16_lora(o["X"], o["W"], C, o["A"], o["B"], o["ids"], o["scales"],
                                            **k)), [C]
    out = [t.full_like(o["X"], float("nan")), t.full_like(o["dA0"], float("nan")),
           t.full_like(o["dB0"], float("nan"))]
    return (lambda **k: g.gemm_f16_lora_grad(o["G"], o["X"], o["W"], o["A"], o["B"], o["ids"],
                                             o["scales"], *out, **k)), out


def moe_call(t, T, H, I, E, k, seed):
    import dense_gemm_03_gb300 as g
    o = {n: v.cuda() for n, v in moe_operands(t, seed, T, H, I, E).items()}
    Y = t.full_like(o["Y0"], float("nan"))
    return (lambda **s: g.gemm_f16_moe(o["X"], o["Wr"], o["W1"], o["W2"], Y, k, **s)), [Y]


def gemm_call(t, M, N, K, seed):
    import dense_gemm_03_gb300 as g
    gen = t.Generator(device="cuda").manual_seed(seed)
    A, B = (t.randn(s, generator=gen, device="cuda").half() for s in ((M, K), (K, N)))
    C = t.full((M, N), float("nan"), dtype=t.float16, device="cuda")
    return (lambda **k: g.gemm_f16(A, B, C, **k)), [C]


KINDS = {
    # small call, then one that needs more of the same scratch
    "decode": (lambda t: lora_call(t, 8, 1024, 2048, 16, 6, 51),
               lambda t: lora_call(t, 1500, 1001, 2048, 8, 6, 52)),
    "tiles": (lambda t: lora_call(t, 2300, 1290, 512, 16, 6, 53),
              lambda t: lora_call(t, 3000, 1930, 1032, 40, 6, 54)),
    "grad": (lambda t: lora_call(t, 40, 512, 1024, 16, 6, 55, True),
             lambda t: lora_call(t, 2500, 1288, 1032, 16, 6, 56, True)),
    "moe": (lambda t: moe_call(t, 3, 512, 256, 16, 4, 57),
            lambda t: moe_call(t, 64, 2048, 1024, 32, 8, 58)),
    "dense": (lambda t: gemm_call(t, 300, 501, 3000, 59),
              lambda t: gemm_call(t, 2000, 2601, 4096, 60)),
}


@pytest.mark.parametrize("kind,larger", [(k, k) for k in sorted(KINDS)] +
                         [("decode", "moe"), ("moe", "grad"), ("grad", "tiles"), ("dense", "tiles")])
def test_a_graph_outlives_larger_calls_on_its_stream(kind, larger):
    """Replays of a graph give its results, and write nowhere else, after calls
    on the same stream that outgrew the scratch it was captured with."""
    import dense_gemm_03_gb300 as g
    t = torch()
    g.release()
    small, large = KINDS[kind][0](t), KINDS[larger][1](t)
    run, outs = small
    s = t.cuda.Stream()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.stream(s):
        run()
        s.synchronize()
        want = [x.clone() for x in outs]
        s.synchronize()
        with t.cuda.graph(graph, stream=s):
            run()
        large[0]()
        s.synchronize()
        want_large = [x.clone() for x in large[1]]
    t.cuda.synchronize()
    # whatever the larger call freed may go to these
    mine = [t.full((n,), 7.0, device="cuda") for n in [1 << 18] * 8 + [1 << 22] * 4]
    for _ in range(3):
        for x in outs:
            x.fill_(float("nan"))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(want, outs))
    with t.cuda.stream(s):
        large[0]()
    t.cuda.synchronize()
    assert g.debug_status() == 0
    assert all(t.equal(a, b) for a, b in zip(want_large, large[1]))
    assert all(bool((x == 7.0).all()) for x in mine)
    del graph
    g.release()


@pytest.mark.parametrize("kind", ["decode", "tiles", "grad", "moe", "f16", "f32"])
def test_first_call_of_a_host_thread(kind):
    """A thread whose first use of CUDA is a call of the library."""
    import dense_gemm_03_gb300 as g
    t = torch()
    dt = t.float32 if kind == "f32" else t.float16
    A, B = (t.randn(256, 256, device="cuda").to(dt) for _ in range(2))
    C = t.empty_like(A)
    run, out = {"f16": lambda: (lambda: g.gemm_f16(A, B, C), [C]),
                "f32": lambda: (lambda: g.sgemm_f32(A, B, C), [C])}.get(
                    kind, lambda: KINDS[kind][0](t))()
    run()
    t.cuda.synchronize()
    want = [x.clone() for x in out]
    for x in out:
        x.fill_(float("nan"))
    t.cuda.synchronize()
    errors = []

    def work():
        try:
            run()
        except Exception as e:      # reported on the main thread
            errors.append(repr(e))

    th = threading.Thread(target=work)
    th.start()
    th.join()
    t.cuda.synchronize()
    assert not errors, errors
    assert g.debug_status() == 0
    assert all(t.equal(a, b) for a, b in zip(want, out))


PER_THREAD = 2      # the handle cudaStreamPerThread


@pytest.mark.parametrize("shared", [True, False])
def test_host_threads(shared):
    """Threads that call different operators, all on one stream or each on its
    per-thread stream (one handle value for all of them), get the bits each call
    gives alone; the scratch grows meanwhile."""
    import dense_gemm_03_gb300 as g
    t = torch()
    makers = [lambda i: lora_call(t, 8 + i, 1024, 2048, 16, 6, 100 + i),
              lambda i: lora_call(t, 300 + 300 * i, 512, 1024, 16, 6, 110 + i, True),
              lambda i: moe_call(t, 2 + 5 * i, 512, 256, 16, 4, 120 + i),
              lambda i: moe_call(t, 40 + i, 1024, 512, 32, 4, 130 + i),
              lambda i: lora_call(t, 2300, 1290, 256 + 256 * i, 16, 6, 140 + i),
              lambda i: gemm_call(t, 300, 501, 1500 * (1 + i), 150 + i)]
    jobs = [[m(i) for i in range(4)] for m in makers]
    want = []
    for calls in jobs:
        for run, _ in calls:
            run()
        t.cuda.synchronize()
        want.append([[x.clone() for x in out] for _, out in calls])
        for _, out in calls:
            for x in out:
                x.fill_(float("nan"))
    t.cuda.synchronize()
    g.release()
    s = t.cuda.Stream()
    handle = s.cuda_stream if shared else PER_THREAD
    errors, gate = [], threading.Barrier(len(jobs))

    def work(calls):
        try:
            gate.wait()
            for _ in range(12):
                for run, _ in calls:
                    run(stream=handle)
        except Exception as e:      # reported on the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(c,)) for c in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    t.cuda.synchronize()
    assert not errors, errors
    assert g.debug_status() == 0
    for calls, refs in zip(jobs, want):
        for (_, out), ref in zip(calls, refs):
            assert all(t.equal(a, b) for a, b in zip(out, ref))


def test_release_beside_calls():
    """gemm_release() waits for calls in progress on other threads, and they go
    on after it."""
    import dense_gemm_03_gb300 as g
    t = torch()
    run, out = lora_call(t, 16, 512, 1024, 16, 4, 160)
    run()
    t.cuda.synchronize()
    want = out[0].clone()
    s, stop, errors = t.cuda.Stream(), threading.Event(), []

    def work():
        try:
            while not stop.is_set():
                run(stream=s.cuda_stream)
        except Exception as e:
            errors.append(repr(e))

    th = threading.Thread(target=work)
    th.start()
    for _ in range(20):
        g.release()
    stop.set()
    th.join()
    t.cuda.synchronize()
    assert not errors, errors
    assert g.debug_status() == 0 and t.equal(want, out[0])


def test_counters_that_grow_start_at_zero():
    """Tiles' arrival counters: a call with more split tiles than the first buffer
    has counters for, after one whose counts that buffer held (the larger buffer
    may lie at the same address)."""
    import dense_gemm_03_gb300 as g
    t = torch()
    g.release()
    s = t.cuda.Stream()
    prev, prev_splits = g.force_path(g.PATH_SPLITK), g.force_splits(2)
    K = 128
    try:
        for M, N in ((256, 256), (64, 256 * 16400), (256, 512)):
            gen = t.Generator(device="cuda").manual_seed(M + N)
            A, B = (t.randint(-1, 2, shape, generator=gen, device="cuda", dtype=t.float16)
                    for shape in ((M, K), (K, N)))
            C = t.full((M, N), float("nan"), dtype=t.float16, device="cuda")
            t.cuda.synchronize()
            g.gemm_f16(A, B, C, stream=s)
            assert ".splitk" in g.last_path()
            s.synchronize()
            assert g.debug_status() == 0
            cols = t.randint(0, N, (512,), generator=gen, device="cuda")
            want = A.float() @ B[:, cols].float()
            assert t.equal(C[:, cols], want.half()) and not C.isnan().any()
    finally:
        g.force_path(prev)
        g.force_splits(prev_splits)
        g.release()
