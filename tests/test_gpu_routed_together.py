"""The row-routed products together: the example program, and calls of several
operators on two streams at once."""
import importlib.util
import os

import pytest

from helpers import torch
from test_gpu_lora import operands as lora_operands
from test_gpu_moe import operands as moe_operands

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_03_gb300 import build
    build.build()


def test_example():
    spec = importlib.util.spec_from_file_location(
        "adapters_and_experts", os.path.join(ROOT, "examples", "adapters_and_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main()
    # both ways round the same hidden rows to half once per operator: a few
    # units in the last place of values of at most about 16
    assert r["same_experts"] >= 2 and r["decode_difference"] <= 4 * 16 * 2.0 ** -10
    assert r["loss_after"] < 0.2 * r["loss_before"]


@pytest.mark.parametrize("M,T", [(2, 3), (64, 16), (700, 64)])
def test_two_streams_at_once(M, T):
    """Calls whose kernels share the SMs give the bits they give alone (a
    mixture-of-experts kernel waits for its own other thread blocks, which may
    not all be running)."""
    import dense_gemm_03_gb300 as g
    t = torch()
    lo = {k: v.cuda() for k, v in lora_operands(t, 41, M, 1024, 2048, 16, 6, "mixed").items()}
    mo = {k: v.cuda() for k, v in moe_operands(t, 42, T, 1024, 512, 16).items()}

    def lora(C, dX, dA, dB):
        g.gemm_f16_lora(lo["X"], lo["W"], C, lo["A"], lo["B"], lo["ids"], lo["scales"])
        g.gemm_f16_lora_grad(lo["G"], lo["X"], lo["W"], lo["A"], lo["B"], lo["ids"], lo["scales"],
                             dX, dA, dB)

    def moe(Y):
        g.gemm_f16_moe(mo["X"], mo["Wr"], mo["W1"], mo["W2"], Y, 4)

    def lora_outs():
        return [t.full_like(lo[k], float("nan")) for k in ("C0", "X", "dA0", "dB0")]

    alone, Y = lora_outs(), t.empty_like(mo["Y0"])
    lora(*alone)
    moe(Y)
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in range(3)]
    got = [lora_outs() for _ in range(8)]
    ys = [[t.full_like(Y, float("nan")) for _ in range(8)] for _ in range(2)]
    for i in range(8):
        for j, s in enumerate(streams):
            with t.cuda.stream(s):
                lora(*got[i]) if j == 0 else moe(ys[j - 1][i])
    t.cuda.synchronize()
    assert g.debug_status() == 0
    for i in range(8):
        assert all(t.equal(a, b) for a, b in zip(alone, got[i]))
        assert t.equal(Y, ys[0][i]) and t.equal(Y, ys[1][i])


def test_release_frees_the_scratch_and_calls_work_after():
    import dense_gemm_03_gb300 as g
    t = torch()
    lo = {k: v.cuda() for k, v in lora_operands(t, 43, 300, 512, 256, 16, 4, "runs").items()}
    C, D = t.empty_like(lo["C0"]), t.empty_like(lo["C0"])
    g.gemm_f16_lora(lo["X"], lo["W"], C, lo["A"], lo["B"], lo["ids"], lo["scales"])
    g.release()
    g.gemm_f16_lora(lo["X"], lo["W"], D, lo["A"], lo["B"], lo["ids"], lo["scales"])
    t.cuda.synchronize()
    assert g.debug_status() == 0 and t.equal(C, D)
