"""Clusters whose CTAs hold tensor memory have their SMs to themselves: beside another
such cluster on the same SMs, each could wait for the other's tensor memory for ever."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_gemm_03_gb300", "csrc")


def text(name):
    return open(os.path.join(CSRC, name)).read()


def test_clusters_take_all_shared_memory():
    t = text("narrow.cuh")
    assert re.search(r"cfg\.dynamicSmemBytes = chunks > 1 \? kSmemMax : smem;", t)
    # 228 KB of an SM, less 1 KB that the system takes of every CTA's
    assert int(re.search(r"kSmemMax = (\d+)", t).group(1)) == 228 * 1024 - 1024
    for name in ("narrow_stream.cu", "i8_stream.cu"):
        assert "cudaLaunchKernel" not in text(name) and "launch_narrow(" in text(name)
