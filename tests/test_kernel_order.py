"""Kernels that allocate tensor memory let their dependents start only after
they have it: a dependent that shares the SM holds its own until the first kernel
ends, and the first would wait for it without limit."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_gemm_03_gb300", "csrc")


def kernels():
    """(file, name, body) of every __global__ function."""
    for f in sorted(os.listdir(CSRC)):
        if not f.endswith((".cu", ".cuh")):
            continue
        text = open(os.path.join(CSRC, f)).read()
        starts = [m.start() for m in re.finditer(r"__global__\s", text)]
        for a in starts:
            end = text.find("\n}\n", a)
            name = re.search(r"(\w+_kernel)\s*\(", text[a:])
            yield f, name.group(1), text[a:end]


def test_kernels_are_found():
    names = {n for _, n, _ in kernels()}
    assert {"gemm_f16_tc_kernel", "lora_shrink_tc_kernel", "row_stream_kernel", "lora_outer_kernel",
            "moe_stream_kernel"} <= names


@pytest.mark.parametrize("f,name,body", [pytest.param(*k, id=k[1]) for k in kernels()
                                         if "tmem_alloc" in k[2]])
def test_tensor_memory_before_dependents(f, name, body):
    alloc = body.rindex("tmem_alloc")
    for m in re.finditer(r"griddep_launch_dependents\(\)", body):
        line = body[body.rfind("\n", 0, m.start()) + 1:m.start()]
        # blocks without tensor memory may announce at once
        assert m.start() > alloc or line.strip().startswith("if (b >= p.first_list)"), (f, name)
