"""Kernels that allocate tensor memory let the next kernel on the stream start
only once they have it.  An allocation waits, without a limit, until its columns
are free; a successor that got on the SM before that could take them, and would
then wait for the very kernel that waits for it.  Read from the sources: the
order of the three steps in each kernel's prologue."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "fp8_w8a8_quantized_gb300", "csrc")
STEP = re.compile(r"\btmem_alloc(?:_pair)?\(|\bpdl_launch_dependents\(\)|\b__syncthreads\(\)")


def prologues(text):
    """The steps of each kernel from its allocation to its launch of dependents, and what lies before it."""
    kernels = re.split(r"__global__", re.sub(r"//[^\n]*", "", text))[1:]
    for k in kernels:
        steps = [m.group().split("(")[0].replace("_pair", "") for m in STEP.finditer(k)]
        if "tmem_alloc" in steps and "pdl_launch_dependents" in steps:
            yield steps[: steps.index("pdl_launch_dependents") + 1]


@pytest.mark.parametrize("name", ["attention_prompt.cu", "attention_prefix.cu", "gemm_pair.cu", "gemm_decode.cu",
                                  "gemm_blockwise.cu"])
def test_successors_start_behind_the_allocation(name):
    with open(os.path.join(CSRC, name)) as f:
        found = list(prologues(f.read()))
    assert found, name
    for steps in found:
        assert steps[-3:] == ["tmem_alloc", "__syncthreads", "pdl_launch_dependents"], (name, steps)


def test_every_kernel_with_tensor_memory_is_looked_at():
    users = {f for f in os.listdir(CSRC) if f.endswith(".cu")
             and re.search(r"\btmem_alloc(_pair)?\(", open(os.path.join(CSRC, f)).read())}
    assert users - {"selftest.cu"} == {"attention_prompt.cu", "attention_prefix.cu", "gemm_pair.cu", "gemm_decode.cu",
                                       "gemm_blockwise.cu"}
