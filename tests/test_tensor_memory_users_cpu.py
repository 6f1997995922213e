"""Every kernel that allocates tensor memory, by whatever helper, lets the next
kernel on the stream start only once it has it: an allocation waits without a
limit, and a successor that took the columns would then wait for this kernel.
The helpers are found in the sources, so that a new one cannot be missed."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "fp8_w8a8_quantized_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def functions(text):
    """(name, body) of the functions of a header."""
    for m in re.finditer(r"__device__ __forceinline__ [\w:<>*& ]+?\b(\w+)\(", text):
        begin = text.index("{", m.end())
        depth, end = 1, begin + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield m.group(1), text[begin:end]


def allocating(texts):
    """Names of all functions that allocate, themselves or through another."""
    bodies = [f for t in texts for f in functions(t)]
    names = {n for n, body in bodies if "tcgen05.alloc" in body}
    while True:
        more = {n for n, body in bodies if any(re.search(rf"\b{a}\b\s*[<(]", body) for a in names)}
        if more <= names:
            return names
        names |= more


def order_of(kernel, names):
    """Allocations, barriers and launches of dependents of a kernel in the order of its text."""
    calls = "|".join(sorted(names))
    step = re.compile(rf"\b(?:{calls})(?:<[^<>()]*>)?\(|\bpdl_launch_dependents\(|\b__syncthreads\(")
    return [m.group().rstrip("(").split("<")[0] for m in step.finditer(kernel)]


def check(texts, kernels_of):
    names = allocating(texts)
    users = set()
    for file, text in kernels_of.items():
        for kernel in re.split(r"__global__", text)[1:]:
            steps = order_of(kernel, names)
            taken = [i for i, s in enumerate(steps) if s in names]
            if not taken:
                continue
            users.add(file)
            if "pdl_launch_dependents" not in steps:
                continue
            launch = steps.index("pdl_launch_dependents")
            assert max(taken) < launch, (file, steps)
            assert steps[launch - 2] in names and steps[launch - 1] == "__syncthreads", (file, steps)
    return names, users


def test_successors_start_behind_every_allocation():
    headers = [f for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    kernels = [f for f in os.listdir(CSRC) if f.endswith(".cu")]
    names, users = check([source(f) for f in headers + kernels], {f: source(f) for f in kernels})
    assert {"tmem_alloc", "tmem_alloc_pair", "tmem_take"} <= names
    assert users == {"attention_prompt.cu", "attention_prefix.cu", "gemm_pair.cu", "gemm_decode.cu", "gemm_blockwise.cu",
                     "gemm_grouped.cu", "selftest.cu"}
    for f in kernels:
        assert "tcgen05.alloc" not in source(f), f


def test_a_helper_over_helpers_is_found():
    header = """
    __device__ __forceinline__ void low(int n) { asm volatile("tcgen05.alloc.x"); }
    template <bool kPair>
    __device__ __forceinline__ void high(int n) { if (n) { low(n); } }
    __device__ __forceinline__ void other(int n) { n += 1; }
    """
    good = "__global__ void k() { high<true>(4); __syncthreads(); pdl_launch_dependents(); }"
    assert check([header], {"good.cu": good}) == ({"low", "high"}, {"good.cu"})
    for bad in ("__global__ void k() { pdl_launch_dependents(); high<true>(4); __syncthreads(); }",
                "__global__ void k() { high<false>(4); pdl_launch_dependents(); __syncthreads(); }",
                "__global__ void k() { low(4); __syncthreads(); pdl_launch_dependents(); high<true>(4); }"):
        with pytest.raises(AssertionError):
            check([header], {"bad.cu": bad})
