"""Which rows the experts of a grouped product get from bounds that may be anything
(CPU only): within 0 .. R, none with two experts, and as they are where the bounds
are in order.  The code is the kernel's own (grouped_plan.h), compiled here as host
code by nvcc; nothing runs on a GPU."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "fp8_w8a8_quantized_gb300", "csrc")

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>
#include "grouped_plan.h"
using namespace fp8k::grouped;

int main() {
    std::mt19937 rng(5);
    int fails = 0, went_back = 0, in_order = 0;
    for (int round = 0; round < 20000; ++round) {
        const int E = 1 + rng() % 12, R = rng() % 4 ? rng() % 100 : 1 << 30;
        std::vector<int> off(E + 1);
        for (int& o : off) {
            o = static_cast<int>(rng() % (R + 1u));
            if (rng() % 8 == 0) o = static_cast<int>(rng());           // any number
            if (rng() % 16 == 0) o = rng() % 2 ? 2147483647 : -2147483647 - 1;
        }
        if (round % 3 == 0) std::sort(off.begin(), off.end());
        // each bound cut to 0 .. R, then the largest up to it
        std::vector<int> want(E + 1);
        int most = 0;
        for (int e = 0; e <= E; ++e) want[e] = most = std::max(most, std::min(std::max(off[e], 0), R));
        std::vector<int> begin(E), end(E);
        bool back = false;
        for (int e = 0; e < E; ++e) {
            const Bounds b = bounds_within(off[e], off[e + 1], R);
            begin[e] = b.begin, end[e] = b.end;
            back |= b.back;
            if (b.begin < 0 || b.end < b.begin || b.end > R) ++fails;
        }
        if (back) ++went_back, put_in_order(begin.data(), end.data(), E);
        else ++in_order;
        for (int e = 0; e < E; ++e)
            if (begin[e] != want[e] || end[e] != want[e + 1]) {
                if (++fails < 10) std::printf("expert %d: %d-%d, not %d-%d\n", e, begin[e], end[e], want[e], want[e + 1]);
            }
    }
    std::printf("%d went back, %d in order, %d fails\n", went_back, in_order, fails);
    return fails != 0 || went_back < 1000 || in_order < 1000;
}
"""


def test_no_row_has_two_experts(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("needs nvcc")
    src, exe = tmp_path / "bounds.cu", tmp_path / "bounds"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
