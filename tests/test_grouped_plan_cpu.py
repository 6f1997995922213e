"""How the workers of a grouped product share its tiles (CPU only): every stage of
every tile belongs to exactly one worker, a worker has at most one piece that
begins and one that ends a cut tile, and the workers of a cut tile are the ones
that the kernel counts.  The code is the kernel's own (grouped_plan.h), compiled
here as host code by nvcc; nothing runs on a GPU."""
import os
import re
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "fp8_w8a8_quantized_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "grouped_plan.h"
using namespace fp8k::grouped;

static int fails = 0, cut = 0;
#define CHECK(c, ...) do { if (!(c)) { if (++fails < 20) { std::printf(__VA_ARGS__); std::printf("\n"); } } } while (0)

static void check(int tiles, int n, int nk, Costs costs) {
    std::vector<int> done(tiles, 0);                  // stages of a tile so far, by the workers in order
    std::vector<int> begun(n, 0), ended(n, 0);
    std::vector<std::vector<int>> of(tiles);          // workers of a tile
    int64_t most = 0, least = int64_t(1) << 60;
    for (int w = 0; w < n; ++w) {
        Walk walk(tiles, n, w, nk, costs);
        int64_t mine = 0;
        bool parts = false;
        while (walk.advance()) {
            CHECK(walk.tile >= 0 && walk.tile < tiles, "tile %d of %d", walk.tile, tiles);
            CHECK(walk.kb0 >= 0 && walk.kb0 < walk.kb1 && walk.kb1 <= nk, "stages %d-%d", walk.kb0, walk.kb1);
            const bool whole = walk.kb0 == 0 && walk.kb1 == nk;
            CHECK(whole || walk.tile >= walk.whole, "part of a whole tile");
            CHECK(walk.kb0 == done[walk.tile], "tile %d: stage %d after %d", walk.tile, walk.kb0, done[walk.tile]);
            done[walk.tile] = walk.kb1;
            of[walk.tile].push_back(w);
            if (walk.tile >= walk.whole) {
                parts = true;
                mine += walk.kb1 - walk.kb0;
                if (!whole) {
                    // where the part goes in the workspace: two slots a worker
                    if (walk.kb0 == 0) ++begun[w];
                    else ++ended[w];
                    const int64_t unit = static_cast<int64_t>(walk.tile - walk.whole) * nk;
                    CHECK(walk.worker_of(unit + walk.kb0) == w && walk.worker_of(unit + walk.kb1 - 1) == w,
                          "worker %d has stages of %d and %d", w, walk.worker_of(unit + walk.kb0),
                          walk.worker_of(unit + walk.kb1 - 1));
                }
            }
        }
        CHECK(begun[w] <= 1 && ended[w] <= 1, "worker %d: %d parts begin, %d go on", w, begun[w], ended[w]);
        if (walk.units && parts) {
            most = mine > most ? mine : most;
            least = mine < least ? mine : least;
        }
    }
    Walk walk(tiles, n, 0, nk, costs);
    if (walk.units) {
        ++cut;
        CHECK(most - least <= 1, "shares of %lld to %lld stages", (long long)least, (long long)most);
        for (int t = walk.whole; t < tiles; ++t) {
            const int64_t unit = static_cast<int64_t>(t - walk.whole) * nk;
            const int first = walk.worker_of(unit), last = walk.worker_of(unit + nk - 1);
            CHECK((int)of[t].size() == last - first + 1 && of[t].front() == first && of[t].back() == last,
                  "tile %d: %d workers from %d to %d, counted %d to %d", t, (int)of[t].size(), of[t].front(),
                  of[t].back(), first, last);
        }
    }
    for (int t = 0; t < tiles; ++t) CHECK(done[t] == nk, "tile %d of %d: %d of %d stages", t, tiles, done[t], nk);
}

int main() {
    const Costs some[] = {{0.44f, 0.0054f, 3.0f, 0.9f}, {0.44f, 0.0054f, 3.0f, 3.6f}, {0.3f, 0.0f, 3.0f, 7.2f},
                          {1.0f, 0.0f, 0.0f, 0.01f}};
    for (const Costs& c : some)
        for (int n : {1, 2, 7, 75, 76, 148, 152})
            for (int nk : {1, 2, 3, 11, 32, 112, 1000})
                for (int tiles : {0, 1, 2, 3, 16, 32, 75, 76, 77, 151, 152, 153, 224, 300, 700}) check(tiles, n, nk, c);
    check(40, 152, 1 << 23, some[0]);  // (stages that pass 2^31 in all)
    CHECK(cut > 100, "%d lists cut", cut);
    std::printf("%d lists cut, %d fails\n", cut, fails);
    return fails != 0;
}
"""


def test_every_stage_has_one_worker(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("needs nvcc")
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, "-O2", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_successors_start_behind_the_allocation_of_tensor_memory():
    # (an allocation waits without a limit: a successor that got on the SM before it could take the
    # columns, and would then wait for this kernel)
    with open(os.path.join(CSRC, "gemm_grouped.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = 0
    for kernel in re.split(r"__global__", text)[1:]:
        steps = re.findall(r"\btmem_take<|\bpdl_launch_dependents\(\)|\b__syncthreads\(\)", kernel)
        if "tmem_take<" in steps:
            found += 1
            assert steps[: steps.index("pdl_launch_dependents()") + 1] == [
                "tmem_take<", "__syncthreads()", "pdl_launch_dependents()"]
    assert found == 1
