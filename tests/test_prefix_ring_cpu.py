"""The shared-prefix kernel's order of reads and writes, on the host.

A CTA's warps meet at barriers only, so whether a place in shared memory may be
written again follows from what the barriers order.  The model below has an
event for every read and write of the key and value ring and of the words that
say which tokens exist, an edge for every wait and every step of a warp, and
asks for each place that all reads of what it holds come before the next write.
Indices and plan are the kernel's own (attention_plan.h, compiled here)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT
from test_gpu_attention_prefix import CASES

CSRC = os.path.join(ROOT, "fp8_w8a8_quantized_gb300", "csrc")
LOAD_WARPS = 7
PROGRAM = r"""
#include "attention_plan.h"
using namespace fp8k;
extern "C" {
int stages() { return kPrefixStages; }
int key(int j) { return key_stage(j); }
int value(int j) { return value_stage(j); }
int there(int j) { return there_row(j); }
void plan(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t prefix, int64_t* out) {
    const PrefixPlan p = prefix_plan(B, Hq, Hkv, D, prefix);
    out[0] = p.splits, out[1] = p.cluster, out[2] = p.tiles, out[3] = p.row_blocks, out[4] = p.parts_bytes();
}
}
"""


@pytest.fixture(scope="module")
def P(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cpp", d / "plan.so"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    got = ctypes.CDLL(str(lib))
    got.plan.argtypes = [ctypes.c_int64] * 5 + [ctypes.POINTER(ctypes.c_int64)]
    return got


def plan_of(P, B, Hq, Hkv, D, prefix):
    out = (ctypes.c_int64 * 5)()
    P.plan(B, Hq, Hkv, D, prefix, out)
    return dict(zip(("splits", "cluster", "tiles", "row_blocks", "bytes"), out))


class Order:
    """Events in the order in which they are added; after(e): all that come before e."""

    def __init__(self):
        self.index, self.before = {}, []

    def add(self, event, *earlier):
        mask = 0
        for e in earlier:
            i = self.index[e]
            mask |= self.before[i] | 1 << i
        self.index[event] = len(self.before)
        self.before.append(mask)

    def ordered(self, a, b):
        return bool(self.before[self.index[b]] >> self.index[a] & 1)


def events(tiles, query_tiles, stages):
    """The kernel's events for that many key tiles: load(m, q) writes 32 tokens of ring tile m (2 j: keys of
    key tile j, 2 j + 1: values) and, of keys, their word; read(x, j): softmax of query tile x reads the words;
    s(x, j), pv(x, j): the MMAs are complete."""
    o = Order()
    last = {}  # of each load warp

    def load(m):
        for q in range(4):
            warp = (4 * m + q) % LOAD_WARPS
            earlier = [last[warp]] if warp in last else []
            if m >= stages:
                earlier.append(("free", m - stages))
            o.add(("load", m, q), *earlier)
            last[warp] = ("load", m, q)

    def landed(m):
        return [("load", m, q) for q in range(4)]

    loaded = 0

    def load_upto(m):
        nonlocal loaded
        while loaded <= min(m, 2 * tiles - 1):
            load(loaded)
            loaded += 1

    load_upto(stages - 1)
    issued = []  # what the issuer has seen or done
    for j in range(tiles + 1):
        if j < tiles:
            issued += landed(2 * j)
        for x in range(query_tiles):
            if j > 0:
                issued.append(("p", x, j - 1))
                o.add(("pv", x, j - 1), *issued)
            if j < tiles:
                o.add(("s", x, j), *issued)
        for x in range(query_tiles):
            if j < tiles:
                o.add(("read", x, j), ("s", x, j), *([("p", x, j - 1)] if j else []))
                o.add(("p", x, j), ("read", x, j))
        # (a commit is behind all MMAs that were issued before it)
        if j > 0:
            o.add(("free", 2 * j - 1), *[("pv", x, j - 1) for x in range(query_tiles)],
                  *[("s", x, j) for x in range(query_tiles) if j < tiles])
        if j < tiles:
            o.add(("free", 2 * j), *[("s", x, j) for x in range(query_tiles)],
                  *[("pv", x, j - 1) for x in range(query_tiles) if j > 0])
        if j < tiles:
            load_upto(2 * j + stages)
            issued += landed(2 * j + 1)
    return o


def word_faults(o, tiles, query_tiles, row):
    """Reads of a key tile's words that a later key tile's write of the same place may overtake."""
    return [(j, k) for j in range(tiles) for k in range(j + 1, tiles) if row(j) == row(k)
            for x in range(query_tiles) for q in range(4)
            if not o.ordered(("read", x, j), ("load", 2 * k, q))]


@pytest.mark.parametrize("query_tiles", [1, 2])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 5, 8, 13])
def test_nothing_is_written_while_it_is_read(P, tiles, query_tiles):
    stages = P.stages()
    o = events(tiles, query_tiles, stages)
    for j in range(tiles):
        assert P.key(j) == 2 * j % stages and P.value(j) == (2 * j + 1) % stages  # (as the barriers' phases count)
        for x in range(query_tiles):
            for q in range(4):
                assert o.ordered(("load", 2 * j, q), ("read", x, j))
                assert o.ordered(("load", 2 * j + 1, q), ("pv", x, j))
    for m in range(2 * tiles - stages):
        for x in range(query_tiles):
            for q in range(4):
                done = ("pv", x, m // 2) if m % 2 else ("s", x, m // 2)
                assert o.ordered(done, ("load", m + stages, q))
    assert not word_faults(o, tiles, query_tiles, P.there)


@pytest.mark.parametrize("query_tiles", [1, 2])
def test_the_model_sees_words_that_are_overtaken(P, query_tiles):
    # words kept by ring stage are written again when the keys are read, not when the words are
    o = events(6, query_tiles, P.stages())
    assert word_faults(o, 6, query_tiles, lambda j: 2 * j % P.stages())
    assert not word_faults(o, 2, query_tiles, lambda j: 2 * j % P.stages())


def test_the_gpu_cases_go_round_the_ring(P):
    """The GPU tests' cases use the kernel and wait for free stages: three key tiles a CTA or more, in the last
    part as well as in the others, with one and with two query tiles, in clusters of every size."""
    seen = set()
    for B, Hq, Hkv, D, page, prefix in CASES:
        p = plan_of(P, B, Hq, Hkv, D, prefix)
        assert p["splits"] > 0 and p["tiles"] >= 3, (B, Hq, Hkv, D, prefix, p)
        assert p["splits"] % p["cluster"] == 0 and p["bytes"] > 0
        tpt = 128 // (Hq // Hkv)
        seen.add((p["cluster"], B > tpt, D > 64, prefix % 128 != 0))
    assert {c for c, *_ in seen} == {1, 2, 4}
    assert {(two, wide) for _, two, wide, _ in seen} == {(a, b) for a in (False, True) for b in (False, True)}


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (8, 8, 64), (64, 1, 112), (14, 2, 64), (6, 3, 80)])
def test_the_plan_covers_the_prefix(P, Hq, Hkv, D):
    for B in (1, 2, 3, 17, 64, 130, 1000):
        for prefix in (0, 1, 127, 128, 129, 700, 4001, 8200, 32768, 100001):
            p = plan_of(P, B, Hq, Hkv, D, prefix)
            if p["splits"] == 0:
                assert p["bytes"] == 0
                continue
            tiles = -(-prefix // 128)
            assert p["splits"] * p["tiles"] >= tiles and p["splits"] % p["cluster"] == 0
            assert (p["splits"] - p["cluster"]) * p["tiles"] < tiles  # no cluster without tokens
            assert 2 * (128 // (Hq // Hkv)) * p["row_blocks"] >= B
            assert p["bytes"] == p["splits"] // p["cluster"] * B * Hq * ((64 if D <= 64 else 128) * 4 + 8)
