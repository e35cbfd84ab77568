"""How the gated feed-forward product is cut (CPU only).  The library's own planning code, which needs no CUDA, is compiled into a
small program that prints its plans; they are checked over the sizes that the entry points accept: every launch fits a grid,
every part of a sum is there and none is empty, and the workspace holds what the plan puts there."""
import json
import os
import random
import shutil
import subprocess

import pytest

from neighborhood_attention_fwd_gb300 import build as nabuild

BF16, FP32, FP16 = 0, 1, 2
ROWS, WIDTH, ELEMENTS = 2 ** 31 - 256, 2 ** 20, 2 ** 40   # what the entry points accept

PROGRAM = r"""
#include <cstdio>
#include "na_glu_plan.h"
using namespace na::glu;
static void fma(const char* name, Product which, long long T, int D, int F, const FmaTile& t) {
    const FmaGrid g = fma_grid(which, T, D, F, t);
    std::printf(", \"%s\": {\"rows\": %d, \"cols\": %d, \"splits\": %d, \"run\": %lld, \"grid\": [%u, %u, %u]}", name, t.rows, t.cols, t.splits, t.run, g.x, g.y, g.z);
}
static void tiles(const char* name, const GluTiles& t) {
    std::printf(", \"%s\": {\"pairs\": %d, \"few\": %d, \"rows\": %u, \"cols\": %u, \"steps\": %u, \"run\": %u, \"splits\": %u, \"ways\": %u, \"last_nf\": %u, \"span\": %u, \"groups\": %u, \"workers\": %u}",
                name, t.pairs, t.few, t.rows, t.cols, t.steps, t.run, t.splits, t.ways, t.last_nf, t.span, t.groups, t.workers);
}
int main() {
    long long T;
    int D, F, type;
    while (std::scanf("%lld %d %d %d", &T, &D, &F, &type) == 4) {
        const na_dtype dt = static_cast<na_dtype>(type);
        const GluPlan n = plan_glu(T, D, F, dt);
        std::printf("{\"tensor\": %d, \"width\": %d, \"pitch\": %lld, \"array\": %zu, \"sum_rows\": %lld, \"sum_pitch\": %d, \"sums\": %zu, \"runs\": %d, \"column_run\": %lld, \"partial\": %zu, \"workspace\": %zu",
                    n.tensor, n.width, n.pitch, n.array, n.sum_rows, n.sum_pitch, n.sums, n.runs, n.column_run, n.partial, glu_workspace(n));
        if (n.tensor) {
            tiles("forward", plan_tiles(kForward, T, n.width, F));
            tiles("slopes", n.slopes);
            tiles("tokens", n.tokens);
            tiles("weights", n.weights);
        } else {
            fma("forward", kForward, T, D, F, plan_fma(kForward, T, D, F));
            fma("slopes", kSlopes, T, D, F, n.slopes_fma);
            fma("tokens", kTokens, T, D, F, n.tokens_fma);
            fma("weights", kWeights, T, D, F, n.weights_fma);
        }
        std::printf("}\n");
    }
}
"""


@pytest.fixture(scope="session")
def planner(tmp_path_factory):
    """A function from [(T, D, F, type)] to the plans."""
    compiler = shutil.which("g++") or shutil.which("c++")
    if compiler is None:
        pytest.skip("no C++ compiler")
    here = tmp_path_factory.mktemp("plan")
    src, exe = str(here / "plan.cpp"), str(here / "plan")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run([compiler, "-std=c++17", "-O2", "-Wall", "-I" + nabuild.CSRC, "-I" + os.path.join(nabuild.ROOT, "include"), src, "-o", exe], check=True)

    def plans(sizes):
        r = subprocess.run([exe], input="".join("%d %d %d %d\n" % s for s in sizes), capture_output=True, text=True, check=True)
        return [json.loads(line) for line in r.stdout.splitlines()]

    return plans


def up(a, b):
    return -(-a // b)


def accepted(T, D, F):
    return 1 <= T <= ROWS and 1 <= D <= WIDTH and 1 <= F <= WIDTH and T * max(D, F) <= ELEMENTS


def sizes(n, seed=7):
    rng = random.Random(seed)
    out = []
    while len(out) < n:
        T, D, F = (max(1, int(2 ** rng.uniform(0, top))) for top in (31, 20, 20))
        T = rng.choice([T, T, ROWS, T // 64 * 64 + 1])
        if accepted(T, D, F):
            out.append((T, D, F, rng.choice([BF16, FP32, FP16])))
    return out


def check(size, p):
    T, D, F, dtype = size
    D = p["width"]
    es = 4 if dtype == FP32 else 2
    chunk = 16 // es
    assert p["pitch"] == up(F, chunk) * chunk and p["array"] >= T * p["pitch"] * es
    assert p["workspace"] >= 2 * p["array"] + p["partial"]
    # dbg and dbu: rows of sums over a tile's tokens, then runs of those rows, then the runs; no sum takes more than 8192 terms
    rows = up(T, p["slopes"]["rows"]) if not p["tensor"] else 1 if p["slopes"]["few"] else up(T, 32)
    assert p["sum_rows"] == rows and p["sum_pitch"] % 4 == 0 and F <= p["sum_pitch"] < F + 4
    assert 0 < (p["runs"] - 1) * p["column_run"] + 1 <= rows <= p["runs"] * p["column_run"] and p["column_run"] <= 8192 and p["runs"] <= 8192
    assert p["sums"] % 256 == 0 and p["sums"] >= 4 * rows * 2 * p["sum_pitch"] and p["partial"] >= p["sums"] + 4 * p["runs"] * 2 * F
    for name, size_ in (("tokens", T * D), ("weights", 2 * F * D)):
        if p[name]["splits"] > 1:
            assert p["partial"] >= 4 * p[name]["splits"] * size_
    if not p["tensor"]:
        for name in ("forward", "slopes", "tokens", "weights"):
            x, y, z = p[name]["grid"]
            assert 1 <= x < 2 ** 31 and 1 <= y <= 65535 and 1 <= z <= 65535, name
        pieces = 2 * up(F, 16)
        for name, n in (("tokens", pieces), ("weights", T)):
            t = p[name]
            assert (t["splits"] - 1) * t["run"] < n <= t["splits"] * t["run"], name
            assert t["run"] * (16 if name == "tokens" else 1) <= 8192   # products in one sum
        for name in ("forward", "slopes"):   # more than 8192 channels: kernels that add up runs of them
            assert D <= 8192 or p[name]["rows"] == p[name]["cols"]
        x, _, z = p["weights"]["grid"]
        tiles = up(F, p["weights"]["rows"])
        assert x % tiles == 0 and z % 2 == 0 and (x // tiles) * (z // 2) >= p["weights"]["splits"]   # places of the splits
        return
    assert D % 8 == 0
    for name in ("forward", "slopes"):
        t = p[name]
        if t["few"]:
            assert T <= t["few"] and t["rows"] * 64 >= F and (t["splits"] - 1) * t["run"] < t["steps"] <= t["splits"] * t["run"]
            continue
        m = 256 if t["pairs"] else 128
        assert t["rows"] == up(T, m) and t["cols"] == up(F, m // 2) and t["groups"] == up(t["cols"], t["span"]) and t["rows"] * t["groups"] < 2 ** 31
        assert 0 < F - (t["cols"] - 1) * (m // 2) <= t["last_nf"] <= m // 2 and t["last_nf"] % (16 if t["pairs"] else 8) == 0
        assert t["steps"] == up(D, 64) and (t["span"] == 1 or t["steps"] <= (6 if name == "forward" else 5))
    for name in ("tokens", "weights"):
        t = p[name]
        m = 256 if t["pairs"] else 128
        assert t["rows"] == (2 * up(F, m) if name == "weights" else up(T, m)) and t["cols"] == up(D, m)
        assert t["steps"] == (up(T, 64) if name == "weights" else 2 * up(F, 64))
        turns, rest = divmod(t["splits"], t["ways"])
        assert rest == 0 and t["run"] <= 384   # 24576 products in one accumulator
        # part w + ways t takes the steps w + ways (t run + j), j < run: all of them, and none is empty
        least, most = t["steps"] // t["ways"], up(t["steps"], t["ways"])
        assert (turns - 1) * t["run"] < least and turns * t["run"] >= most
    if p["tokens"]["workers"]:
        t, w = p["tokens"], p["weights"]
        assert t["pairs"] and w["pairs"] and t["splits"] == 1
        assert 0 < t["workers"] < 76 and 76 - t["workers"] == w["ways"] * w["rows"] * w["cols"]


def test_plans_of_accepted_sizes(planner):
    some = sizes(4000)
    some += [(T, D, F, t) for t in (BF16, FP32, FP16) for T in (1, 16, 17, 128, 129, 4097) for D in (1, 8, 63, 1000, 65536) for F in (1, 8, 100, 2001)]
    for size, p in zip(some, planner(some)):
        try:
            check(size, p)
        except AssertionError as e:
            raise AssertionError(f"{size}: {p}") from e
