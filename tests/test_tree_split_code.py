"""How the CTAs are divided between pairs and single items of trees, and what an item
costs (csrc/attention_plan.cuh, compiled for the host): both kinds get CTAs, the slower
kind of the chosen division is no slower than of any other, workspaces hold the pieces."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from w4a16_moe_expert_sync_gb300 import build

SOURCE = """
#include "attention_plan.cuh"
using namespace w4::plan;
extern "C" {
int c_ctas(int singles, int pairs, int grid) { return tree_pair_ctas(singles, pairs, grid); }
int c_cost(int tree, int pair) { return item_cost(tree, pair); }
int c_begin(int all, int workers, int w) { return worker_begin(all, workers, w); }
int c_of(int all, int workers, int x) { return worker_of(all, workers, x); }
double c_weight() { return kTreeSingleWeight; }
}
"""


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("split")
    (d / "s.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC,
                    str(d / "s.cpp"), "-o", str(d / "s.so")], check=True)
    lib = ctypes.CDLL(str(d / "s.so"))
    lib.c_weight.restype = ctypes.c_double
    return lib


def test_the_kernel_runs_this_code():
    with open(os.path.join(build.CSRC, "attention.cu")) as f:
        text = f.read()
    assert "plan::tree_pair_ctas(" in text and "item_cost(TREE, " in text


def test_costs(code):
    assert code.c_cost(0, 0) == code.c_cost(0, 1) == code.c_cost(1, 0) == 2
    assert code.c_cost(1, 1) == 5


@pytest.mark.parametrize("seed", range(40))
def test_division(code, seed):
    r = random.Random(seed)
    weight = code.c_weight()
    for _ in range(300):
        singles, pairs = (r.choice([0, 1, 3, r.randint(1, 300), r.randint(1, 10 ** 5), 10 ** 7])
                          for _ in range(2))
        grid = r.choice([2, 3, 7, 148, 152, 256])
        n = code.c_ctas(singles, pairs, grid)
        assert 0 <= n <= min(pairs, grid) and (n > 0) == (pairs > 0)
        assert singles == 0 or grid - n > 0
        if not singles or not pairs or n == pairs:
            continue

        def slower(ctas):
            return max(pairs / ctas, weight * singles / (grid - ctas))
        best = min(slower(x) for x in range(1, grid))
        # the quotients are 32-bit ones: 2^-22 between two alike
        assert slower(n) <= best * (1 + 2.0 ** -22), (singles, pairs, grid, n)


@pytest.mark.parametrize("seed", range(40))
def test_items_are_cut_into_pieces(code, seed):
    """Every tile of every item is in one worker's piece, whatever the item's cost."""
    r = random.Random(seed)
    for pair in (0, 1):
        cost = code.c_cost(1, pair)
        spans = [cost + r.choice([1, 2, 3, 40]) for _ in range(r.choice([1, 3, 60, 700]))]
        total = sum(spans)
        workers = min(total, r.choice([1, 2, 7, 151, 302]))
        at, places = 0, set()
        for number, span in enumerate(spans):
            got = []
            for w in range(code.c_of(total, workers, at), code.c_of(total, workers, at + span - 1) + 1):
                assert number + w not in places            # pieces are numbered by item + worker
                places.add(number + w)
                lo, hi = (code.c_begin(total, workers, x) - at - cost for x in (w, w + 1))
                got += range(max(lo, 0), min(hi, span - cost))
            assert got == list(range(span - cost))
            at += span
        assert max(places) < len(spans) + workers
