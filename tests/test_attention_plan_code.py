"""The index functions that attention's kernels run (csrc/attention_plan.cuh), compiled
for the host: every tile of every item is in exactly one piece, each piece has a place
of its own within its workspace, the joining kernel's loop meets an item's pieces, and
the streams' fills are the loader's order.  A CTA has pairs or single items, as in the
kernel."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from w4a16_moe_expert_sync_gb300 import build

COST, ROWS, KEYS = 2, 128, 128

SOURCE = """
#include "attention_plan.cuh"
using namespace w4::plan;
extern "C" {
int c_worker_begin(int all, int workers, int w) { return worker_begin(all, workers, w); }
int c_worker_of(int all, int workers, int x) { return worker_of(all, workers, x); }
int c_pair_ctas(int s, int p, int grid) { return pair_ctas(s, p, grid); }
int c_key_tiles(int k0, int k1, int shift) { return key_tiles(k0, k1, shift); }
int c_is_pair(int rows) { return is_pair(rows); }
int c_row_tiles(int rows) { return row_tiles(rows); }
int c_causal_tiles(int k1, int t, int base, int last, int rep)
{ return causal_tiles(k1, t, base, last, rep); }
int c_fill_of(int a, int b, int which, int r) { return fill_of(a, b, which, r); }
void c_caps(long long T, long long rep, int B, int G, int Hkv, int grid, int *out)
{ Caps c = caps_of(T, rep, B, G, Hkv, grid); out[0] = c.pairs; out[1] = c.groups; out[2] = c.singles; }
int c_constant(int i) { return i == 0 ? kItemCost : i == 1 ? kRows : kKeys; }
}
"""


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, str(src), "-o",
                    str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.c_caps.argtypes = [ctypes.c_longlong, ctypes.c_longlong] + [ctypes.c_int] * 4 + \
        [ctypes.c_void_p]
    assert [lib.c_constant(i) for i in range(3)] == [COST, ROWS, KEYS]
    return lib


def test_the_kernels_run_this_code():
    with open(os.path.join(build.CSRC, "attention.cu")) as f:
        text = f.read()
    assert '#include "attention_plan.cuh"' in text
    for name in ("worker_begin(", "worker_of(", "pair_ctas(", "plan::key_tiles(", "plan::row_tiles(",
                 "plan::causal_tiles(", "plan::fill_of(", "plan::caps_of("):
        assert name in text, name


@pytest.mark.parametrize("seed", range(40))
def test_shares_and_owners(code, seed):
    r = random.Random(seed)
    total = r.choice([1, 2, 5, 151, 152, 4000, 1 << 21, (1 << 22) - 1, 1 << 22, 2 ** 31 - 5000])
    workers = min(total, r.choice([1, 7, 152, 304, 512]))
    begin = [code.c_worker_begin(total, workers, w) for w in range(workers + 1)]
    assert begin[0] == 0 and begin[-1] == total
    assert all(a < b for a, b in zip(begin, begin[1:]))
    for w in range(workers):
        for x in {begin[w], begin[w + 1] - 1, r.randrange(begin[w], begin[w + 1])}:
            assert code.c_worker_of(total, workers, x) == w


@pytest.mark.parametrize("seed", range(40))
def test_ctas_of_pairs_and_singles(code, seed):
    r = random.Random(seed)
    for _ in range(200):
        singles, pairs = (r.choice([0, 1, 3, 100, 5000, 10 ** 7]) for _ in range(2))
        grid = r.choice([2, 7, 148, 152])
        n = code.c_pair_ctas(singles, pairs, grid)
        assert 0 <= n <= min(pairs, grid)
        assert (n > 0) == (pairs > 0)
        assert singles == 0 or grid - n > 0


@pytest.mark.parametrize("seed", range(40))
def test_fills_are_the_loaders_order(code, seed):
    r = random.Random(seed)
    tiles = [r.choice([0, 1, 2, 5, 13, 40]) for _ in range(2)]
    order = []
    for t in range(max(tiles)):
        order += [(s, t) for s in (0, 1) if t < tiles[s]]
    for n, (s, t) in enumerate(order):
        assert code.c_fill_of(tiles[0], tiles[1], s, t) == n
    assert [code.c_fill_of(0, 0, 2, t) for t in range(9)] == list(range(9))


@pytest.mark.parametrize("seed", range(80))
def test_every_tile_is_in_one_piece_and_met_once(code, seed):
    r = random.Random(1000 + seed)
    grid = r.choice([2, 7, 148, 152])
    shift, Hkv, rep = r.choice([4, 5, 6, 7]), r.choice([1, 2, 8]), r.choice([1, 2, 3, 8])
    page, causal = 1 << shift, r.random() < 0.6
    max_q = r.choice([1, 1, 5, 33, 300, 2048])
    sizes = [r.choice([0, 1, 2, 7, 33]) for _ in range(r.choice([0, 1, 3, 9]))]
    alone = r.choice([1, 1, 40])
    G, B = len(sizes), sum(sizes) + alone
    shared, lens, group = [], [], []
    for g, n in enumerate(sizes):
        shared.append(r.choice([0, 1, 17, 128, 5000]))
        lens += [shared[-1] + r.choice([0, 1, 40, 900]) for _ in range(n)]
        group += [g] * n
    lens += [r.choice([0, 1, 500, 3001]) for _ in range(alone)]
    group += [-1] * alone
    nq = [r.choice([0, 1, max_q]) for _ in range(B)]
    qo = [sum(nq[:b]) for b in range(B + 1)]
    go = [sum(sizes[:g]) for g in range(G + 1)]
    caps = (ctypes.c_int * 3)()
    code.c_caps(qo[-1], rep, B, G, Hkv, grid, caps)
    cap = {True: caps[0], False: caps[2]}
    # (queries, first key, end) of the groups' prefixes and of the sequences' own keys
    want = [(qo[go[g + 1]] - qo[go[g]], 0, min(shared[g], lens[go[g]]) if sizes[g] else 0)
            for g in range(G)]
    want += [(nq[b], min(shared[group[b]], lens[go[group[b]]], lens[b]) if group[b] >= 0 else 0,
              lens[b]) for b in range(B)]
    items = {False: [], True: []}              # (entry, item of it, span) in their order
    for e, (tokens, k0, k1) in enumerate(want):
        rows = tokens * rep
        if rows > 0 and k1 > k0:
            span = code.c_key_tiles(k0, k1, shift) + COST
            base = k0 // page * page
            assert base + (span - COST) * KEYS >= k1 > base + (span - COST - 1) * KEYS
            pair = bool(code.c_is_pair(rows))
            assert pair == (rows > ROWS)
            n = code.c_row_tiles(rows)
            assert n * (2 if pair else 1) * ROWS >= rows
            items[pair] += [(e, i, span, n) for i in range(n * Hkv)]
    total = {p: sum(x[2] for x in items[p]) for p in items}
    ctas = code.c_pair_ctas(total[False], total[True], grid)
    workers = {True: ctas, False: min(total[False], 2 * (grid - ctas))}
    for pair, own in items.items():
        at, seen = 0, {}
        for number, (e, i, span, n) in enumerate(own):
            lo, hi = (code.c_worker_of(total[pair], workers[pair], x) for x in (at, at + span - 1))
            tokens, k0, k1 = want[e]
            got = []
            for w in range(lo, hi + 1):
                place = number + w
                assert 0 <= place < cap[pair] and place not in seen
                assert pair or e >= G or place < caps[1]
                seen[place] = w
                first = max(code.c_worker_begin(total[pair], workers[pair], w) - at - COST, 0)
                end = min(code.c_worker_begin(total[pair], workers[pair], w + 1) - at - COST,
                          span - COST)
                if causal and e >= G:
                    step = (2 if pair else 1) * ROWS
                    row0 = i % n * step
                    last = min(row0 + step, tokens * rep) - 1
                    end = min(end, code.c_causal_tiles(k1, tokens, k0 // page * page, last, rep))
                got += range(first, end)
            # the tiles with a key that one of the rows sees, each once and in order
            sees = span - COST
            if causal and e >= G:
                limit = k1 - tokens + last // rep + 1
                sees = min(sees, -(-max(limit - k0 // page * page, 0) // KEYS))
            assert got == list(range(sees))
            at += span
        assert at == total[pair]
