"""CPU models of the attention kernel's bookkeeping: the split of tiles over
workers and pieces, the order of the ring's fills, and the ring itself under
random interleavings."""
import random

import pytest


def worker_begin(tiles, workers, w):
    return tiles * w // workers


def worker_of(tiles, workers, x):
    return ((x + 1) * workers - 1) // tiles


@pytest.mark.parametrize("seed", range(30))
def test_every_tile_has_one_piece_and_no_two_pieces_share_a_place(seed):
    r = random.Random(seed)
    items = [r.choice([0, 1, 2, 3, 17, 200]) for _ in range(r.choice([1, 2, 9, 120]))]
    starts, total = [], 0
    for n in items:
        starts.append(total)
        total += n
    if total == 0:
        return
    workers = min(total, r.choice([1, 7, 152, 304]))
    pieces = {}
    for w in range(workers):
        lo, hi = worker_begin(total, workers, w), worker_begin(total, workers, w + 1)
        assert hi > lo
        for i, n in enumerate(items):
            a, b = max(lo, starts[i]), min(hi, starts[i] + n)
            if a < b:
                assert i + w not in pieces
                pieces[i + w] = (i, a, b)
                assert worker_of(total, workers, a) == w == worker_of(total, workers, b - 1)
    seen = sorted((a, b) for _, a, b in pieces.values())
    assert seen[0][0] == 0 and seen[-1][1] == total
    assert all(x[1] == y[0] for x, y in zip(seen, seen[1:]))
    assert max(pieces) < len(items) + workers
    # the joining kernel's loop meets exactly an item's pieces
    for i, n in enumerate(items):
        if n:
            w0 = worker_of(total, workers, starts[i])
            w1 = worker_of(total, workers, starts[i] + n - 1)
            assert all(pieces[i + w][0] == i for w in range(w0, w1 + 1))
            assert sum(pieces[i + w][2] - pieces[i + w][1] for w in range(w0, w1 + 1)) == n


def fill_of(tiles, which, r):
    if which == 2:
        return r
    return tiles[2] + r + (min(r, tiles[1]) if which == 0 else min(r + 1, tiles[0]))


def load_order(tiles):
    order = [(2, r) for r in range(tiles[2])]
    for r in range(max(tiles[0], tiles[1])):
        order += [(s, r) for s in (0, 1) if r < tiles[s]]
    return order


def run_ring(slots, tiles, r, exact=True, early=False):
    """Loader, landings, two issuers and two softmax groups as state machines
    under a random interleaving.  Barriers are parity waits: a wait for phase n
    passes when the completed phases' count differs from n in parity, right or
    not; the phase meant is asserted.  Copies land in any order.  With early, V is
    awaited before its P."""
    order = load_order(tiles)
    for n, (s, t) in enumerate(order):
        assert fill_of(tiles, s, t) == n
    full = [0] * slots               # completed phases of full[slot]
    empty = [0] * slots              # completed phases of empty[slot]
    content = [None] * slots
    flying, requested = [], [0]

    def passes(done, phase):
        return (done - phase) % 2 == 1

    def loader():
        for fill, (s, t) in enumerate(order):
            for part in (0, 1):
                n = 2 * fill + part
                slot, use = n % slots, n // slots
                if use:
                    while not passes(empty[slot], use - 1):
                        yield
                    assert empty[slot] == use
                flying.append((slot, (s, t, part)))
                requested[0] = n + 1
                yield

    def landing():
        while True:
            if flying:
                slot, what = flying.pop(r.randrange(len(flying)))
                content[slot] = what
                full[slot] += 1
            yield

    s_full, p_ready, pairs_done = [0, 0], [0, 0], []

    def landed(which, t, part):
        n = 2 * fill_of(tiles, which, t) + part
        slot, count = n % slots, n // slots
        while exact and requested[0] <= n:
            yield
        while not passes(full[slot], count):
            yield
        assert full[slot] == count + 1 and content[slot] == (which, t, part)

    def use(which, t, part, last):
        n = 2 * fill_of(tiles, which, t) + part
        slot, count = n % slots, n // slots
        yield from landed(which, t, part)
        yield
        if last:
            empty[slot] += 1
        yield

    def wait_p(stream, n):
        while not passes(p_ready[stream], n - 1):
            yield
        assert p_ready[stream] == n

    def issuer(stream):
        if stream == 0:
            for t in range(tiles[2]):
                for st in (0, 1):
                    if t == 0:
                        yield from use(2, 0, 0, st == 1)
                        s_full[st] += 1
                if early:
                    yield from landed(2, t, 1)
                for st in (0, 1):
                    yield from wait_p(st, t + 1)
                    yield from use(2, t, 1, st == 1)
                    if t + 1 < tiles[2]:
                        yield from use(2, t + 1, 0, st == 1)
                        s_full[st] += 1
            pairs_done.append(1)
        while not pairs_done:
            yield
        for t in range(tiles[stream]):
            yield from use(stream, t, 0, True)
            s_full[stream] += 1
            if early:
                yield from landed(stream, t, 1)
            yield from wait_p(stream, tiles[2] + t + 1)
            yield from use(stream, t, 1, True)

    def softmax(stream):
        for n in range(tiles[2] + tiles[stream]):
            while not passes(s_full[stream], n):
                yield
            assert s_full[stream] == n + 1
            yield
            p_ready[stream] += 1

    roles = [loader(), issuer(0), issuer(1), softmax(0), softmax(1)]
    back = landing()
    slow = r.choice([1, 3, 20])
    for _ in range(400000):
        if not roles:
            break
        if r.randrange(slow + 1) == 0:
            next(back)
        g = r.choice(roles)
        try:
            next(g)
        except StopIteration:
            roles.remove(g)
    assert not roles


@pytest.mark.parametrize("slots", [5, 10])
@pytest.mark.parametrize("seed", range(40))
def test_ring_fills_and_releases(slots, seed):
    r = random.Random(seed)
    run_ring(slots, [r.choice([0, 1, 2, 5, 13, 40]) for _ in range(3)], r)


@pytest.mark.parametrize("slots", [5, 10])
@pytest.mark.parametrize("seed", range(40))
def test_ring_of_a_cta_with_pairs_or_singles(slots, seed):
    """As the kernel has it: pairs or single items, V awaited before P."""
    r = random.Random(100 + seed)
    n = [r.choice([0, 1, 2, 5, 13, 40]) for _ in range(2)]
    run_ring(slots, [0, 0, n[0]] if seed % 2 else [*n, 0], r, early=True)


def ceil(a, b):
    return -(-a // b)


def pair_ctas(singles, pairs, grid):
    if pairs == 0 or singles == 0:
        return min(pairs, grid)
    part = pairs / (pairs + 0.7 * singles)
    return min(pairs, max(1, min(grid - 1, int(part * grid + 0.5))))


@pytest.mark.parametrize("seed", range(60))
def test_plan_and_join_meet_every_tile_once(seed):
    """The plan's pieces of random batches: each within its workspace, no two in
    one place, and the joining kernel's loop over an item finds exactly its
    tiles."""
    r = random.Random(seed)
    grid, rows, cost, keys = r.choice([2, 7, 152, 152]), 128, 2, 128
    page, Hkv, rep = r.choice([16, 32, 64, 128]), r.choice([1, 2, 8]), r.choice([1, 2, 3, 8])
    max_q, causal = r.choice([1, 1, 5, 33, 300]), r.random() < 0.5
    sizes = [r.choice([0, 1, 2, 7, 33]) for _ in range(r.choice([0, 1, 3, 9]))]
    alone = r.choice([0, 1, 40])
    G, B = len(sizes), sum(sizes) + alone
    if B == 0:
        return
    shared, lens, nq, group = [], [], [], []
    for g, n in enumerate(sizes):
        shared.append(r.choice([0, 1, 17, 128, 5000]))
        for _ in range(n):
            lens.append(shared[-1] + r.choice([0, 1, 40, 900]))
            group.append(g)
    lens += [r.choice([0, 1, 500, 3001]) for _ in range(alone)]
    group += [-1] * alone
    nq = [r.choice([0, 1, max_q]) for _ in range(B)]
    go = [sum(sizes[:g]) for g in range(G + 1)]
    qo = [sum(nq[:b]) for b in range(B + 1)]
    T = qo[-1]
    cap_a = 2 * T * rep // rows * Hkv + 256
    cap_g = G * Hkv + 512
    cap_b = cap_g + B * Hkv
    want = [(qo[go[g + 1]] - qo[go[g]], 0, min(shared[g], lens[go[g]]) if sizes[g] else 0)
            for g in range(G)]
    want += [(nq[b], min(shared[group[b]], lens[go[group[b]]], lens[b]) if group[b] >= 0 else 0,
              lens[b]) for b in range(B)]
    entries, start, at = [], [], {False: [0, 0], True: [0, 0]}
    for tokens, k0, k1 in want:
        n = tokens * rep
        span, pair, tiles = 0, False, 0
        if n > 0 and k1 > k0:
            span = ceil(k1 - k0 // page * page, keys) + cost
            pair = n > rows
            tiles = ceil(n, 2 * rows) if pair else 1
        entries.append((span, pair, tiles))
        start.append((tuple(at[False]), tuple(at[True])))
        at[pair][0] += tiles * Hkv * span
        at[pair][1] += tiles * Hkv
    ctas = pair_ctas(at[False][0], at[True][0], grid)
    workers = {True: ctas, False: min(at[False][0], 2 * (grid - ctas))}
    assert (at[True][0] == 0) == (workers[True] == 0)
    assert (at[False][0] == 0) == (workers[False] == 0)

    def find(pair, which, x):                  # as the kernel's search
        lo, hi = 0, len(entries) - 1
        while lo < hi:
            mid = (lo + hi + 1) >> 1
            if start[mid][pair][which] <= x:
                lo = mid
            else:
                hi = mid - 1
        assert entries[lo][0] > 0 and entries[lo][1] == pair
        return lo

    pieces, done = {}, set()
    for pair in (False, True):
        total = at[pair][0]
        for w in range(workers[pair]):
            lo, hi = worker_begin(total, workers[pair], w), worker_begin(total, workers[pair], w + 1)
            ends = [find(pair, 0, x) for x in (lo, hi - 1)]
            first, last = [start[e][pair][1] + (x - start[e][pair][0]) // entries[e][0]
                           for e, x in zip(ends, (lo, hi - 1))]
            assert last + w < (cap_a if pair else cap_b)
            for item in range(first, last + 1):
                e = find(pair, 1, item)
                span, _, row_tiles = entries[e]
                local = item - start[e][pair][1]
                assert 0 <= local < row_tiles * Hkv
                begin = start[e][pair][0] + local * span + cost
                tile0, end = max(lo - begin, 0), min(hi - begin, span - cost)
                tokens, k0, k1 = want[e]
                row0 = local % row_tiles * (2 if pair else 1) * rows
                here = min((2 if pair else 1) * rows, tokens * rep - row0)
                assert here > 0
                if causal and e >= G:
                    limit = k1 - tokens + (row0 + here - 1) // rep + 1
                    end = min(end, ceil(max(limit - k0 // page * page, 0), keys))
                assert (pair, item + w) not in pieces
                assert e >= G or pair or item + w < cap_g
                pieces[pair, item + w] = (e, local, tile0, max(end - tile0, 0))
    for e, (span, pair, row_tiles) in enumerate(entries):
        for local in range(row_tiles * Hkv if span else 0):
            x = start[e][pair][0] + local * span
            w0, w1 = (worker_of(at[pair][0], workers[pair], y) for y in (x, x + span - 1))
            mine = [pieces[pair, start[e][pair][1] + local + w] for w in range(w0, w1 + 1)]
            assert all(m[:2] == (e, local) for m in mine)
            tiles = [t for m in mine for t in range(m[2], m[2] + m[3])]
            assert tiles == list(range(len(tiles))) and len(tiles) <= span - cost
            if not (causal and e >= G):
                assert len(tiles) == span - cost
            done.update((pair, start[e][pair][1] + local + w) for w in range(w0, w1 + 1))
    assert done == set(pieces)


def test_the_model_tells_a_wait_by_parity_alone():
    """A slot's fills alternate between the streams: without looking whether
    the fill has been requested, a wait can pass a phase early."""
    failed = 0
    for seed in range(60):
        r = random.Random(seed)
        try:
            run_ring(5, [40, 40, 0], r, exact=False)
        except AssertionError:
            failed += 1
    assert failed > 0


def test_refusals_without_launching():
    import ctypes

    import w4a16_moe_expert_sync_gb300 as w4
    from w4a16_moe_expert_sync_gb300 import build as w4build
    w4build.build()
    lib = w4.load_library()
    P = ctypes.c_void_p
    f, odd, odd4 = P(0x10000), P(0x10004), P(0x10002)
    ok = [f, 2048, 128, f, f, 16384, 1024, 128, 50, 16, f, 8, f, f, 6, 3, 4, f, f, 1, 16, 8, 128, 0,
          1, 0.1, f, 1 << 40, f, None, None]

    def bad(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return lib.w4_attn_shared_prefix(*a)
    for i in (0, 3, 4, 10, 12, 13, 17, 18, 28):
        assert bad(**{f"a{i}": None}) == 1, i
    assert bad(a14=-1) == 1 and bad(a16=0) == 1 and bad(a23=2) == 1 and bad(a25=0.0) == 1
    assert bad(a25=float("nan")) == 1 and bad(a25=float("inf")) == 1
    assert bad(a22=96) == 2 and bad(a9=24) == 2 and bad(a20=12) == 2 and bad(a15=4096) == 2
    assert bad(a11=1 << 28) == 2 and bad(a14=1 << 21) == 2
    assert bad(a0=odd) == 3 and bad(a3=odd) == 3 and bad(a1=2044) == 3 and bad(a7=4) == 3
    assert bad(a10=odd4) == 3 and bad(a26=P(0x10010)) == 3
    assert bad(a26=None) == 6 and bad(a27=100) == 6
    assert bad(a14=0) == 0 and bad(a15=0) == 0
    ws = lib.w4_attn_shared_prefix_workspace_size
    assert ws(6, 3, 1, 4, 16, 8, 128) > 0 and ws(6, 3, 1, 4, 16, 5, 128) == 0
