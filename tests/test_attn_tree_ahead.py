"""CPU model of a pair's pipeline with three S buffers (trees, heads of 64): a warp that
issues the PVs and one for the QKs, two streams' softmax, MMAs that run later, each
warp's in the order issued, K and V landing at any time, under random interleavings.  Every wait by parity must pass exactly when the phase
that it means is complete; no MMA may write a buffer in use, and O may change only when
the PV before is done."""
import random

import pytest


class Barrier:
    def __init__(self, arrivals=1):
        self.need, self.got, self.phases = arrivals, 0, 0

    def arrive(self):
        self.got += 1
        if self.got == self.need:
            self.got, self.phases = 0, self.phases + 1

    def passes(self, phase):
        """A wait for `phase` by its parity; asserts that it tells the truth."""
        ok = (self.phases & 1) != (phase & 1)
        assert ok == (self.phases > phase), "a wait by parity mistook the phase"
        return ok


def run(pieces, seed, barriers=2, wait_done=True):
    r = random.Random(seed)
    total = sum(pieces)
    s_full, p_ready, o_done = ([[Barrier() for _ in range(barriers)] for _ in range(2)]
                               for _ in range(3))
    o_full, q_ready = ([Barrier() for _ in range(2)] for _ in range(2))
    landed = [False] * total, [False] * total                  # K, V
    queues = {"qk": [], "pv": []}                               # MMAs issued, in order by warp
    holder = [None] * 3                                         # (what, stream, tile) in a buffer
    done_pv = [0, 0]

    def which(tile):
        return tile % barriers, tile // barriers

    def pvs():
        at = 0
        for tiles in pieces:
            for n in range(2 * tiles):
                st, tile = n & 1, at + (n >> 1)
                while not landed[1][tile]:
                    yield
                b, phase = which(tile)
                while not p_ready[st][b].passes(phase):
                    yield
                queues["pv"].append((st, tile, (2 * at + n) % 3, n >> 1 == tiles - 1))
                yield
            at += tiles

    def qks():
        at = begun = 0
        for tiles in pieces:
            for n in range(2 * tiles):
                st, tile = n & 1, at + (n >> 1)
                while not landed[0][tile]:
                    yield
                while n < 2 and not q_ready[st].passes(begun):
                    yield
                before = 2 * at + n - 3
                if before >= 0 and wait_done:
                    b, phase = which(before >> 1)
                    while not o_done[before & 1][b].passes(phase):
                        yield
                queues["qk"].append((st, tile, (2 * at + n) % 3))
                yield
            at += tiles
            begun += tiles > 0

    def tensor(kind):
        for _ in range(2 * total):
            while not queues[kind]:
                yield
            op = queues[kind][0]
            if kind == "qk":
                assert holder[op[2]] is None, "S written while in use"
                holder[op[2]] = ("s", op[0], op[1])
            else:
                assert holder[op[2]] == ("p", op[0], op[1])
            for _ in range(r.choice([0, 1, 7])):
                yield
            queues[kind].pop(0)
            b, _ = which(op[1])
            if kind == "qk":
                s_full[op[0]][b].arrive()
            else:
                holder[op[2]] = None
                done_pv[op[0]] += 1
                o_done[op[0]][b].arrive()
                if op[3]:
                    o_full[op[0]].arrive()
            yield

    def softmax(st):
        tile, began, buf = 0, 0, st
        if any(pieces):
            q_ready[st].arrive()
        left = sum(n > 0 for n in pieces)
        for tiles in pieces:
            if tiles == 0:
                continue
            for t in range(tiles):
                b, phase = which(tile)
                while not s_full[st][b].passes(phase):
                    yield
                assert holder[buf] == ("s", st, tile)
                if t > 0 and r.random() < 0.5:                  # O is rescaled
                    b0, phase0 = which(tile - 1)
                    while not o_done[st][b0].passes(phase0):
                        yield
                    assert done_pv[st] == tile
                for _ in range(r.choice([0, 0, 1, 9])):
                    yield
                holder[buf] = ("p", st, tile)
                p_ready[st][b].arrive()
                buf = (buf + 2) % 3
                tile += 1
                yield
            began += 1
            left -= 1
            if left:
                q_ready[st].arrive()
            while not o_full[st].passes(began - 1):
                yield
            assert done_pv[st] == tile                          # its sums are read
            yield

    def loader():
        for i in range(total):
            for kind in (0, 1):
                for _ in range(r.choice([0, 0, 3, 40])):
                    yield
                landed[kind][i] = True

    procs = [pvs(), qks(), tensor("qk"), tensor("pv"), softmax(0), softmax(1), loader()]
    weights = [r.choice([1, 1, 5, 30]) for _ in procs]
    idle = 0
    while procs:
        i = r.choices(range(len(procs)), weights)[0]
        try:
            next(procs[i])
        except StopIteration:
            del procs[i], weights[i]
        idle += 1
        assert idle < 200000, "nothing goes on"
    assert done_pv == [total, total] and all(h is None for h in holder)


@pytest.mark.parametrize("seed", range(120))
def test_pipeline(seed):
    r = random.Random(seed)
    run([r.choice([0, 1, 2, 3, 5, 12]) for _ in range(r.choice([1, 2, 4]))] + [1], seed)


def test_the_model_tells_a_missing_wait():
    """Without the wait for the PV that read it last an S is written too early."""
    failed = 0
    for seed in range(60):
        try:
            run([12, 5], seed, wait_done=False)
        except AssertionError:
            failed += 1
    assert failed > 0


def test_the_model_tells_one_barrier_for_all_tiles():
    """With one barrier a stream either side can be two phases ahead of the other."""
    failed = 0
    for seed in range(60):
        try:
            run([12, 5], seed, barriers=1)
        except AssertionError:
            failed += 1
    assert failed > 0
