"""CPU model of a pair's pipeline with three S buffers (trees, heads of 64): the issuer,
two streams' softmax, MMAs that run later in the order issued, K and V landing at any
time, under random interleavings.  Every wait by parity must pass exactly when the phase
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


def run(pieces, seed, barriers=2, buffers=3):
    r = random.Random(seed)
    total = sum(pieces)
    s_full = [[Barrier() for _ in range(barriers)] for _ in range(2)]
    p_ready = [[Barrier() for _ in range(barriers)] for _ in range(2)]
    o_done, o_full, q_ready = ([Barrier() for _ in range(2)] for _ in range(3))
    landed = [False] * total, [False] * total                  # K, V
    queue = []                                                  # MMAs issued, in order
    holder = [None] * buffers                                   # (what, stream, tile) in a buffer
    done_pv = [0, 0]

    def which(tile):
        return tile % barriers, tile // barriers

    def issuer():
        at = 0
        for i, tiles in enumerate(pieces):
            if tiles == 0:
                continue
            while not landed[0][at]:
                yield
            for st in (0, 1):
                while not q_ready[st].passes(sum(n > 0 for n in pieces[:i])):
                    yield
                queue.append(("qk", st, at, st))
            if tiles > 1:
                while not landed[0][at + 1]:
                    yield
                queue.append(("qk", 0, at + 1, 2 % buffers))
            for n in range(2 * tiles):
                st, t = n & 1, n >> 1
                while not landed[1][at + t]:
                    yield
                b, phase = which(at + t)
                while not p_ready[st][b].passes(phase):
                    yield
                queue.append(("pv", st, at + t, n % buffers, t == tiles - 1))
                ahead = (n + 3) >> 1
                if ahead < tiles:
                    while not landed[0][at + ahead]:
                        yield
                    queue.append(("qk", st ^ 1, at + ahead, (n + 3) % buffers))
                yield
            at += tiles

    def tensor():
        for _ in range(4 * total):
            while not queue:
                yield
            op = queue[0]
            if op[0] == "qk":
                assert holder[op[3]] is None, "S written while in use"
                holder[op[3]] = ("s", op[1], op[2])
            else:
                assert holder[op[3]] == ("p", op[1], op[2])
            yield
            queue.pop(0)
            if op[0] == "qk":
                b, _ = which(op[2])
                s_full[op[1]][b].arrive()
            else:
                holder[op[3]] = None
                done_pv[op[1]] += 1
                o_done[op[1]].arrive()
                if op[4]:
                    o_full[op[1]].arrive()

    def softmax(st):
        tile, began = 0, 0
        if any(pieces):
            q_ready[st].arrive()
        left = sum(n > 0 for n in pieces)
        for tiles in pieces:
            if tiles == 0:
                continue
            buf = st
            for t in range(tiles):
                b, phase = which(tile)
                while not s_full[st][b].passes(phase):
                    yield
                assert holder[buf] == ("s", st, tile)
                if t > 0 and r.random() < 0.5:                  # O is rescaled
                    while not o_done[st].passes(tile - 1):
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

    procs = [issuer(), tensor(), softmax(0), softmax(1), loader()]
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


def test_the_model_tells_one_barrier_for_all_tiles():
    """With one barrier a stream either side can be two phases ahead of the other."""
    failed = 0
    for seed in range(60):
        try:
            run([12, 5], seed, barriers=1)
        except AssertionError:
            failed += 1
    assert failed > 0
