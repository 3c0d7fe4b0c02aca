"""Lengths that the caller has lowered: the pages behind them stay with their slot,
are used again when it grows and counted once, and no page that several slots hold
is grown into."""
import random

import pytest

from test_gpu_kv import Device, Model, _ints, _model

import w4a16_moe_expert_sync_gb300 as w4

pytestmark = pytest.mark.gpu


class Lowered(Model):
    """The model of the cache, with pages held past a slot's length."""

    def reserve(self, slots, lens):
        kept, good = [], []
        for i, (s, n) in enumerate(zip(slots, lens)):
            ok = 0 <= s < self.B and s not in slots[:i] and n >= self.lens[s] and \
                -(-n // self.page) <= self.W
            first = -(-self.lens[s] // self.page) if ok else 0
            if ok and n > self.lens[s]:
                c = self.lens[s] // self.page
                while ok and c < -(-n // self.page) and self.table[s][c] >= 0:
                    ok = self.refs[self.table[s][c]] == 1
                    c += 1
                first = max(first, c)
            kept.append(first)
            good.append(ok)
        wants = [max(-(-n // self.page) - f, 0) if ok else 0 for n, f, ok in zip(lens, kept, good)]
        status = 0 if all(good) else w4.W4_DEV_BAD_SLOT
        for s, n, f, ok, pages in zip(slots, lens, kept, good, self.hand_out(wants)):
            if not ok:
                continue
            if pages is None:
                status |= w4.W4_DEV_NO_PAGES
                continue
            self.table[s][f:f + len(pages)] = pages
            self.lens[s] = n
        return status

    def fork(self, parents, children):
        held = [0 <= b < self.B and self.table[b][0] >= 0 for b in children]
        # a child that holds pages is refused: out of range, to the plain model
        return super().fork(parents, [-1 if h else b for h, b in zip(held, children)])


def _state(planes, P, page, B, W, seed=0):
    m = _model(planes, P, page, 1, 8, B, W, seed)
    m.__class__ = Lowered
    return m, Device(m)


def _lower(m, d, slot, n):
    m.lens[slot] = n
    d.lens[slot] = n


def test_tokens_taken_back_lose_no_page(lib):
    import torch
    m, d = _state((1, 2), 20, 4, 4, 8)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def reserve(slots, lens):
        st.zero_()
        want = m.reserve(slots, lens)
        lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints(slots), _ints(lens), 4, dev_status=st)
        assert int(st) == want
        d.check(m)
    reserve([0, 2], [14, 9])
    _lower(m, d, 0, 5)
    reserve([0], [6])                        # within a page that it holds
    reserve([0, 1], [20, 3])                 # three pages kept, one more
    _lower(m, d, 2, 0)
    reserve([2], [12])
    assert sum(m.refs) == 5 + 1 + 3
    _lower(m, d, 0, 8)
    m.free([0, 1, 2])
    lib.w4_kv_free(d.table, d.lens, d.refs, _ints([0, 1, 2]))
    d.check(m)
    assert int(d.refs.abs().sum()) == 0


def test_a_shared_page_is_not_grown_into(lib):
    import torch
    m, d = _state((1, 2), 20, 4, 4, 8)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.reserve([0], [14])
    lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints([0]), _ints([14]), 4)
    m.fork([0], [1])
    lib.w4_kv_fork(d.pool, d.table, d.lens, d.refs, _ints([0]), _ints([1]))
    d.check(m)
    for n in (10, 8, 4, 0):                  # inside a shared page, at the start of one
        _lower(m, d, 1, n)
        st.zero_()
        assert m.reserve([1], [13]) == w4.W4_DEV_BAD_SLOT
        lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints([1]), _ints([13]), 4, dev_status=st)
        assert int(st) == w4.W4_DEV_BAD_SLOT
        d.check(m)
    # nor is a slot that holds pages a child
    st.zero_()
    assert m.fork([0], [1]) == w4.W4_DEV_BAD_SLOT
    lib.w4_kv_fork(d.pool, d.table, d.lens, d.refs, _ints([0]), _ints([1]), dev_status=st)
    assert int(st) == w4.W4_DEV_BAD_SLOT
    d.check(m)
    _lower(m, d, 1, 13)                      # its own last page
    assert m.reserve([1], [17]) == 0
    st.zero_()
    lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints([1]), _ints([17]), 4, dev_status=st)
    assert int(st) == 0
    d.check(m)


@pytest.mark.parametrize("planes,P,page,B,W", [((1, 2), 60, 4, 8, 9), ((2, 2), 300, 16, 12, 40),
                                               ((2, 1), 5000, 2, 40, 150)])
def test_random_histories_with_lowered_lengths(lib, planes, P, page, B, W):
    import torch
    m, d = _state(planes, P, page, B, W, seed=3)
    r = random.Random(P)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(60):
        st.zero_()
        kind = r.choice(["reserve", "reserve", "lower", "lower", "fork", "free", "compact"])
        n = r.randint(1, B)
        slots = r.sample(range(B), n)
        want = 0
        if kind == "reserve":
            lens = [min(W * page, m.lens[s] + r.randint(0, 3 * P * page // B)) for s in slots]
            want = m.reserve(slots, lens)
            lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints(slots), _ints(lens), page,
                              dev_status=st)
        elif kind == "lower":
            for s in slots[:max(1, n // 2)]:
                _lower(m, d, s, r.choice([0, m.lens[s] // 2, max(m.lens[s] - 3, 0)]))
        elif kind == "fork":
            children = [s for s in range(B) if m.lens[s] == 0][:n] or slots[:1]
            parents = [r.randrange(B) for _ in children]
            want = m.fork(parents, children)
            lib.w4_kv_fork(d.pool, d.table, d.lens, d.refs, _ints(parents), _ints(children),
                           dev_status=st)
        elif kind == "free":
            want = m.free(slots[:max(1, n // 3)])
            lib.w4_kv_free(d.table, d.lens, d.refs, _ints(slots[:max(1, n // 3)]), dev_status=st)
        else:
            m.compact()
            lib.w4_kv_compact(d.pool, d.table, d.refs, dev_status=st)
        assert int(st) == want, (step, kind)
        d.check(m)
        held = {}
        for row in m.table:
            for p in row:
                if p >= 0:
                    held[p] = held.get(p, 0) + 1
        assert [held.get(p, 0) for p in range(P)] == m.refs


def test_requests_that_need_no_page_are_served_behind_one_that_lacks_some(lib):
    import torch
    m, d = _state((1, 2), 8, 4, 6, 8)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.reserve([1, 2], [6, 8])
    lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints([1, 2]), _ints([6, 8]), 4)
    d.check(m)                               # four pages in use, four free
    args = [0, 1, 3, 4, 2], [20, 8, 1, 0, 9]     # five pages; none; one; none; one
    assert m.reserve(*args) == w4.W4_DEV_NO_PAGES
    lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints(args[0]), _ints(args[1]), 4, dev_status=st)
    assert int(st) == w4.W4_DEV_NO_PAGES
    d.check(m)
    assert m.lens == [0, 8, 8, 0, 0, 0]
    m.reserve([0, 1], [12, 10])              # one is left behind: seven and one in use
    lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints([0, 1]), _ints([12, 10]), 4)
    d.check(m)
    st.zero_()
    args = [1, 2], [3, 4]                    # a tail page, and full pages alone
    assert m.fork(*args) == w4.W4_DEV_NO_PAGES
    lib.w4_kv_fork(d.pool, d.table, d.lens, d.refs, _ints(args[0]), _ints(args[1]), dev_status=st)
    assert int(st) == w4.W4_DEV_NO_PAGES
    d.check(m)
    assert m.lens == [12, 10, 8, 0, 8, 0]
