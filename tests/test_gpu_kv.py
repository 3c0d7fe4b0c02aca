"""The paged cache's operations against a plain model of the same state: page
tables, lengths, reference counts and every value of the pool, exactly."""
import ctypes
import random

import pytest

import w4a16_moe_expert_sync_gb300 as w4


class Model:
    """The cache's state and rules in plain Python; pool as a float tensor."""

    def __init__(self, pool, B, W, page):
        self.pool, self.B, self.W, self.page = pool, B, W, page
        self.P = pool.shape[-4]
        self.table = [[-1] * W for _ in range(B)]
        self.lens = [0] * B
        self.refs = [0] * self.P

    def planes(self):
        return self.pool.view(-1, *self.pool.shape[-4:])

    def hand_out(self, wants):
        """wants: list of counts; returns the pages of each, None from the
        first that lacks one on."""
        free = [p for p in range(self.P) if self.refs[p] == 0]
        out, short = [], False
        for n in wants:
            if n and (short or n > len(free)):
                short = True
                out.append(None)
                continue
            out.append(free[:n])
            free = free[n:]
        for pages in out:
            for p in pages or []:
                self.refs[p] = 1
        return out

    def reserve(self, slots, lens):
        good = []
        for i, (s, n) in enumerate(zip(slots, lens)):
            ok = 0 <= s < self.B and s not in slots[:i] and n >= self.lens[s] and \
                -(-n // self.page) <= self.W
            good.append(ok)
        first = [-(-self.lens[s] // self.page) if ok else 0 for s, ok in zip(slots, good)]
        wants = [-(-n // self.page) - f if ok else 0 for n, f, ok in zip(lens, first, good)]
        status = 0 if all(good) else w4.W4_DEV_BAD_SLOT
        for s, n, f, ok, pages in zip(slots, lens, first, good, self.hand_out(wants)):
            if not ok:
                continue
            if pages is None:
                status |= w4.W4_DEV_NO_PAGES
                continue
            self.table[s][f:f + len(pages)] = pages
            self.lens[s] = n
        return status

    def free(self, slots):
        status = 0
        for s in slots:
            if not 0 <= s < self.B:
                status |= w4.W4_DEV_BAD_SLOT
                continue
            for p in self.table[s]:
                if p >= 0:
                    self.refs[p] -= 1
            self.table[s] = [-1] * self.W
            self.lens[s] = 0
        return status

    def fork(self, parents, children):
        before = list(self.lens)
        good = [0 <= a < self.B and 0 <= b < self.B and a != b and before[b] == 0 and
                b not in children[:i] for i, (a, b) in enumerate(zip(parents, children))]
        wants = [int(before[a] % self.page != 0) if ok else 0 for a, ok in zip(parents, good)]
        status = 0 if all(good) else w4.W4_DEV_BAD_SLOT
        rows = [list(self.table[a]) if ok else None for a, ok in zip(parents, good)]
        for a, b, row, ok, pages in zip(parents, children, rows, good, self.hand_out(wants)):
            if not ok:
                continue
            if pages is None:
                status |= w4.W4_DEV_NO_PAGES
                continue
            full, tail = divmod(before[a], self.page)
            self.table[b][:full] = row[:full]
            for p in row[:full]:
                self.refs[p] += 1
            if tail:
                self.table[b][full] = pages[0]
                self.planes()[:, pages[0], :tail] = self.planes()[:, row[full], :tail]
            self.lens[b] = before[a]
        return status

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, self.P) if self.refs[p] > 0]
        move = dict(zip(movers, holes))
        for a, b in move.items():
            self.planes()[:, b] = self.planes()[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[move.get(p, p) for p in row] for row in self.table]

    def append(self, k, v, offs):
        kp, vp = self.planes()[0], self.planes()[1]
        for b in range(len(offs) - 1):
            for i in range(offs[b], offs[b + 1]):
                pos = self.lens[b] - (offs[b + 1] - i)
                p = self.table[b][pos // self.page]
                kp[p, pos % self.page], vp[p, pos % self.page] = k[i], v[i]


class Device:
    def __init__(self, m):
        import torch
        self.pool = m.pool.cuda()
        self.table = torch.tensor(m.table, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(m.lens, dtype=torch.int32, device="cuda")
        self.refs = torch.tensor(m.refs, dtype=torch.int32, device="cuda")

    def check(self, m):
        import torch
        assert self.table.tolist() == m.table
        assert self.lens.tolist() == m.lens
        assert self.refs.tolist() == m.refs
        assert torch.equal(self.pool.cpu().view(torch.int16), m.pool.view(torch.int16))


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _model(planes, P, page, Hkv, D, B, W, seed=0, dtype="bfloat16"):
    import torch
    g = torch.Generator().manual_seed(seed)
    pool = torch.randn((*planes, P, page, Hkv, D), generator=g).to(getattr(torch, dtype))
    return Model(pool, B, W, page)


@pytest.mark.gpu
@pytest.mark.parametrize("planes,P,page,Hkv,D,B,W", [
    ((1, 2), 40, 4, 1, 8, 6, 9), ((2, 2), 300, 16, 2, 64, 12, 40), ((2, 2), 64, 1, 1, 8, 5, 30),
    ((3, 2), 5000, 2, 1, 16, 40, 150), ((1, 2), 9000, 32, 1, 8, 33, 400)])
def test_random_histories_match_the_model(lib, planes, P, page, Hkv, D, B, W):
    import torch
    m = _model(planes, P, page, Hkv, D, B, W)
    d = Device(m)
    r = random.Random(P)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(30):
        st.zero_()
        kind = r.choice(["reserve", "reserve", "fork", "free", "compact", "append"])
        n = r.randint(1, B)
        slots = r.sample(range(B), n)
        if kind == "reserve":
            lens = [min(W * page, m.lens[s] + r.randint(0, 3 * P * page // B)) for s in slots]
            want = m.reserve(slots, lens)
            lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints(slots), _ints(lens), page,
                              dev_status=st)
        elif kind == "fork":
            empty = [s for s in range(B) if m.lens[s] == 0]
            children = empty[:n] or slots[:1]
            parents = [r.randrange(B) for _ in children]
            want = m.fork(parents, children)
            lib.w4_kv_fork(d.pool, d.table, d.lens, d.refs, _ints(parents), _ints(children),
                           dev_status=st)
        elif kind == "free":
            want = m.free(slots[:max(1, n // 3)])
            lib.w4_kv_free(d.table, d.lens, d.refs, _ints(slots[:max(1, n // 3)]), dev_status=st)
        elif kind == "compact":
            m.compact()
            want = 0
            lib.w4_kv_compact(d.pool, d.table, d.refs, dev_status=st)
        else:
            # only onto tokens of pages that this slot alone holds
            counts = []
            for b in range(B):
                mine = 0
                while mine < m.lens[b] and m.refs[
                        m.table[b][(m.lens[b] - mine - 1) // page]] == 1:
                    mine += 1
                counts.append(r.randint(0, min(mine, 40)))
            offs = [0]
            for c in counts:
                offs.append(offs[-1] + c)
            kv = torch.randn((offs[-1], 3, Hkv, D)).to(m.pool.dtype)
            m.append(kv[:, 0], kv[:, 2], offs)
            want = 0
            g = kv.cuda()
            lib.w4_kv_append(d.pool.view(-1, *d.pool.shape[-4:])[0],
                             d.pool.view(-1, *d.pool.shape[-4:])[1], d.table, d.lens, g[:, 0],
                             g[:, 2], _ints(offs), dev_status=st)
        assert int(st) == want, (step, kind)
        d.check(m)


@pytest.mark.gpu
def test_running_out_of_pages_leaves_the_rest_alone(lib):
    import torch
    m = _model((1, 2), 10, 4, 1, 8, 6, 8)
    d = Device(m)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = ([3, 1, 4, 0, 5], [8, 13, 0, 20, 1])      # 2 + 4 + 0 + 5 > 4 left; then 1
    want = m.reserve(*args)
    lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints(args[0]), _ints(args[1]), 4, dev_status=st)
    assert want == w4.W4_DEV_NO_PAGES == int(st)
    d.check(m)
    assert m.lens == [0, 13, 0, 8, 0, 0]


@pytest.mark.gpu
def test_bad_slots_and_pages_are_flagged_and_skipped(lib):
    import torch
    m = _model((1, 2), 12, 4, 1, 8, 5, 3)
    d = Device(m)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    # out of range, repeated, too long, shrinking
    slots, lens = [-1, 5, 2, 2, 3, 2 ** 30], [4, 4, 6, 7, 13, 1]
    assert m.reserve(slots, lens) == w4.W4_DEV_BAD_SLOT
    lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints(slots), _ints(lens), 4, dev_status=st)
    assert int(st) == w4.W4_DEV_BAD_SLOT
    d.check(m)
    st.zero_()
    assert m.reserve([2], [5]) == w4.W4_DEV_BAD_SLOT
    lib.w4_kv_reserve(d.table, d.lens, d.refs, _ints([2]), _ints([5]), 4, dev_status=st)
    assert int(st) == w4.W4_DEV_BAD_SLOT
    d.check(m)
    st.zero_()
    parents, children = [2, 2, 2, 2, 9, 1], [0, 0, 2, 7, 1, 4]
    assert m.fork(parents, children) == w4.W4_DEV_BAD_SLOT
    lib.w4_kv_fork(d.pool, d.table, d.lens, d.refs, _ints(parents), _ints(children), dev_status=st)
    assert int(st) == w4.W4_DEV_BAD_SLOT
    d.check(m)
    st.zero_()
    lib.w4_kv_free(d.table, d.lens, d.refs, _ints([0, 0, -3, 5]), dev_status=st)
    m.free([0])
    assert int(st) == w4.W4_DEV_BAD_SLOT
    d.check(m)
    # page ids that are none
    st.zero_()
    before = d.pool.clone()
    lib.w4_kv_copy_pages(d.pool, _ints([0, 12, -1, 3]), _ints([12, 1, 2, -5]), dev_status=st)
    assert int(st) == w4.W4_DEV_BAD_PAGE and torch.equal(d.pool, before)
    st.zero_()
    d.table[2, 1] = 99
    kv = torch.randn((6, 1, 8), device="cuda").bfloat16()
    offs = _ints([0, 0, 0, 6, 6, 6])
    lib.w4_kv_append(d.pool[0, 0], d.pool[0, 1], d.table, d.lens, kv, kv, offs, dev_status=st)
    assert int(st) == w4.W4_DEV_BAD_PAGE
    p = int(d.table[2, 0])
    assert torch.equal(d.pool[0, 0, p], kv[:4]) and torch.equal(d.pool[0, 1, p], kv[:4])
    st.zero_()
    lib.w4_kv_compact(d.pool, d.table, d.refs, table_out=torch.empty_like(d.table),
                      refs_out=torch.empty_like(d.refs), dev_status=st)
    assert int(st) == w4.W4_DEV_BAD_PAGE
    st.zero_()
    lib.w4_kv_append(d.pool[0, 0], d.pool[0, 1], d.table, d.lens, kv, kv,
                     _ints([0, -4, 9, 6, 6, 99]), dev_status=st)
    assert int(st) & w4.W4_DEV_BAD_SLOT


@pytest.mark.gpu
def test_a_captured_step_and_another_stream(lib):
    import torch
    m = _model((2, 2), 64, 8, 2, 16, 8, 8)
    m.reserve([0, 1], [37, 16])
    d = Device(m)
    parents, children = [0, 1, 0, 0], [2, 3, 4, 5]
    args = (_ints(parents), _ints(children))
    ws = torch.empty(lib.w4_kv_workspace_size(64, 4), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lib.w4_kv_fork(d.pool, d.table, d.lens, d.refs, *args, workspace=ws)
    s.synchronize()
    m.fork(parents, children)
    d.check(m)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.w4_kv_free(d.table, d.lens, d.refs, args[1])
        lib.w4_kv_fork(d.pool, d.table, d.lens, d.refs, *args, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    d.check(m)                                        # the same pages again


@pytest.mark.gpu
def test_strided_pages_and_inputs(lib):
    import torch
    P, page, Hkv, D = 6, 4, 2, 24
    big = torch.zeros((P, page, Hkv + 1, D + 8), device="cuda").half()
    both = torch.stack((big, big))
    kp, vp = both[0, :, :, :Hkv, :D], both[1, :, :, :Hkv, :D]
    table, lens = _ints([[4, 1, -1]]), _ints([7])
    src = torch.randn((5, 4, 2 * D), device="cuda").half()
    k, v = src[:, :2, :D], src[:, 2:, D:]
    lib.w4_kv_append(kp, vp, table, lens, k, v, _ints([0, 5]))
    got_k, got_v = kp[[4, 1]].flatten(0, 1), vp[[4, 1]].flatten(0, 1)
    assert torch.equal(got_k[2:7], k) and torch.equal(got_v[2:7], v)
    assert int((both != 0).sum()) == int((kp != 0).sum() + (vp != 0).sum())   # nothing beside them
    assert bool((got_k[:2] == 0).all()) and bool((got_k[7:] == 0).all())


def test_refusals_without_launching():
    from w4a16_moe_expert_sync_gb300 import build as w4build
    w4build.build()
    lib = w4.load_library()
    P = ctypes.c_void_p
    f, odd, odd4 = P(0x10000), P(0x10004), P(0x10002)
    big = 1 << 30
    assert lib.w4_kv_workspace_size(100, 7) == 16 + 4 * 200
    assert lib.w4_kv_workspace_size(1, 7) == 56
    # reserve
    ok = [f, 4, 8, f, f, 100, f, f, 2, 16, None, None]

    def bad(call, args, i, v):
        a = list(args)
        a[i] = v
        return call(*a)
    for i, v, rc in [(0, None, 1), (3, None, 1), (4, None, 1), (6, None, 1), (7, None, 1), (1, 0, 1),
                     (2, -1, 1), (5, 0, 1), (8, -1, 1), (9, 0, 1), (8, 1025, 2), (2, 1 << 29, 2),
                     (0, odd4, 3), (8, 0, 0)]:
        assert bad(lib.w4_kv_reserve, ok, i, v) == rc, (i, v)
    ok = [f, 4, 8, f, f, 100, f, 2, None, None]
    for i, v, rc in [(0, None, 1), (6, None, 1), (7, -1, 1), (5, 1 << 30, 2), (7, 0, 0)]:
        assert bad(lib.w4_kv_free, ok, i, v) == rc, (i, v)
    ok = [f, 4, 4096, f, 4, 8, f, f, 100, f, f, 2, 16, f, big, None, None]
    for i, v, rc in [(0, None, 1), (1, 0, 1), (2, 0, 1), (2, 4104, 2), (1, 65536, 2), (0, odd, 3),
                     (9, None, 1), (10, None, 1), (11, 1025, 2), (12, 0, 1), (13, None, 6),
                     (14, 815, 6), (13, odd, 3), (11, 0, 0)]:
        assert bad(lib.w4_kv_fork, ok, i, v) == rc, (i, v)
    ok = [f, 4, 4096, 100, f, f, 2, None, None]
    for i, v, rc in [(0, None, 1), (2, 4100, 2), (3, 0, 1), (4, None, 1), (0, odd, 3), (6, 0, 0)]:
        assert bad(lib.w4_kv_copy_pages, ok, i, v) == rc, (i, v)
    ok = [f, 4, 4096, f, 4, 8, f, 100, f, f, f, big, None, None]
    for i, v, rc in [(0, None, 1), (3, None, 1), (6, None, 1), (8, None, 1), (9, None, 1),
                     (9, odd4, 3), (10, None, 6), (11, 815, 6), (10, odd, 3)]:
        assert bad(lib.w4_kv_compact, ok, i, v) == rc, (i, v)
    ok = [f, f, 2048, 128, 64, 100, 16, 2, 64, f, 4, 8, f, f, 128, 64, f, 128, 64, f, 5, None, None]
    for i, v, rc in [(0, None, 1), (1, None, 1), (9, None, 1), (12, None, 1), (13, None, 1),
                     (19, None, 1), (6, 0, 1), (7, 0, 1), (8, 60, 2), (3, 100, 3), (14, 4, 3),
                     (0, odd, 3), (13, odd, 3), (20, -1, 1), (20, 0, 0)]:
        assert bad(lib.w4_kv_append, ok, i, v) == rc, (i, v)


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import torch
    t = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.w4_kv_free(t, t[:, 0], t[0], t[0])
    with pytest.raises(ValueError):
        w4.w4_kv_copy_pages(torch.zeros(3), t[0], t[0])
