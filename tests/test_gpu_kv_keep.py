"""w4_kv_keep against a plain model: every value of the pool and every length, exactly."""
import ctypes
import random

import pytest

import w4a16_moe_expert_sync_gb300 as w4

gpu = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(sizes):
    out = [0]
    for n in sizes:
        out.append(out[-1] + n)
    return out


def _build(befores, news, kept, layers, page, Hkv, D, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = [a + n for a, n in zip(befores, news)]
    need = [-(-n // page) for n in lens]
    P, W = sum(need) + 3, max(need + [1]) + 2
    perm = list(range(P))
    random.Random(seed).shuffle(perm)
    table, refs, at = [], [0] * P, 0
    for n in need:
        table.append(perm[at:at + n] + [-1] * (W - n))
        at += n
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    pool = torch.randn((layers, 2, P, page, Hkv, D), generator=g, device="cuda").bfloat16()
    return dict(pool=pool, table=_ints(table), lens=_ints(lens), refs=_ints(refs),
                q_offsets=_ints(_offsets(news)), kept=_ints([k for ks in kept for k in ks]),
                kept_offsets=_ints(_offsets([len(ks) for ks in kept])))


def _want(c, skip=()):
    """Pool and lengths after the call; the slots in `skip` are left alone."""
    pool, lens = c["pool"].clone(), c["lens"].tolist()
    page = pool.shape[3]
    table, qo, ko = c["table"].tolist(), c["q_offsets"].tolist(), c["kept_offsets"].tolist()
    kept = c["kept"].tolist()
    for b in range(len(lens)):
        if b in skip:
            continue
        base = lens[b] - (qo[b + 1] - qo[b])
        ks = kept[ko[b]:ko[b + 1]]
        for i, k in enumerate(ks):
            s, d = base + k, base + i
            pool[:, :, table[b][d // page], d % page] = \
                c["pool"][:, :, table[b][s // page], s % page]
        lens[b] = base + len(ks)
    return pool, lens


def _call(lib, c, **kw):
    return lib.w4_kv_keep(c["pool"], c["table"], c["lens"], c["refs"], c["q_offsets"], c["kept"],
                          c["kept_offsets"], **kw)


@gpu
@pytest.mark.parametrize("befores,news,kept,layers,page,Hkv,D", [
    ([5], [1], [[0]], 1, 16, 1, 8),
    ([0], [1], [[]], 2, 16, 2, 64),
    ([16], [9], [[0, 3, 8]], 3, 16, 2, 64),
    ([15, 0, 31], [4, 3, 2], [[1, 2, 3], [], [1]], 2, 16, 2, 64),
    ([40, 3, 7, 100], [25, 0, 64, 30], [[0, 1, 5, 24], [], list(range(64)), [29]], 4, 32, 4, 128),
    ([1000], [600], [list(range(20, 600, 2))], 2, 64, 1, 64),       # more than are staged at once
    ([7] * 90, [33] * 90, None, 5, 16, 8, 128),
    ([3], [40], [[7, 8, 9, 30]], 40, 5, 8, 128),                    # a cluster of eight, odd pages
])
@pytest.mark.parametrize("in_place", [False, True])
def test_kept_tokens(lib, befores, news, kept, layers, page, Hkv, D, in_place):
    import torch
    if kept is None:
        r = random.Random(1)
        kept = [sorted(r.sample(range(n), r.randint(0, n))) for n in news]
    c = _build(befores, news, kept, layers, page, Hkv, D)
    pool, lens = _want(c)
    state = [c[n].clone() for n in ("table", "refs", "lens")]
    status, out = _ints([0]), c["lens"] if in_place else torch.full_like(c["lens"], -9)
    got = _call(lib, c, dev_status=status, **({} if in_place else dict(lens_out=out)))
    assert got is out and out.tolist() == lens and int(status) == 0
    assert torch.equal(c["pool"], pool)
    assert torch.equal(c["table"], state[0]) and torch.equal(c["refs"], state[1])
    if not in_place:
        assert torch.equal(c["lens"], state[2])


@gpu
def test_what_makes_no_sense_leaves_its_slot(lib):
    import torch

    def run(change):
        c = _build([20, 30, 40], [10, 10, 10], [[1, 4], [0, 3, 9], [5]], 2, 16, 2, 64)
        change(c)
        status = _ints([0])
        before = c["lens"].clone()
        pool, lens = _want(c, skip=(1,))
        _call(lib, c, dev_status=status)
        assert c["lens"].tolist() == lens and torch.equal(c["pool"], pool)
        assert int(c["lens"][1]) == int(before[1])
        return int(status)

    def put(name, i, v):
        return lambda c: c[name].view(-1)[i].fill_(v)
    for i, v in ((2, 3), (3, 0), (3, -1), (4, 10), (3, 9)):          # kept: not ascending, outside
        assert run(put("kept", i, v)) == w4.W4_DEV_BAD_SLOT
    for n in (9, -3, 0):                                            # fewer tokens than are new
        assert run(put("lens", 1, n)) == w4.W4_DEV_BAD_SLOT
    assert run(put("lens", 1, 10 ** 6)) == w4.W4_DEV_BAD_SLOT       # beyond the table

    def hole(c):
        c["table"][1, 31 // 16] = -1
    assert run(hole) == w4.W4_DEV_BAD_PAGE

    def shared(c):
        c["refs"][c["table"][1, 31 // 16].long()] = 2
    assert run(shared) == w4.W4_DEV_BAD_SLOT


@gpu
def test_pages_that_are_only_read_may_be_shared(lib):
    """What is written belongs to the slot alone; a token in its place is not written."""
    import torch
    c = _build([32], [20], [[0, 1, 17]], 2, 16, 1, 64)
    c["refs"][c["table"][0, :2].long()] = 3                         # the prefix
    pool, lens = _want(c)
    status = _ints([0])
    _call(lib, c, dev_status=status)
    assert int(status) == 0 and c["lens"].tolist() == lens and torch.equal(c["pool"], pool)
    # nothing moves: the new tokens' pages may be anyone's
    c = _build([32], [20], [[0, 1, 2]], 2, 16, 1, 64)
    c["refs"].fill_(2)
    before = c["pool"].clone()
    _call(lib, c, dev_status=status)
    assert int(status) == 0 and c["lens"].tolist() == [35] and torch.equal(c["pool"], before)


@gpu
def test_captured(lib):
    """Replayed with other lists and lengths in the same memory."""
    import torch
    lists = [[[0, 2], [1, 4, 5]], [[3, 5], [0, 1, 2]]]
    c = _build([20, 9], [6, 6], lists[0], 2, 16, 2, 64)
    before = c["lens"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(lib, c)
    for kept in lists:
        c["kept"].copy_(_ints([k for ks in kept for k in ks]))
        c["lens"].copy_(before)
        pool, lens = _want(c)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c["pool"], pool) and c["lens"].tolist() == lens


def test_calls_refused():
    lib = w4.load_library()
    at = 0x10000

    def keep(pool=at, planes=2, pb=2048, table=at, B=2, W=4, lens=at, refs=at, P=8, offs=at, kept=at,
             ko=at, n=3, page=16, out=at):
        return lib.w4_kv_keep(pool, planes, ctypes.c_int64(pb), table, B, W, lens, refs, P, offs,
                              kept, ko, n, page, out, None, None)
    for kw, want in [(dict(pool=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
                     (dict(refs=None), 1), (dict(offs=None), 1), (dict(kept=None), 1),
                     (dict(ko=None), 1), (dict(out=None), 1), (dict(planes=0), 1), (dict(B=-1), 1),
                     (dict(n=-1), 1), (dict(page=0), 1), (dict(pb=2040), 2), (dict(W=1 << 30), 2),
                     (dict(W=1 << 28, page=16, pb=256), 2), (dict(pool=at + 8), 3),
                     (dict(offs=at + 2), 3), (dict(kept=at + 1), 3), (dict(out=at + 2), 3)]:
        assert keep(**kw) == want, kw
    assert keep(B=0) == 0


def test_binding_refuses_before_anything_is_launched():
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.w4_kv_keep(torch.zeros((1, 4, 16, 1, 8)), i.view(1, 2), i[:1], i, i, i, i)
