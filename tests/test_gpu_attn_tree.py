"""w4_attn_tree against a plain float64 evaluation.  Tolerance as in
test_gpu_attention.py (the masks change nothing in it)."""
import ctypes
import random

import pytest

import w4a16_moe_expert_sync_gb300 as w4
from test_gpu_attention import _build

gpu = pytest.mark.gpu


def _tree(parents):
    """Each node's ancestors and itself as a number's bits."""
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | (1 << i))
    return seen


def _random_tree(r, n):
    return _tree([-1] + [r.randint(-1 if r.random() < 0.1 else 0, i - 1) for i in range(1, n)])


def _words(bits, words):
    import torch
    rows = [[(b >> 32 * i) & 0xFFFFFFFF for i in range(words)] for b in bits]
    return torch.tensor([[w - (1 << 32) if w >> 31 else w for w in row] for row in rows],
                        dtype=torch.int32, device="cuda").view(len(bits), words)


def _reference(c, bits):
    import torch
    q, (k, v) = c["q"].double(), c["cache"].unbind(0)
    Hq, D = q.shape[1:]
    page, Hkv = k.shape[1], k.shape[2]
    out, A, small = (torch.zeros_like(q) for _ in range(3))
    offs = c["q_offsets"].tolist()
    for b, L in enumerate(c["lens"].tolist()):
        nq = offs[b + 1] - offs[b]
        if nq == 0 or L == 0:
            continue
        pages = c["table"][b, :-(-L // page)].long()
        kk = k[pages].flatten(0, 1)[:L].double().repeat_interleave(Hq // Hkv, 1)
        vv = v[pages].flatten(0, 1)[:L].double().repeat_interleave(Hq // Hkv, 1)
        s = torch.einsum("thd,lhd->htl", q[offs[b]:offs[b + 1]], kk) / D ** 0.5
        seen = torch.ones((nq, L), dtype=torch.bool)
        for i in range(nq):
            for j in range(nq):
                seen[i, L - nq + j] = bool(bits[offs[b] + i] >> j & 1)
        s = s.masked_fill(~seen.to(s.device), float("-inf"))
        top = s.amax(-1, keepdim=True)
        e = torch.where(top.isinf(), 0.0, torch.exp(s - torch.where(top.isinf(), 0.0, top)))
        l = e.sum(-1, keepdim=True)
        p = torch.where(l > 0, e / torch.where(l > 0, l, 1.0), 0.0)
        rows = slice(offs[b], offs[b + 1])
        out[rows] = torch.einsum("htl,lhd->thd", p, vv)
        A[rows] = torch.einsum("htl,lhd->thd", p, vv.abs())
        small[rows] = vv.abs().sum(0)[None]
    return out, A, small


def _check(got, c, bits):
    import torch
    ref, A, small = _reference(c, bits)
    u = torch.finfo(got.dtype).eps / 2
    tol = u * (ref.abs() + A) * (1 + 2.0 ** -6) + 2.0 ** -14 * A
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25 * small
    assert not bool(got.isnan().any())
    bad = (got.double() - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:5].tolist())


def _run(lib, c, tree, **kw):
    return lib.w4_attn_tree(c["q"], c["cache"][0], c["cache"][1], c["table"], c["lens"],
                            c["q_offsets"], tree, c["group_offsets"], c["shared"],
                            max_q=c["max_q"], **kw)


CASES = [
    # befores, nodes, groups, shared, Hq, Hkv, D, page, type
    ([0], [1], [], [], 4, 2, 64, 16, "bfloat16"),
    ([1], [1], [], [], 1, 1, 128, 16, "float16"),
    ([203], [25], [], [], 16, 8, 128, 16, "bfloat16"),
    ([127], [33], [], [], 8, 2, 64, 32, "float16"),              # the window crosses tiles
    ([100, 5, 300], [31, 32, 33], [], [], 4, 4, 128, 64, "bfloat16"),
    ([0, 90], [64, 1], [], [], 6, 2, 64, 16, "float16"),         # a tree and nothing before it
    ([500, 510, 530], [7, 60, 21], [3], [480], 32, 4, 128, 64, "bfloat16"),
    ([77, 1700], [130, 65], [], [], 8, 1, 128, 16, "bfloat16"),  # five words, pairs of row tiles
    ([40, 41, 42, 300, 7], [3, 0, 9, 20, 2], [2, 2], [33, 40], 24, 4, 64, 16, "float16"),
    ([64] * 33, [5] * 33, [33], [64], 8, 2, 64, 32, "bfloat16"),
    ([250], [300], [], [], 2, 1, 64, 128, "bfloat16"),
]


@gpu
@pytest.mark.parametrize("befores,nodes,groups,shared,Hq,Hkv,D,page,dtype", CASES)
def test_trees(lib, befores, nodes, groups, shared, Hq, Hkv, D, page, dtype):
    import torch
    r = random.Random(sum(befores))
    c = _build([a + n for a, n in zip(befores, nodes)], nodes, groups, shared, Hq, Hkv, D, page,
               dtype, seed=len(nodes))
    bits = [b for n in nodes if n for b in _random_tree(r, n)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tree = _words(bits, -(-max(nodes) // 32))
    got = _run(lib, c, tree, dev_status=status)
    _check(got, c, bits)
    assert int(status) == 0
    # more words than are needed, with bits that are nobody's: no matter
    wide = torch.full((len(bits), tree.shape[1] + 2), -1, dtype=torch.int32, device="cuda")
    wide[:, :tree.shape[1]] = tree
    assert torch.equal(_run(lib, c, wide), got)
    for i, n in enumerate(nodes):                               # bits past a sequence's own
        for t in range(sum(nodes[:i]), sum(nodes[:i + 1])):
            b = bits[t] | ((1 << 32 * tree.shape[1]) - (1 << n))
            wide[t, :tree.shape[1]] = _words([b], tree.shape[1])[0]
    assert torch.equal(_run(lib, c, wide), got)


@gpu
@pytest.mark.parametrize("page,D,dtype", [(16, 128, "bfloat16"), (64, 64, "float16")])
def test_any_masks(lib, page, D, dtype):
    """Not trees: any bits, rows that see none of the new tokens, and rows that see
    nothing at all."""
    import torch
    r = random.Random(3)
    nodes = [40, 33, 70, 5]
    befores = [130, 0, 0, 9]
    c = _build([a + n for a, n in zip(befores, nodes)], nodes, [], [], 8, 2, D, page, dtype, seed=2)
    bits = [r.getrandbits(n) for n in nodes for _ in range(n)]
    for t in (0, 5, 41, 72, 73, 100, 140, 147):
        bits[t] = 0
    bits[74] = 1 << 69                                          # one key alone
    got = _run(lib, c, _words(bits, 3))
    _check(got, c, bits)
    for t in (41, 72, 73, 100, 140):
        assert bool((got[t] == 0).all())


@gpu
def test_masked_scores_may_be_anything(lib):
    """Keys of other branches whose scores are infinite or NaN do not reach a query."""
    import math
    import torch
    nodes = [20, 20]
    c = _build([300, 20], nodes, [], [], 4, 2, 128, 32, "bfloat16", seed=5)
    seen = [b for _ in nodes for b in _tree([-1] + [0, 0] + [1 + i % 2 for i in range(17)])]
    tree = _words(seen, 1)
    want = _run(lib, c, tree)
    for b, L in ((0, 300), (1, 20)):
        for j, v in ((3, math.inf), (6, math.nan)):             # leaves that only they see
            at = L - 20 + j
            c["cache"][0, int(c["table"][b, at // 32]), at % 32] = v
    got = _run(lib, c, tree)
    rest = [t for t in range(40) if t % 20 not in (3, 6)]
    assert torch.equal(got[rest], want[rest])


@gpu
def test_chains_are_causal_attention(lib):
    """A tree of one branch is causal attention; with every bit set it is the other
    attention without a mask, bit for bit."""
    import torch
    nodes = [9, 1, 50]
    c = _build([309, 41, 250], nodes, [2], [30], 16, 4, 128, 16, "float16", seed=6)
    bits = [b for n in nodes for b in _tree(list(range(-1, n - 1)))]
    _check(_run(lib, c, _words(bits, 2)), c, bits)
    causal = lib.w4_attn_shared_prefix(c["q"], c["cache"][0], c["cache"][1], c["table"], c["lens"],
                                       c["q_offsets"], c["group_offsets"], c["shared"], max_q=50)
    _check(causal, c, bits)
    everything = [(1 << n) - 1 for n in nodes for _ in range(n)]
    whole = lib.w4_attn_shared_prefix(c["q"], c["cache"][0], c["cache"][1], c["table"], c["lens"],
                                      c["q_offsets"], c["group_offsets"], c["shared"], max_q=50,
                                      causal=False)
    assert torch.equal(_run(lib, c, _words(everything, 2)), whole)


@gpu
def test_shared_prefix_that_reaches_into_the_tree(lib):
    """Members may share new tokens too: bits count there as well."""
    c = _build([100, 100], [30, 30], [2], [90], 8, 2, 64, 16, "bfloat16", seed=7)
    r = random.Random(9)
    bits = _random_tree(r, 30) + _random_tree(r, 30)
    _check(_run(lib, c, _words(bits, 1)), c, bits)


@gpu
def test_rows_of_no_sequence_strides_streams_and_graphs(lib):
    import torch
    nodes = [12, 20]
    c = _build([112, 420], nodes, [], [], 8, 2, 128, 64, "bfloat16", seed=8)
    r = random.Random(1)
    bits = [b for n in nodes for b in _random_tree(r, n)]
    tree = _words(bits, 1)
    want = _run(lib, c, tree)
    # queries as a view of a projection's output, three rows behind the last sequence
    qkv = torch.zeros((35, 12, 128), device="cuda").bfloat16()
    qkv[:32, :8] = c["q"]
    padded = torch.cat((tree, torch.full((3, 1), -1, dtype=torch.int32, device="cuda")))
    out = torch.full((35, 8, 128), 9.0, device="cuda").bfloat16()
    d = dict(c, q=qkv[:, :8])
    _run(lib, d, padded, out=out)
    assert torch.equal(out[:32], want) and bool((out[32:] == 9).all())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _run(lib, c, tree, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph, held = torch.cuda.CUDAGraph(), torch.empty_like(want)
    with torch.cuda.graph(graph):
        _run(lib, c, tree, out=held)
    alone = [1 << i for i in list(range(12)) + list(range(20))]
    tree.copy_(_words(alone, 1))
    graph.replay()
    torch.cuda.synchronize()
    _check(held, c, alone)


@gpu
def test_more_queries_than_max_q_are_flagged(lib):
    import torch
    c = _build([112, 420], [12, 20], [], [], 8, 2, 128, 64, "bfloat16", seed=8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bits = _tree(list(range(-1, 11))) + _tree(list(range(-1, 19)))
    _run(lib, c, _words(bits, 1))
    c["max_q"] = 12
    _run(lib, c, _words(bits, 1), dev_status=status)
    assert int(status) == w4.W4_DEV_BAD_SLOT


@gpu
@pytest.mark.parametrize("befores,nodes,Hq,Hkv,D,page", [
    ([5000, 300], [90, 40], 12, 2, 64, 16),                     # pairs, three S in turn
    ([700] * 6, [9] * 6, 4, 2, 64, 64),                         # single items
    ([3000], [70], 16, 4, 128, 16)])
def test_waits_that_give_up(lib, befores, nodes, Hq, Hkv, D, page):
    """The first keys never land: the status says so, and the context goes on."""
    import time
    import torch
    r = random.Random(4)
    c = _build([a + n for a, n in zip(befores, nodes)], nodes, [], [], Hq, Hkv, D, page, "bfloat16")
    tree = _words([b for n in nodes for b in _random_tree(r, n)], 3)
    want, hooks = _run(lib, c, tree), lib.load_library().w4_test_pipeline_hooks
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t = time.monotonic()
    try:
        hooks(2_000_000, 1)
        _run(lib, c, tree, dev_status=status)
        torch.cuda.synchronize()
    finally:
        hooks(0, 0)
    assert int(status) & w4.W4_DEV_PIPELINE_TIMEOUT and time.monotonic() - t < 30
    status.zero_()
    for _ in range(3):
        assert torch.equal(_run(lib, c, tree, dev_status=status), want)
    assert int(status) == 0


@gpu
@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 32)])
def test_long_sequences_and_many_calls(lib, D, page):
    """Items that are cut for many CTAs, several pieces a CTA, pages that are none, the same
    bits every time."""
    import torch
    r = random.Random(7)
    befores, nodes = [20000, 9000, 1, 130], [64, 100, 128, 3]
    c = _build([a + n for a, n in zip(befores, nodes)], nodes, [], [], 12, 2, D, page, "float16",
               poison=False, seed=3)
    bits = [b for n in nodes for b in _random_tree(r, n)]
    tree = _words(bits, 4)
    want = _run(lib, c, tree)
    _check(want, c, bits)
    assert all(torch.equal(_run(lib, c, tree), want) for _ in range(60))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c["table"][3, 0] = 10 ** 6
    got = _run(lib, c, tree, dev_status=status)
    assert int(status) == w4.W4_DEV_BAD_PAGE
    assert torch.equal(got[:292], want[:292])


def test_calls_refused():
    lib = w4.load_library()
    at = 0x10000

    def attn(q=at, tree=at, words=1, max_q=8, D=64, page=16, Hq=4, ws=0, out=at, T=8, B=1):
        return lib.w4_attn_tree(q, 256, 64, at, at, 2048, 128, 64, 8, page, at, 4, at, at, T, B,
                                max_q, tree, words, None, None, 0, Hq, 2, D, 0, ctypes.c_float(0.125),
                                at, ws, out, None, None)
    for kw, want in [(dict(tree=None), 1), (dict(words=0), 1), (dict(words=-1), 1),
                     (dict(words=1, max_q=33), 1), (dict(max_q=0), 1), (dict(q=None), 1),
                     (dict(out=None), 1), (dict(D=96), 2), (dict(page=8), 2), (dict(Hq=3), 2),
                     (dict(tree=at + 2), 3), (dict(q=at + 4), 3), (dict(), 6)]:
        assert attn(**kw) == want, kw
    assert attn(T=0) == 0 and attn(B=0) == 0
