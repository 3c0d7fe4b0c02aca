"""w4_attn_shared_prefix against a plain float64 evaluation.

Tolerance, derived beforehand, with A = sum_l p_l |v_l| per output element and
u the half step of the type (bf16 2^-8, fp16 2^-11): the rounding of every
weight p_l to the type (u A), the rounding of the result (u |o|), fp32 scores,
exponentials and sums (below 2^-14 A: a score is at most ~30 with an error of
2^-20, the exponential 2^-22), and for fp16 the weights below its normal range
(at most 2^-25 absolute, against a largest weight of at least 1)."""
import pytest


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _build(lens, nqs, groups, shared, Hq, Hkv, D, page, dtype, seed=0, poison=True, spread=1.0):
    """A cache with the pages in random order; everything that no token fills
    holds NaN.  groups: sizes; shared: lengths."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, used, copies, b = [], 0, [], 0
    sizes = list(groups) + [1] * (len(lens) - sum(groups))
    cuts = list(shared) + [0] * (len(sizes) - len(shared))
    for n, s in zip(sizes, cuts):
        full = s // page
        first = list(range(used, used + full))
        used += full
        for i in range(n):
            mine = -(-lens[b] // page) - full if lens[b] >= s else 0
            ids = list(range(used, used + mine))
            used += mine
            if i == 0:
                head = ids[:1]
            elif s % page and ids:
                copies.append((head[0], ids[0], s % page))
            rows.append((first + ids)[:-(-lens[b] // page)])
            b += 1
    P = used + 3
    perm = torch.randperm(P, generator=g, device="cuda").tolist()
    W = max([len(r) for r in rows] + [1]) + 1
    table = [[perm[p] for p in r] + [-1] * (W - len(r)) for r in rows]
    cache = torch.full((2, P, page, Hkv, D), float("nan") if poison else 0.0, device="cuda")
    for i, r in enumerate(table):
        for j, p in enumerate(r):
            n = min(page, lens[i] - j * page)
            if p >= 0 and bool(cache[0, p, 0, 0, 0].isnan()) | (not poison):
                cache[:, p, :n] = torch.randn((2, n, Hkv, D), generator=g, device="cuda") * spread
    for a, c, t in copies:
        cache[:, perm[c], :t] = cache[:, perm[a], :t]
    cache = cache.to(getattr(torch, dtype))
    T = sum(nqs)
    q = (torch.randn((T, Hq, D), generator=g, device="cuda") * 1.5).to(cache.dtype)
    offs = [0]
    for n in nqs:
        offs.append(offs[-1] + n)
    go = [0]
    for n in groups:
        go.append(go[-1] + n)
    return dict(q=q, cache=cache, table=_ints(table), lens=_ints(lens), q_offsets=_ints(offs),
                group_offsets=_ints(go) if groups else None,
                shared=_ints(list(shared)) if groups else None, max_q=max(nqs + [1]))


def _reference(c, causal):
    """(out, A, weight of the absolute term) in float64."""
    import torch
    q, (k, v) = c["q"].double(), c["cache"].unbind(0)
    T, Hq, D = q.shape
    page, Hkv = k.shape[1], k.shape[2]
    out = torch.zeros_like(q)
    A, small = torch.zeros_like(q), torch.zeros_like(q)
    offs = c["q_offsets"].tolist()
    for b, L in enumerate(c["lens"].tolist()):
        nq = offs[b + 1] - offs[b]
        if nq == 0 or L == 0:
            continue
        pages = c["table"][b, :-(-L // page)].long()
        kk = k[pages].flatten(0, 1)[:L].double().repeat_interleave(Hq // Hkv, 1)
        vv = v[pages].flatten(0, 1)[:L].double().repeat_interleave(Hq // Hkv, 1)
        s = torch.einsum("thd,lhd->htl", q[offs[b]:offs[b + 1]], kk) / D ** 0.5
        if causal:
            lim = L - nq + 1 + torch.arange(nq, device="cuda")
            s = s.masked_fill(torch.arange(L, device="cuda")[None] >= lim[:, None], float("-inf"))
        top = s.amax(-1, keepdim=True)
        e = torch.where(top.isinf(), 0.0, torch.exp(s - torch.where(top.isinf(), 0.0, top)))
        l = e.sum(-1, keepdim=True)
        p = torch.where(l > 0, e / torch.where(l > 0, l, 1.0), 0.0)
        out[offs[b]:offs[b + 1]] = torch.einsum("htl,lhd->thd", p, vv)
        A[offs[b]:offs[b + 1]] = torch.einsum("htl,lhd->thd", p, vv.abs())
        small[offs[b]:offs[b + 1]] = vv.abs().sum(0)[None]
    return out, A, small


def _run(lib, c, causal, **kw):
    return lib.w4_attn_shared_prefix(c["q"], c["cache"][0], c["cache"][1], c["table"], c["lens"],
                                     c["q_offsets"], c["group_offsets"], c["shared"],
                                     max_q=c["max_q"], causal=causal, **kw)


def _check(got, c, causal):
    import torch
    ref, A, small = _reference(c, causal)
    u = torch.finfo(got.dtype).eps / 2
    tol = u * (ref.abs() + A) * (1 + 2.0 ** -6) + 2.0 ** -14 * A
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25 * small
    bad = (got.double() - ref).abs() > tol
    assert not bool(got.isnan().any())
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:5].tolist())


CASES = [
    # lens, queries, group sizes, shared, Hq, Hkv, D, page, dtype, causal
    ([1], [1], [], [], 1, 1, 64, 16, "bfloat16", True),
    ([17], [1], [], [], 2, 1, 128, 16, "bfloat16", True),
    ([128], [1], [], [], 4, 4, 128, 128, "float16", False),
    ([129, 127, 1], [1, 1, 1], [], [], 8, 2, 128, 16, "bfloat16", True),
    ([300], [300], [], [], 2, 1, 64, 32, "bfloat16", True),
    ([300], [300], [], [], 3, 1, 128, 64, "float16", False),
    ([200, 200], [1, 1], [2], [192], 4, 2, 128, 16, "bfloat16", True),
    ([203, 240, 203], [1, 1, 1], [3], [203], 16, 8, 128, 16, "bfloat16", True),
    ([1000, 1100, 1033, 2000], [1, 2, 3, 0], [2, 2], [777, 999], 24, 4, 64, 16, "float16", True),
    ([5, 900, 640, 17, 4, 0], [5, 40, 1, 17, 2, 0], [1, 2], [0, 513], 6, 2, 128, 32, "bfloat16",
     True),
    ([2000] * 20, [1] * 20, [20], [1900], 8, 1, 128, 64, "bfloat16", True),
    ([640] * 3, [130, 64, 200], [3], [400], 4, 2, 128, 128, "float16", False),
    ([3000] * 140, [1] * 140, [70, 70], [2999, 2900], 8, 4, 64, 16, "bfloat16", True),
    ([9000], [1], [], [], 32, 4, 128, 64, "bfloat16", True),
    ([40000, 40007], [2, 2], [2], [39990], 5, 1, 128, 16, "bfloat16", True),
    ([33] * 300, [1] * 300, [], [], 4, 4, 128, 16, "bfloat16", True),
    ([700, 700], [1, 1], [2], [650], 200, 1, 64, 32, "bfloat16", False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_matches_float64(lib, case):
    import torch
    *shape, causal = case
    c = _build(*shape, seed=len(shape[0]))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(lib, c, causal, dev_status=st)
    assert int(st) == 0
    _check(got, c, causal)
    # a dirty workspace, the same bits
    need = lib.w4_attn_shared_prefix_workspace_size(
        got.shape[0], len(shape[0]), len(shape[2]), c["max_q"], got.shape[1], shape[5], shape[6])
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(_run(lib, c, causal, workspace=ws), got)


@pytest.mark.gpu
def test_queries_that_see_nothing_are_zero(lib):
    c = _build([2, 40, 0], [5, 1, 3], [], [], 4, 2, 64, 16, "bfloat16")
    got = _run(lib, c, True)
    _check(got, c, True)
    assert bool((got[:3] == 0).all()) and bool((got[6:] == 0).all())


@pytest.mark.gpu
def test_large_scores_and_a_late_maximum(lib):
    """Scores that grow along the sequence move the reference many times."""
    import torch
    c = _build([700, 690], [1, 1], [2], [600], 4, 2, 128, 16, "float16", poison=False, spread=1.0)
    pages = c["table"][0, :44].long()
    k = c["cache"][0]
    ramp = torch.linspace(0, 6, 44, device="cuda").half()
    for i, p in enumerate(pages.tolist()):
        if p >= 0:
            k[p] = k[p] * 0.1 + c["q"][0, 0].sign() * ramp[i]
    c["cache"][0][c["table"][1, 37:44].long()] = c["cache"][0][c["table"][0, 37:44].long()]
    got = _run(lib, c, True)
    _check(got, c, True)


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [45, 250, 271, 17])
@pytest.mark.parametrize("nq", [1, 40])
def test_a_prefix_is_read_through_the_first_alone(lib, shared, nq):
    """The others' own pages may hold anything before the shared length, and
    their tables nothing where a page lies wholly before it."""
    import torch
    page = 32
    c = _build([shared + 60, shared + nq, shared + 130], [nq, nq, nq], [3], [shared], 8, 2, 64,
               page, "bfloat16", seed=shared)
    want = _run(lib, c, True)
    _check(want, c, True)
    full, part = divmod(shared, page)
    for b in (1, 2):
        c["table"][b, :full] = -1
        if part:
            c["cache"][:, c["table"][b, full].long(), :part] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert torch.equal(_run(lib, c, True, dev_status=st), want) and int(st) == 0


@pytest.mark.gpu
def test_sharing_changes_nothing_but_rounding(lib):
    import torch
    c = _build([1500] * 6, [1] * 6, [6], [1300], 8, 2, 128, 16, "bfloat16", seed=3)
    shared = _run(lib, c, True)
    c["group_offsets"] = c["shared"] = None
    _check(_run(lib, c, True), c, True)
    _check(shared, c, True)
    assert not torch.equal(shared, torch.zeros_like(shared))


@pytest.mark.gpu
def test_strided_inputs_other_stream_and_graph(lib):
    import torch
    c = _build([450, 500, 470], [2, 1, 3], [3], [430], 8, 4, 128, 32, "bfloat16", seed=4)
    want = _run(lib, c, True)
    T, Hq, D = c["q"].shape
    qkv = torch.randn((T, Hq + 8, D), device="cuda").bfloat16()
    qkv[:, 4:4 + Hq] = c["q"]
    big = torch.full((2, 5, *c["cache"].shape[1:]), float("nan"), device="cuda").bfloat16()
    big[:, 3] = c["cache"]
    big = big.transpose(3, 4).contiguous().transpose(3, 4)       # heads outside tokens
    d = dict(c, q=qkv[:, 4:4 + Hq], cache=big[:, 3])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = _run(lib, d, True)
    s.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(lib.w4_attn_shared_prefix_workspace_size(T, 3, 1, 3, Hq, 4, D),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(lib, d, True, workspace=ws, out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # the graph reads lengths when it runs: one token less
    c["lens"] -= 1
    graph.replay()
    torch.cuda.synchronize()
    _check(out, c, True)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_layouts_of_the_pages(lib, page, D):
    """Heads inside the tokens, outside them, outside them in a wider pool, and
    tokens wider than their heads: the same values, the same result."""
    import torch
    c = _build([450, 20, 470, 300], [2, 1, 3, 1], [3], [17], 8, 4, D, page, "bfloat16", seed=page)
    want = _run(lib, c, True)
    _check(want, c, True)
    P, Hkv = c["cache"].shape[1], 4
    outside = c["cache"].transpose(2, 3).contiguous().transpose(2, 3)
    wider = torch.full((2, P, Hkv + 2, page, D), float("nan"), device="cuda").bfloat16()
    wider = wider[:, :, 1:1 + Hkv].transpose(2, 3)
    tokens = torch.full((2, P, page, Hkv + 1, D), float("nan"), device="cuda").bfloat16()[:, :, :, 1:]
    apart = torch.full((2, P, page, Hkv, D + 8), float("nan"), device="cuda").bfloat16()[..., :D]
    for x in (outside, wider, tokens, apart):
        x.copy_(c["cache"])
        assert torch.equal(_run(lib, dict(c, cache=x), True), want)


@pytest.mark.gpu
def test_bad_inputs_on_the_device_are_flagged(lib):
    import torch
    good = _build([100, 90, 80], [1, 1, 1], [], [], 4, 2, 64, 16, "bfloat16", seed=6)
    want = _run(lib, good, True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad, rows in ((-7, [0, 2]), (10 ** 6, [0, 2])):
        c = dict(good, table=good["table"].clone())
        c["table"][1, 2] = bad
        st.zero_()
        got = _run(lib, c, True, dev_status=st)
        assert int(st) == lib.W4_DEV_BAD_PAGE and torch.equal(got[rows], want[rows])
    c = dict(good, lens=_ints([100, -5, 80]))
    st.zero_()
    got = _run(lib, c, True, dev_status=st)
    assert int(st) == lib.W4_DEV_BAD_SLOT and torch.equal(got[[0, 2]], want[[0, 2]])
    c = dict(good, q_offsets=_ints([0, 1, 9, 3]))
    st.zero_()
    _run(lib, c, True, dev_status=st)          # nothing is computed
    assert int(st) == lib.W4_DEV_BAD_SLOT
    c = dict(good, q_offsets=_ints([0, 2, 3, 3]))
    st.zero_()
    got = _run(lib, c, True, dev_status=st)    # two queries where max_q is one
    assert int(st) == lib.W4_DEV_BAD_SLOT and not bool(got[2].isnan().any())
    c = dict(good, group_offsets=_ints([0, 7]), shared=_ints([64]))
    st.zero_()
    _run(lib, c, True, dev_status=st)
    assert int(st) & lib.W4_DEV_BAD_SLOT


@pytest.mark.gpu
def test_empty_batch(lib):
    import torch
    c = _build([10], [1], [], [], 4, 2, 64, 16, "bfloat16")
    c["q"], c["q_offsets"] = c["q"][:0], _ints([0, 0])
    assert _run(lib, c, True).shape == (0, 4, 64)


def test_binding_refuses_what_does_not_fit():
    import torch

    import w4a16_moe_expert_sync_gb300 as w4
    z = torch.zeros((2, 16, 1, 64))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.w4_attn_shared_prefix(z[:, 0], z, z, i[None], i, i)


@pytest.mark.gpu
def test_binding_refuses_other_types_and_shapes(lib):
    import torch
    c = _build([100, 90], [1, 2], [2], [64], 4, 2, 64, 16, "bfloat16", seed=1)
    k = c["cache"][0]
    assert _run(lib, c, True).shape == c["q"].shape
    for bad in (dict(q=c["q"].half()), dict(q=c["q"][:, :, :32]), dict(q=c["q"].float()),
                dict(q=c["q"][0]), dict(table=c["table"].long()), dict(table=c["table"][:1]),
                dict(table=c["table"][:, ::2]), dict(lens=c["lens"].float()),
                dict(lens=c["lens"][:1]), dict(q_offsets=c["q_offsets"].cpu()),
                dict(group_offsets=c["group_offsets"].long()), dict(shared=None),
                dict(shared=c["shared"].repeat(2)), dict(cache=torch.stack((k, k)).float())):
        with pytest.raises(ValueError):
            _run(lib, dict(c, **bad), True)
    for bad in (dict(out=c["q"][:2]), dict(out=torch.empty_like(c["q"]).half()),
                dict(dev_status=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            _run(lib, c, True, **bad)
