"""w4_qk_norm_rope and w4_kv_append_rope against a plain float64 evaluation.

Tolerance, derived beforehand.  With a, b a pair's normed values and A the amplitude:
the norm in fp32 (256 squares summed in 13 steps at most, halved by the root, its
reciprocal to 2^-22, two products) is off by less than 2^-20 relative; the cosine and
sine by less than 2^-22 (an angle of up to a half turn in fp32, sincospif to an ulp, the
amplitude's product); two products and a sum.  Together less than 2^-18 (|a| + |b|) A,
and the result's rounding, u |ref| with u half a step of the type (fp16: 2^-25 at least,
its subnormals' half step)."""
import math

import pytest

import w4a16_moe_expert_sync_gb300 as w4

gpu = pytest.mark.gpu


def _ints(v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _frequencies(rot, base=10000.0):
    import torch
    return torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)


def _reference(x, weight, positions, freq, interleaved, amplitude, eps):
    """(result, bound of the fp32 error) in float64."""
    import torch
    u = x.double()
    if weight is not None:
        u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + eps) * weight.double()
    rot = 2 * freq.numel()
    t = positions.double()[:, None, None] * freq.to(x.device)
    c, s = torch.cos(t) * amplitude, torch.sin(t) * amplitude
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = u[..., i], u[..., j]
    ref, mass = u.clone(), u.abs()
    ref[..., i], ref[..., j] = a * c - b * s, a * s + b * c
    mass[..., i] = mass[..., j] = (a.abs() + b.abs()) * abs(amplitude)
    return ref, mass * 2.0 ** -18


def _check(got, ref, slack):
    import torch
    tol = torch.finfo(got.dtype).eps / 2 * ref.abs() * (1 + 2.0 ** -10) + slack
    if got.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:5].tolist())


def _inputs(T, Hq, Hkv, D, dtype, seed=0, norm=True):
    """Queries, keys and values as views of one projection's output, and weights."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, dtype)
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda")
    x = (x * torch.exp(torch.randn((T, Hq + 2 * Hkv, 1), generator=g, device="cuda"))).to(dt)
    w = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt) if norm else None
         for _ in range(2)]
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], w


@gpu
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,interleaved,dtype,norm", [
    (1, 16, 8, 128, 128, False, "bfloat16", True),
    (1, 1, 1, 8, 0, False, "bfloat16", True),
    (1, 1, 1, 16, 16, True, "float16", True),
    (7, 4, 2, 64, 64, True, "bfloat16", True),
    (33, 5, 1, 64, 32, False, "float16", False),
    (130, 3, 3, 80, 80, False, "bfloat16", True),
    (65, 6, 2, 96, 48, True, "float16", True),
    (19, 8, 1, 200, 112, False, "bfloat16", True),
    (257, 40, 8, 128, 64, False, "float16", True),
    (5, 32, 4, 256, 256, True, "bfloat16", False),
    (1023, 2, 1, 72, 16, False, "bfloat16", True),
    (3, 300, 7, 24, 16, True, "float16", True),
])
def test_norm_and_rotation(lib, T, Hq, Hkv, D, rot, interleaved, dtype, norm):
    import torch
    q, k, _, (wq, wk) = _inputs(T, Hq, Hkv, D, dtype, T + D, norm)
    pos = torch.randint(0, 100000, (T,), device="cuda", dtype=torch.int32)
    got = lib.w4_qk_norm_rope(q, k, pos, lib.w4_rope_steps(rot), q_weight=wq, k_weight=wk, eps=1e-5,
                              interleaved=interleaved, amplitude=1.25)
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        assert y.shape == x.shape and y.is_contiguous()
        _check(y, *_reference(x, w, pos, _frequencies(rot) if rot else _frequencies(0),
                              interleaved, 1.25, 1e-5))


@gpu
def test_positions_far_and_negative(lib):
    import torch
    pos = _ints([0, 1, -1, 2 ** 23, -2 ** 23, 2 ** 23 + 1, 1048575, 7])
    q, k, _, _ = _inputs(8, 2, 1, 128, "bfloat16", 3, False)
    got = lib.w4_qk_norm_rope(q, k, pos, lib.w4_rope_steps(128, 500000.0))
    f = _frequencies(128, 500000.0)
    _check(got[0], *_reference(q, None, pos, f, False, 1.0, 0.0))
    _check(got[1], *_reference(k, None, pos, f, False, 1.0, 0.0))
    # the ends of int32 are as good as any other position: finite, and their opposite turns back
    pos = _ints([2 ** 31 - 1, -2 ** 31 + 1] * 4)
    there = lib.w4_qk_norm_rope(q, k, pos, lib.w4_rope_steps(128))[0]
    back = lib.w4_qk_norm_rope(there, k, -pos, lib.w4_rope_steps(128))[0]
    # twice the bf16 rounding of a pair's values, turned
    pair = q.double().unflatten(-1, (2, 64)).norm(dim=-2, keepdim=True).expand(-1, -1, 2, -1)
    assert bool(((back.double() - q.double()).abs().unflatten(-1, (2, 64)) <=
                 2.0 ** -6.9 * pair).all())


@gpu
def test_one_of_the_two_alone_and_one_norm(lib):
    import torch
    q, k, _, (wq, wk) = _inputs(9, 4, 2, 64, "bfloat16", 5)
    pos, steps = torch.arange(9, device="cuda", dtype=torch.int32), lib.w4_rope_steps(64)
    both = lib.w4_qk_norm_rope(q, k, pos, steps, q_weight=wq)
    assert torch.equal(lib.w4_qk_norm_rope(q, k[:, :0], pos, steps, q_weight=wq)[0], both[0])
    assert torch.equal(lib.w4_qk_norm_rope(q[:, :0], k, pos, steps)[1], both[1])
    f = _frequencies(64)
    _check(both[0], *_reference(q, wq, pos, f, False, 1.0, 1e-6))
    _check(both[1], *_reference(k, None, pos, f, False, 1.0, 1e-6))
    none = lib.w4_qk_norm_rope(q[:0], k[:0], pos[:0], steps)
    assert none[0].shape == (0, 4, 64) and none[1].shape == (0, 2, 64)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_strided_results(lib, interleaved):
    """Over the inputs themselves, and into heads-first memory."""
    import torch
    q, k, v, (wq, wk) = _inputs(70, 6, 2, 128, "float16", 6)
    pos, steps = torch.arange(70, device="cuda", dtype=torch.int32) + 400, lib.w4_rope_steps(64)
    kw = dict(q_weight=wq, k_weight=wk, interleaved=interleaved)
    want = lib.w4_qk_norm_rope(q, k, pos, steps, **kw)
    qh = torch.full((6, 70, 136), 7.0, device="cuda").half()
    kh = torch.full((2, 70, 136), 7.0, device="cuda").half()
    lib.w4_qk_norm_rope(q, k, pos, steps, q_out=qh[..., :128].transpose(0, 1),
                        k_out=kh[..., :128].transpose(0, 1), **kw)
    assert torch.equal(qh[..., :128].transpose(0, 1), want[0])
    assert torch.equal(kh[..., :128].transpose(0, 1), want[1])
    assert bool((qh[..., 128:] == 7).all()) and bool((kh[..., 128:] == 7).all())
    values = v.clone()
    got = lib.w4_qk_norm_rope(q, k, pos, steps, q_out=q, k_out=k, **kw)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(v, values)


@gpu
def test_zeros_infinities_and_nan_stay_in_their_head(lib):
    import torch
    q, k, _, (wq, wk) = _inputs(4, 4, 2, 64, "bfloat16", 8)
    q = q.clone()
    pos, steps = torch.arange(4, device="cuda", dtype=torch.int32), lib.w4_rope_steps(64)
    want = lib.w4_qk_norm_rope(q, k, pos, steps, q_weight=wq, k_weight=wk)[0]
    q[0, 1], q[1, 2, 5], q[2, 3, 63] = 0.0, math.nan, math.inf
    got = lib.w4_qk_norm_rope(q, k, pos, steps, q_weight=wq, k_weight=wk)[0]
    assert bool((got[0, 1] == 0).all())
    assert bool(got[1, 2].isnan().all()) and bool(got[2, 3].isnan().any())
    same = torch.ones((4, 4), dtype=torch.bool)
    same[0, 1] = same[1, 2] = same[2, 3] = False
    assert torch.equal(got[same], want[same])


def _sequences(news, befores, page, Hkv, D, dtype, seed=0, interleave=False):
    """Pages of a batch, as views of a pool with both planes (interleave: side by side
    in one page), everything in it a known pattern."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-(a + n) // page) for a, n in zip(befores, news)]
    P, W = sum(need) + 4, max(need + [1]) + 1
    perm = torch.randperm(P, generator=g, device="cuda").tolist()
    table, at = [], 0
    for n in need:
        table.append(perm[at:at + n] + [-1] * (W - n))
        at += n
    shape = (P, page, 2, Hkv, D) if interleave else (2, P, page, Hkv, D)
    pool = torch.randn(shape, generator=g, device="cuda").to(getattr(torch, dtype))
    kp, vp = (pool[:, :, 0], pool[:, :, 1]) if interleave else (pool[0], pool[1])
    offs = [0]
    for n in news:
        offs.append(offs[-1] + n)
    return dict(pool=pool, kp=kp, vp=vp, table=_ints(table),
                lens=_ints([a + n for a, n in zip(befores, news)]), q_offsets=_ints(offs))


@gpu
@pytest.mark.parametrize("news,befores,page,Hq,Hkv,D,rot,interleaved,dtype,drafts", [
    ([1], [0], 16, 4, 2, 64, 64, False, "bfloat16", False),
    ([1, 1, 1], [15, 16, 17], 16, 16, 8, 128, 128, False, "bfloat16", False),
    ([3, 0, 40, 1], [0, 9, 30, 63], 32, 4, 4, 64, 32, True, "float16", False),
    ([129, 0, 0, 65, 1], [127, 5, 0, 1, 700], 64, 6, 1, 128, 128, False, "bfloat16", True),
    ([7, 500, 1], [3, 3, 3], 5, 2, 1, 72, 48, False, "float16", True),
    ([12] * 70, list(range(70)), 16, 8, 2, 256, 64, True, "bfloat16", False),
])
@pytest.mark.parametrize("side_by_side", [False, True])
def test_append(lib, news, befores, page, Hq, Hkv, D, rot, interleaved, dtype, drafts, side_by_side):
    """Queries and keys as w4_qk_norm_rope gives them, at their places, and nothing else
    in the pool or behind the last sequence changed."""
    import torch
    pad = 3
    T = sum(news) + pad
    q, k, v, (wq, wk) = _inputs(T, Hq, Hkv, D, dtype, T)
    c = _sequences(news, befores, page, Hkv, D, dtype, T, side_by_side)
    steps, status = lib.w4_rope_steps(rot), _ints([0])
    where = [(b, a + i) for b, (a, n) in enumerate(zip(befores, news)) for i in range(n)]
    place = _ints([p for _, p in where] + [0] * pad)
    pos = torch.randint(0, 5000, (T,), device="cuda", dtype=torch.int32) if drafts else None
    kw = dict(q_weight=wq, k_weight=wk, interleaved=interleaved, amplitude=0.75)
    want_q, want_k = lib.w4_qk_norm_rope(q, k, pos if drafts else place, steps, **kw)
    want = c["pool"].clone()
    planes = (want[:, :, 0], want[:, :, 1]) if side_by_side else (want[0], want[1])
    table = c["table"].tolist()
    for t, (b, p) in enumerate(where):
        for plane, x in zip(planes, (want_k, v)):
            plane[table[b][p // page], p % page] = x[t]
    out = torch.full((T, Hq, D), 5.0, device="cuda").to(q.dtype)
    got = lib.w4_kv_append_rope(c["kp"], c["vp"], c["table"], c["lens"], q, k, v, c["q_offsets"],
                                steps, positions=pos, q_out=out, dev_status=status, **kw)
    assert got is out and int(status) == 0
    assert torch.equal(out[:T - pad], want_q[:T - pad]) and bool((out[T - pad:] == 5).all())
    assert torch.equal(c["pool"], want)


@gpu
def test_append_flags_what_makes_no_sense(lib):
    import torch
    q, k, v, (wq, wk) = _inputs(6, 4, 2, 64, "bfloat16", 1)
    steps = lib.w4_rope_steps(64)

    def run(change):
        c = _sequences([3, 3], [20, 30], 16, 2, 64, "bfloat16", 1)
        change(c)
        before, status = c["pool"].clone(), _ints([0])
        out = torch.full((6, 4, 64), 5.0, device="cuda").bfloat16()
        lib.w4_kv_append_rope(c["kp"], c["vp"], c["table"], c["lens"], q, k, v, c["q_offsets"],
                              steps, q_out=out, dev_status=status)
        return int(status), out, c["pool"], before

    good = run(lambda c: None)
    assert good[0] == 0
    for offsets in ([0, 4, 3], [-1, 3, 6], [0, 3, 7]):
        status, out, pool, before = run(lambda c: c["q_offsets"].copy_(_ints(offsets)))
        assert status == w4.W4_DEV_BAD_SLOT and torch.equal(pool, before)
        assert bool((out == 5).all())
    for page in (-1, 10 ** 6):
        status, out, pool, before = run(lambda c: c["table"][0].fill_(page))
        assert status == w4.W4_DEV_BAD_PAGE and torch.equal(out, good[1])
        assert not torch.equal(pool, before)               # the other sequence's
    # more new tokens than the length, or beyond the table
    for n in (2, -5, 10 ** 6):
        status, out, pool, before = run(lambda c: c["lens"][:1].fill_(n))
        assert status == w4.W4_DEV_BAD_PAGE
        assert torch.equal(out[3:], good[1][3:])


@gpu
def test_captured_and_on_another_stream(lib):
    import torch
    q, k, v, (wq, wk) = _inputs(40, 8, 2, 128, "bfloat16", 9)
    c = _sequences([25, 15], [0, 100], 16, 2, 128, "bfloat16", 9)
    steps, out = lib.w4_rope_steps(128), torch.empty_like(q)

    def call(**kw):
        return lib.w4_kv_append_rope(c["kp"], c["vp"], c["table"], c["lens"], q, k, v,
                                     c["q_offsets"], steps, q_weight=wq, k_weight=wk, **kw)
    c["pool"].zero_()
    want, pool = call().clone(), c["pool"].clone()
    c["pool"].zero_()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(c["pool"], pool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q_out=out)
    for _ in range(2):
        out.zero_()
        c["pool"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(c["pool"], pool)


@gpu
def test_results_that_overlap_are_refused(lib):
    import torch
    q, k, _, _ = _inputs(4, 2, 2, 64, "bfloat16", 3)
    pos, steps = torch.zeros(4, dtype=torch.int32, device="cuda"), lib.w4_rope_steps(64)
    flat = torch.zeros(4 * 2 * 64, dtype=torch.bfloat16, device="cuda")
    for strides in ((0, 64, 1), (128, 0, 1), (128, 56, 1), (56, 256, 1)):
        bad = flat.as_strided((4, 2, 64), strides)
        with pytest.raises(ValueError, match="overlap"):
            lib.w4_qk_norm_rope(q, k, pos, steps, q_out=bad)
        with pytest.raises(ValueError, match="overlap"):
            lib.w4_qk_norm_rope(q, k, pos, steps, k_out=bad)


# ------------------------------------------------------------------- without a GPU
def _steps(rot, *a, **kw):
    return [s % 2 ** 64 for s in w4.w4_rope_steps(rot, *a, device="cpu", **kw).tolist()]


def _check_steps(got, freq):
    for s, f in zip(got, freq):
        want = (f / (2 * math.pi)) % 1.0
        # the power's and the quotient's relative error, a few halves of 2^-53
        assert abs(s / 2.0 ** 64 - want) <= 2.0 ** -50 * f + 2.0 ** -64
    assert len(got) == len(freq)


def test_steps():
    _check_steps(_steps(128), [10000.0 ** (-i / 64) for i in range(64)])
    _check_steps(_steps(2, 1e6), [1.0])
    assert _steps(0) == []
    assert _steps(64, factor=1.0, method="base") == _steps(64)
    assert _steps(64, 500.0, method="parts", trained_len=100, low=1, high=4) == _steps(64, 500.0)
    # a base below one: frequencies of more than a turn a position, of which the part counts
    _check_steps(_steps(16, 1e-4), [1e-4 ** (-i / 8) for i in range(8)])


def test_steps_for_longer_contexts():
    f = [10000.0 ** (-i / 32) for i in range(32)]
    _check_steps(_steps(64, method="linear", factor=4.0), [x / 4 for x in f])
    b = 10000.0 * 8.0 ** (64 / 62)
    base = _steps(64, method="base", factor=8.0)
    _check_steps(base, [b ** (-i / 32) for i in range(32)])
    _check_steps(base[-1:], [f[-1] / 8])
    want = []
    for x in f:
        turns = 8192 * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        want.append(x * keep + x / 16 * (1 - keep))
    got = _steps(64, method="parts", factor=16.0, trained_len=8192, low=1, high=32)
    _check_steps(got, want)
    assert want[0] == f[0] and want[-1] == f[-1] / 16 and got[0] == _steps(64)[0]


@pytest.mark.parametrize("a,kw", [
    ((3,), {}), ((64, 0.0), {}), ((64, -1.0), {}), ((64, math.nan), {}), ((64, math.inf), {}),
    ((64,), dict(factor=0.0)), ((64,), dict(factor=math.nan)), ((2,), dict(method="base", factor=2.0)),
    ((64,), dict(method="parts", factor=2.0)),
    ((64,), dict(method="parts", factor=2.0, trained_len=100, low=3, high=3)),
    ((64,), dict(method="parts", factor=2.0, trained_len=100, low=math.nan, high=3)),
])
def test_steps_refused(a, kw):
    with pytest.raises(w4.W4Error) as e:
        w4.w4_rope_steps(*a, device="cpu", **kw)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        w4.w4_rope_steps(64, method="other", device="cpu")


def test_calls_refused():
    """Shapes, alignment and missing pointers, answered by the library without a launch."""
    import ctypes
    lib = w4.load_library()
    at = 0x10000

    def rope(q=at, k=at, pos=at, steps=at, wq=None, T=2, Hq=4, Hkv=2, D=64, rot=64, dtype=0, eps=1e-6,
             amp=1.0, q_out=at, k_out=at, qs=256, kos=128):
        return lib.w4_qk_norm_rope(q, qs, 64, k, 128, 64, pos, steps, wq, None, T, Hq, Hkv, D, rot, 0,
                                   dtype, eps, amp, q_out, 256, 64, k_out, kos, 64, None)
    for kw, want in [(dict(q=None), 1), (dict(k=None), 1), (dict(pos=None), 1), (dict(steps=None), 1),
                     (dict(q_out=None), 1), (dict(k_out=None), 1), (dict(T=-1), 1), (dict(Hq=-1), 1),
                     (dict(D=0), 1), (dict(dtype=2), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
                     (dict(amp=math.inf), 1), (dict(D=60), 2), (dict(D=264, rot=64), 2),
                     (dict(rot=8), 2), (dict(rot=80), 2), (dict(Hq=70000), 2), (dict(q=at + 2), 3),
                     (dict(wq=at + 4), 3), (dict(steps=at + 4), 3), (dict(pos=at + 2), 3),
                     (dict(qs=260), 3), (dict(kos=132), 3), (dict(k_out=at + 8), 3)]:
        assert rope(**kw) == want, kw
    assert rope(T=0) == 0 and rope(Hq=0, Hkv=0) == 0

    def append(table=at, lens=at, offs=at, kp=at, vp=at, v=at, page=16, T=2, B=1, W=4, P=8, ps=2048,
               rot=64, Hkv=2):
        return lib.w4_kv_append_rope(kp, vp, ps, 128, 64, P, page, table, B, W, lens, at, 256, 64, at,
                                     128, 64, v, 128, 64, offs, None, at, None, None, T, 4, Hkv, 64,
                                     rot, 0, 0, ctypes.c_float(1e-6), ctypes.c_float(1.0), at, 256,
                                     64, None, None)
    for kw, want in [(dict(table=None), 1), (dict(lens=None), 1), (dict(offs=None), 1),
                     (dict(kp=None), 1), (dict(vp=None), 1), (dict(v=None), 1), (dict(page=0), 1),
                     (dict(B=0), 1), (dict(P=0), 1), (dict(Hkv=0), 1), (dict(rot=24), 2),
                     (dict(W=1 << 30), 2), (dict(ps=2044), 3), (dict(kp=at + 8), 3),
                     (dict(v=at + 2), 3), (dict(offs=at + 1), 3)]:
        assert append(**kw) == want, kw
    assert append(T=0) == 0


def test_binding_refuses_before_anything_is_launched():
    import torch
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    pos, steps = torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError):
        w4.w4_qk_norm_rope(x, x, pos, steps)               # not on the GPU
    with pytest.raises(ValueError):
        w4.w4_qk_norm_rope(x.float(), x.float(), pos, steps)
