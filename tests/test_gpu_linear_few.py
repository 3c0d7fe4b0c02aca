"""w4_w4a16_linear_few against a plain float64 evaluation.

Tolerance, derived beforehand.  Codes and activations are exact, products too; sums are
fp32.  With S = sum_k |s| (q + z) |x| over an output's terms (the codes' and the zeros'
parts are summed apart): a group's sum of 128 products in the tensor cores and of its
activations, each off by at most 2^-17 of its absolute sum (128 steps of 2^-24), some 110
groups and the warps' shares another 2^-17; together below 2^-15 S.  y's rounding is
2^-8 |y|."""
import ctypes

import pytest

import w4a16_moe_expert_sync_gb300 as w4

gpu = pytest.mark.gpu


def _inputs(M, K, N, group, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sh = (N, K // group)
    s = (torch.exp(torch.randn(sh, generator=g, device="cuda")) * 0.01).half()
    z = (torch.rand(sh, generator=g, device="cuda") * 15).half()
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    return x, q, s, z


def _reference(x, q, s, z, group):
    """(y, S) in float64."""
    import torch
    c = torch.stack((q & 15, q >> 4), -1).flatten(1).double()
    sc, ze = (t.double().repeat_interleave(group, 1) for t in (s, z))
    return x.double() @ ((c - ze) * sc).T, x.double().abs() @ ((c + ze.abs()) * sc.abs()).T


def _check(got, x, q, s, z, group):
    ref, S = _reference(x, q, s, z, group)
    tol = 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + 2.0 ** -15 * S
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:5].tolist())


@gpu
@pytest.mark.parametrize("M,K,N,group", [
    (1, 128, 1, 128), (1, 64, 1, 64), (1, 2816, 4096, 128), (2, 192, 17, 64), (3, 704, 2815, 64),
    (7, 256, 33, 128), (8, 640, 5000, 128), (9, 1408, 999, 128), (11, 64, 63, 64), (15, 960, 257, 64),
    (16, 2816, 2816, 128), (17, 384, 31, 128), (24, 448, 4864, 64), (25, 2816, 10000, 128),
    (32, 2816, 4111, 128), (32, 64, 20000, 64),
    # activations that do not fit at once: two tiles, one tile of tokens a pass
    (32, 4096, 515, 128), (31, 8192, 130, 64), (19, 6464, 77, 64), (32, 11264, 40, 128),
    (9, 11264, 2500, 64), (1, 11264, 1, 128)])
def test_linear(lib, M, K, N, group):
    x, q, s, z = _inputs(M, K, N, group, M + K)
    y = lib.w4_w4a16_linear_few(x, q, s, z, group)
    _check(y, x, q, s, z, group)
    import torch
    assert torch.equal(lib.w4_w4a16_linear_few(x, q, s, z, group), y)


@gpu
@pytest.mark.parametrize("M,K,N", [
    (9, 512, 40000), (16, 640, 38913), (13, 2816, 39040), (17, 512, 60001), (32, 1408, 38912),
    (25, 2816, 50000), (32, 3200, 39999), (10, 5632, 38912), (31, 5632, 40011), (32, 7168, 38912),
    (9, 2816, 19456), (32, 5632, 19457), (17, 2048, 29185), (32, 2816, 39041), (20, 2944, 41000), (31, 2560, 60007), (12, 5248, 39000), (32, 11264, 38912)])
def test_many_rows(lib, M, K, N):
    """From 19456 or 38912 rows on (on 152 SMs) more than 8 tokens go through the tensor memory, in
    parts of 32 or 16 as they fit, where they do."""
    import torch
    x, q, s, z = _inputs(M, K, N, 128, M + K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = lib.w4_w4a16_linear_few(x, q, s, z, dev_status=status)
    _check(y, x, q, s, z, 128)
    assert torch.equal(lib.w4_w4a16_linear_few(x, q, s, z), y) and int(status) == 0


@gpu
@pytest.mark.parametrize("M,K,N", [
    (9, 512, 77900), (16, 2816, 38912), (32, 2816, 39040), (13, 5632, 19456), (25, 5120, 20001),
    (32, 640, 80007), (11, 704, 80000), (17, 8192, 19456)])
def test_many_rows_groups_of_64(lib, M, K, N):
    """Two groups a step of the tensor memory, where K is whole steps and the activations
    fit; groups of zeros, large values, small ones and zeros of the weights among them."""
    import torch
    x, q, s, z = _inputs(M, K, N, 64, M + K)
    x[1, 64:128], x[2, 5], x[3, 192:256] = 0.0, 3000.0, x[3, 192:256] * 2.0 ** -12
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = lib.w4_w4a16_linear_few(x, q, s, z, 64, dev_status=status)
    _check(y, x, q, s, z, 64)
    for _ in range(20):
        assert torch.equal(lib.w4_w4a16_linear_few(x, q, s, z, 64), y)
    assert int(status) == 0
    # a token by itself among as many, and scaled by a power of two
    one = torch.zeros_like(x)
    one[4] = x[4] * 0.25
    assert torch.equal(lib.w4_w4a16_linear_few(one, q, s, z, 64)[4], y[4] * 0.25)


@gpu
@pytest.mark.parametrize("M", [12, 30])
def test_many_rows_and_odd_activations(lib, M):
    """Groups of zeros, one large value among small ones, subnormals, what is not finite,
    scaling by powers of two, the order of the tokens."""
    import math
    import torch
    x, q, s, z = _inputs(M, 1024, 39000, 128, 3)
    x[1, 128:256], x[2] = 0.0, 0.0
    x[3, 5] = 30000.0
    x[4, 300:400] *= 2.0 ** -12
    x[5] = x[5] * 2.0 ** -120
    x[6, 512:640] = 2.0 ** -133
    want = lib.w4_w4a16_linear_few(x, q, s, z)
    # what activations lose is below 2^-22 of their group's largest, times 15 + 15 scales
    ref, S = _reference(x, q, s, z, 128)
    top = x.double().abs().view(M, 8, 128).amax(-1)
    loss = 2.0 ** -22 * 128 * 15 * top @ s.double().abs().T
    tol = 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + 2.0 ** -15 * S + loss + 2.0 ** -133
    bad = ~((want.double() - ref).abs() <= tol)
    assert not bool(bad.any()), (bad.sum(1).tolist(), ((want.double() - ref).abs() / tol).amax(1))
    assert bool((want[2] == 0).all())
    other = x.clone()
    other[7, 3], other[8, 1000], other[9] = math.nan, math.inf, 1e30
    got = lib.w4_w4a16_linear_few(other, q, s, z)
    same = [t for t in range(M) if t not in (7, 8, 9)]
    assert torch.equal(got[same], want[same])
    assert not bool(got[7].isfinite().any()) and not bool(got[8].isfinite().any())
    order = torch.randperm(M, device="cuda")
    assert torch.equal(lib.w4_w4a16_linear_few(x[order].contiguous(), q, s, z), want[order])
    plain = [t for t in range(M) if t not in (5, 6)]
    for e in (-40, -10, 40):
        y = lib.w4_w4a16_linear_few(x * 2.0 ** e, q, s, z)
        assert torch.equal(y[plain], want[plain] * 2.0 ** e)


@gpu
def test_many_calls_of_many_rows_are_alike(lib):
    """A slot that is filled again while its codes are still read shows in some calls only."""
    import torch
    for M, K in ((31, 5632), (32, 2816)):
        x, q, s, z = _inputs(M, K, 40011, 128, M)
        first = lib.w4_w4a16_linear_few(x, q, s, z)
        out = [lib.w4_w4a16_linear_few(x, q, s, z) for _ in range(150)]
        assert all(torch.equal(y, first) for y in out)


@gpu
def test_a_wait_that_gives_up(lib):
    """The first codes never land: the status says so, the context goes on."""
    import time
    import torch
    for M in (12, 32):
        x, q, s, z = _inputs(M, 1024, 39000, 128, 9)
        want = lib.w4_w4a16_linear_few(x, q, s, z)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        hooks = lib.load_library().w4_test_pipeline_hooks
        t = time.monotonic()
        try:
            assert hooks(2_000_000, 1) == 0
            lib.w4_w4a16_linear_few(x, q, s, z, dev_status=status)
            torch.cuda.synchronize()
        finally:
            hooks(0, 0)
        assert int(status) & w4.W4_DEV_PIPELINE_TIMEOUT and time.monotonic() - t < 30
        status.zero_()
        assert torch.equal(lib.w4_w4a16_linear_few(x, q, s, z, dev_status=status), want)
        assert int(status) == 0


@gpu
def test_every_row_count(lib):
    """Tasks and units that cross warps in every way."""
    for N in list(range(1, 70)) + [151 * 16, 152 * 16 + 1, 153 * 32 + 5, 304 * 16 + 15]:
        for M, K, group in ((1, 384, 128), (20, 320, 64)):
            x, q, s, z = _inputs(M, K, N, group, N)
            _check(lib.w4_w4a16_linear_few(x, q, s, z, group), x, q, s, z, group)


@gpu
def test_tokens_stand_for_themselves(lib):
    """A token's results do not depend on the others', whatever those are; what is not
    finite stays in its token; large and small activations keep their bits."""
    import math
    import torch
    x, q, s, z = _inputs(13, 1024, 200, 128, 5)
    want = lib.w4_w4a16_linear_few(x, q, s, z)
    other = x.clone()
    other[2], other[7], other[8, 3], other[9, 1000] = 0.0, 1e30, math.nan, math.inf
    got = lib.w4_w4a16_linear_few(other, q, s, z)
    same = [t for t in range(13) if t not in (2, 7, 8, 9)]
    assert torch.equal(got[same], want[same])
    assert bool((got[2] == 0).all()) and not bool(got[8].isfinite().any())
    assert not bool(got[9].isfinite().any())
    order = torch.randperm(13, device="cuda")
    assert torch.equal(lib.w4_w4a16_linear_few(x[order].contiguous(), q, s, z), want[order])
    for e in (-40, -10, 40):                   # powers of two change nothing but the exponent
        y = lib.w4_w4a16_linear_few(x * 2.0 ** e, q, s, z)
        assert torch.equal(y, want * 2.0 ** e)


@gpu
def test_extreme_weights(lib):
    """Every code, scales and zeros at the ends of fp16, constant groups."""
    import torch
    x, q, s, z = _inputs(5, 512, 64, 128, 6)
    s[0], s[1], s[2] = 65504.0, 2.0 ** -24, 0.0
    z[3], z[4], z[5] = 0.0, -65504.0, 65504.0
    q[6], q[7] = 0, 255
    s[8] = -0.5
    y = lib.w4_w4a16_linear_few(x, q, s, z)
    ref, S = _reference(x, q, s, z, 128)
    tol = 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + 2.0 ** -15 * S
    assert bool(((y.double() - ref).abs() <= tol).all())
    assert bool((y[:, 2] == 0).all())


@gpu
def test_against_the_dense_linear(lib):
    """The same weights through w4_quantize and the path for more rows."""
    import torch
    W = torch.randn((1, 512, 1024), device="cuda") * 0.02
    q, s, z = (t[0] for t in lib.w4_quantize(W, 128))
    x = torch.randn((32, 1024), device="cuda").bfloat16()
    few, many = lib.w4_w4a16_linear_few(x, q, s, z), lib.w4_w4a16_linear(x, q, s, z)
    # the dense path rounds weights to fp16, either result once
    ref, S = _reference(x, q, s, z, 128)
    assert bool(((few.double() - many.double()).abs() <=
                 2.0 ** -7 * ref.abs() * 1.01 + 2.0 ** -10 * S).all())


@gpu
def test_stream_graph_and_given_result(lib):
    import torch
    x, q, s, z = _inputs(6, 2816, 3000, 128, 7)
    want = lib.w4_w4a16_linear_few(x, q, s, z)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = lib.w4_w4a16_linear_few(x, q, s, z, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    wide = torch.full((8, 3000), 3.0, device="cuda").bfloat16()
    out = wide[1:7]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.w4_w4a16_linear_few(x, q, s, z, out=out)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want * 2)
    assert bool((wide[0] == 3).all()) and bool((wide[7] == 3).all())


def test_calls_refused():
    lib = w4.load_library()
    at = 0x10000

    def linear(x=at, M=1, K=256, N=64, q=at, s=at, z=at, group=128, y=at):
        return lib.w4_w4a16_linear_few(x, M, K, N, q, s, z, group, y, None, None)
    for kw, want in [(dict(x=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(z=None), 1),
                     (dict(y=None), 1), (dict(M=-1), 1), (dict(K=0), 1), (dict(N=-1), 1),
                     (dict(M=33), 2), (dict(K=192), 2), (dict(K=11392), 2), (dict(group=32), 2),
                     (dict(group=256), 2), (dict(N=1 << 30, K=128), 2), (dict(N=1 << 26, K=1 << 13), 2),
                     (dict(x=at + 8), 3), (dict(q=at + 4), 3), (dict(s=at + 1), 3), (dict(y=at + 2), 3)]:
        assert linear(**kw) == want, kw
    assert linear(M=0) == 0 and linear(N=0) == 0
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_binding_refuses_before_anything_is_launched():
    import torch
    x, q = torch.zeros((1, 128), dtype=torch.bfloat16), torch.zeros((4, 64), dtype=torch.uint8)
    s = torch.zeros((4, 1), dtype=torch.float16)
    with pytest.raises(ValueError):
        w4.w4_w4a16_linear_few(x, q, s, s)                 # not on the GPU
    with pytest.raises(ValueError):
        w4.w4_w4a16_linear_few(x[0], q, s, s)
