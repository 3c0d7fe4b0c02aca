"""The few-token layer (w4_moe_layer_few) against a plain float64 evaluation.

Tolerance, derived beforehand.  Per output element, with S = sum_j w_j
sum_i |h_i| |Wd|: the bf16 rounding of the result (2^-8 |ref|), the fp16
rounding of every h_i (2^-11 of it: 2^-11 S at most), and fp32 sums, whose
error (2^-22 of the absolute sums of the two contractions, which are about
sqrt(K) times the sums themselves, K <= 2816) stays below 2^-14 S."""
import ctypes

import pytest

import w4a16_moe_expert_sync_gb300 as w4


def _weights(E, N, K, group, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand((E, N, K // group), generator=g, device="cuda") * 0.01 + 0.002).half()
    z = (torch.rand((E, N, K // group), generator=g, device="cuda") * 4 + 5).half()
    return q, s, z


def _deq(w, e, group):
    import torch
    q = w[0][e]
    c = torch.stack((q & 15, q >> 4), -1).flatten(1).double().view(q.shape[0], -1, group)
    return ((c - w[2][e].double()[..., None]) * w[1][e].double()[..., None]).flatten(1)


def _reference(x, ids, wts, gu, dn):
    """(out, S) in float64; ids outside the experts contribute nothing."""
    import torch
    M, d = x.shape
    m = gu[0].shape[1] // 2
    out = torch.zeros((M, d), dtype=torch.float64, device="cuda")
    S = torch.zeros_like(out)
    for t in range(M):
        for j, e in enumerate(ids[t].tolist()):
            if not 0 <= e < gu[0].shape[0]:
                continue
            g = _deq(gu, e, 128) @ x[t].double()
            h = torch.nn.functional.gelu(g[:m], approximate="tanh") * g[m:]
            W = _deq(dn, e, 64)
            out[t] += wts[t, j].double() * (W @ h)
            S[t] += wts[t, j].double().abs() * (W.abs() @ h.abs())
    return out, S


def _check(got, ref, S):
    assert bool(((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs()
                 + (2.0 ** -11 + 2.0 ** -14) * (1 + 2.0 ** -8) * S).all())


def _inputs(M, d, m, E, k, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + 77)
    x = torch.randn((M, d), generator=g, device="cuda").bfloat16()
    logits = torch.randn((M, E), generator=g, device="cuda")
    return x, logits, _weights(E, 2 * m, d, 128, seed), _weights(E, d, m, 64, seed + 1)


SHAPES = [(1, 128, 64, 1, 1), (1, 256, 128, 8, 2), (5, 384, 192, 12, 3), (9, 128, 64, 3, 3),
          (16, 1152, 320, 40, 4), (17, 256, 128, 4, 1), (32, 384, 192, 12, 8),
          (8, 256, 64, 200, 32), (3, 6144, 64, 4, 2), (2, 128, 2560, 4, 2), (1, 2816, 704, 16, 8),
          (32, 2816, 704, 16, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,d,m,E,k", SHAPES)
def test_layer_matches_float64(lib, M, d, m, E, k):
    import torch
    x, logits, gu, dn = _inputs(M, d, m, E, k)
    ids, wts = lib.w4_moe_route(logits, k)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.w4_moe_layer_few(x, ids, wts, gu, dn, dev_status=st)
    assert int(st) == 0
    _check(got, *_reference(x, ids, wts, gu, dn))
    # from the logits: the same bits, and the same again
    out, ids2, w2 = lib.w4_moe_layer_few_from_logits(x, logits, k, gu, dn, dev_status=st)
    assert int(st) == 0
    assert torch.equal(ids, ids2) and torch.equal(wts, w2) and torch.equal(out, got)
    assert torch.equal(lib.w4_moe_layer_few(x, ids, wts, gu, dn), got)


@pytest.mark.gpu
def test_close_to_the_four_launch_layer(lib):
    x, logits, gu, dn = _inputs(16, 256, 128, 8, 2, seed=5)
    ids, wts = lib.w4_moe_route(logits, 2)
    a = lib.w4_moe_layer_few(x, ids, wts, gu, dn).double()
    b = lib.w4_moe_layer(x, ids, wts, gu, dn).double()
    # both are within 2e-2 of the rms of the same result
    assert float((a - b).abs().max()) <= 4e-2 * float(b.pow(2).mean().sqrt())


@pytest.mark.gpu
def test_skewed_repeated_and_invalid_ids(lib):
    import torch
    M, d, m, E, k = 24, 256, 128, 6, 4
    x, _, gu, dn = _inputs(M, d, m, E, k, seed=9)
    ids = torch.full((M, k), 3, dtype=torch.int32, device="cuda")     # 96 assignments of one
    ids[4] = torch.tensor([0, 0, 5, 5])                               # repeated experts
    ids[5] = torch.tensor([-1, E, 1, 2 ** 30])                        # three invalid
    ids[6] = -7                                                       # none valid
    wts = torch.rand((M, k), device="cuda")
    wts[7] = 0.0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.w4_moe_layer_few(x, ids, wts, gu, dn, dev_status=st)
    assert int(st) == lib.W4_DEV_BAD_EXPERT_ID
    _check(got, *_reference(x, ids, wts, gu, dn))
    assert bool((got[6] == 0).all()) and bool((got[7] == 0).all())


@pytest.mark.gpu
def test_activation_range_is_flagged(lib):
    import torch
    x, logits, gu, dn = _inputs(3, 256, 128, 8, 2, seed=2)
    ids, wts = lib.w4_moe_route(logits, 2)
    clean = lib.w4_moe_layer_few(x, ids, wts, gu, dn)
    y = x.clone()
    y[1, 7] = 1e30
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.w4_moe_layer_few(y, ids, wts, gu, dn, dev_status=st)
    assert int(st) == lib.W4_DEV_FP16_RANGE
    assert torch.equal(got[[0, 2]], clean[[0, 2]])


@pytest.mark.gpu
def test_other_stream_graph_and_dirty_workspace(lib):
    import torch
    x, logits, gu, dn = _inputs(6, 384, 192, 12, 3, seed=4)
    want, _, _ = lib.w4_moe_layer_few_from_logits(x, logits, 3, gu, dn)
    ws = torch.full((lib.w4_moe_layer_few_workspace_size(6, 384, 192, 12, 3),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    out = torch.full_like(x, float("nan"))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lib.w4_moe_layer_few_from_logits(x, logits, 3, gu, dn, workspace=ws, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _, _ = lib.w4_moe_layer_few_from_logits(x, logits, 3, gu, dn, workspace=ws)
    for _ in range(3):
        got.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.gpu
def test_empty_batch(lib):
    import torch
    _, _, gu, dn = _inputs(1, 256, 128, 8, 2)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    out, ids, w = lib.w4_moe_layer_few_from_logits(
        x, torch.empty((0, 8), device="cuda"), 2, gu, dn)
    assert out.shape == (0, 256) and ids.shape == (0, 2) and w.shape == (0, 2)


def test_refusals_without_launching():
    from w4a16_moe_expert_sync_gb300 import build as w4build
    w4build.build()
    lib = w4.load_library()
    P = ctypes.c_void_p
    fake, odd, big = P(0x10000), P(0x10004), 1 << 30

    def call(x=fake, M=4, d=256, m=128, E=8, k=2, gg=128, dg=64, ws=fake, nb=big, out=fake,
             q=fake, ids=fake):
        return lib.w4_moe_layer_few(x, ids, fake, M, d, m, E, k, q, fake, fake, gg, fake, fake,
                                    fake, dg, ws, nb, out, None, None)
    assert call(x=None) == 1 and call(ids=None) == 1 and call(q=None) == 1 and call(M=-1) == 1
    assert call(M=33) == 2 and call(M=32, k=9, E=16) == 2 and call(k=33, M=1, E=64) == 2
    assert call(d=200) == 2 and call(m=96) == 2 and call(gg=64) == 2 and call(dg=128) == 2
    assert call(E=1025) == 2 and call(d=9216) == 2 and call(m=9216) == 2
    assert call(x=odd) == 3 and call(out=odd) == 3 and call(q=P(0x10008)) == 3
    assert call(ids=P(0x10002)) == 3 and call(ws=P(0x10080)) == 3
    assert call(ws=None) == 6 and call(nb=4 * 2 * (128 * 2 + 256 * 4) - 1) == 6
    assert call(x=None, M=0, ws=None, nb=0, out=None, ids=None) == 0
    args = [fake, fake, 4, 256, 128, 8, 2, fake, fake, fake, 128, fake, fake, fake, 64, fake, big,
            fake, fake, fake, None, None]
    bad = list(args)
    bad[1] = None
    assert lib.w4_moe_layer_few_from_logits(*bad) == 1
    bad = list(args)
    bad[6], bad[5] = 9, 8
    assert lib.w4_moe_layer_few_from_logits(*bad) == 2


def test_binding_refuses_mismatched_shapes():
    import torch
    x = torch.zeros((2, 256))
    with pytest.raises(ValueError):
        w4.w4_moe_layer_few(x, x, x, (x, x, x), (x, x, x))


@pytest.mark.gpu
def test_binding_refuses_other_types_and_shapes(lib):
    import torch
    E, d, m, k = 4, 256, 128, 2
    dev = dict(device="cuda")
    gu = (torch.zeros((E, 2 * m, d // 2), dtype=torch.uint8, **dev),
          torch.zeros((E, 2 * m, d // 128), dtype=torch.float16, **dev),
          torch.zeros((E, 2 * m, d // 128), dtype=torch.float16, **dev))
    dn = (torch.zeros((E, d, m // 2), dtype=torch.uint8, **dev),
          torch.zeros((E, d, m // 64), dtype=torch.float16, **dev),
          torch.zeros((E, d, m // 64), dtype=torch.float16, **dev))
    x = torch.zeros((3, d), dtype=torch.bfloat16, **dev)
    ids = torch.zeros((3, k), dtype=torch.int32, **dev)
    w = torch.zeros((3, k), **dev)
    logits = torch.zeros((3, E), **dev)

    def few(**kw):
        a = dict(x=x, topk_ids=ids, topk_weights=w, gu=gu, dn=dn)
        a.update(kw)
        return w4.w4_moe_layer_few(**a)

    def routed(**kw):
        a = dict(x=x, logits=logits, k=k, gu=gu, dn=dn)
        a.update(kw)
        return w4.w4_moe_layer_few_from_logits(**a)
    assert few().shape == x.shape and routed()[1].shape == ids.shape
    for bad in (dict(x=x.half()), dict(x=x[:, :128]), dict(topk_ids=ids.long()),
                dict(topk_ids=ids[:2]), dict(topk_weights=w.half()), dict(topk_weights=w[:, :1]),
                dict(gu=(gu[0], gu[1].float(), gu[2])), dict(gu=(gu[0], gu[1], gu[2][:, :, :1])),
                dict(gu=(gu[0][:, :, ::2], gu[1], gu[2])), dict(gu=(gu[0][:3], gu[1], gu[2])),
                dict(dn=(dn[0], dn[1][:2], dn[2])), dict(dn=(dn[0].short(), dn[1], dn[2])),
                dict(out=x[:2]), dict(out=x.float()), dict(gu_group=64), dict(x=x.cpu())):
        with pytest.raises(ValueError):
            few(**bad)
    for bad in (dict(logits=logits.double()), dict(logits=logits[:, :3]), dict(ids=ids.long()),
                dict(weights=w[:1]), dict(x=x.float())):
        with pytest.raises(ValueError):
            routed(**bad)
