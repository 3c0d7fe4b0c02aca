"""The few-token layer with activations far from 1: rows whose h, and groups whose x,
lie below what fp16 holds unscaled.  The bound is that of test_gpu_few.py: the bf16
rounding of the result, 2^-11 of every h_i (which holds at any magnitude once each
group of h is scaled by a power of two before it is rounded) and the fp32 sums; x is
bf16 and exact."""
import pytest

pytestmark = pytest.mark.gpu


def _routed(lib, M, E, k, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lib.w4_moe_route(torch.randn((M, E), generator=g, device="cuda"), k)


@pytest.mark.parametrize("M,d,m,E,k", [(5, 384, 192, 12, 3), (3, 2816, 704, 16, 8), (3, 6144, 64, 4, 2),
                                       (16, 1152, 320, 40, 4)])
@pytest.mark.parametrize("scale", [1e-2, 1e-3, 1e-4, 1e-5, 1e-8, 1e-12])
def test_small_rows(lib, M, d, m, E, k, scale):
    import torch
    from test_gpu_few import _check, _inputs, _reference
    x, _, gu, dn = _inputs(M, d, m, E, k, seed=3)
    ids, w = _routed(lib, M, E, k, 5)
    x = x.clone()
    x[1:] = (x[1:].float() * scale).bfloat16()          # the first row stays as it is
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.w4_moe_layer_few(x, ids, w, gu, dn, dev_status=st)
    assert int(st) == 0
    _check(got, *_reference(x, ids, w, gu, dn))


def test_rows_of_mixed_groups(lib):
    """Groups of a row from 1e-9 to 1, zeros among them; the large ones' weights are
    zero for the first half of the intermediates, and the second half's for the result,
    so that only the small ones speak."""
    import torch
    from test_gpu_few import _check, _inputs, _reference
    M, d, m, E, k = 4, 1152, 384, 8, 2
    x, _, gu, dn = _inputs(M, d, m, E, k, seed=8)
    ids, w = _routed(lib, M, E, k, 6)
    s = torch.tensor([1, 1e-9, 1, 0, 1e-6, 1, 1e-7, 3e-6, 1e-8], device="cuda")
    x = (x.float().view(M, 9, 128) * s[None, :, None]).view(M, d).bfloat16()
    gs, ds = gu[1].clone(), dn[1].clone()
    for rows in (slice(0, m // 2), slice(m, m + m // 2)):
        gs[:, rows, 0] = gs[:, rows, 2] = gs[:, rows, 5] = 0
    ds[:, :, m // 128:] = 0
    gu, dn = (gu[0], gs, gu[2]), (dn[0], ds, dn[2])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.w4_moe_layer_few(x, ids, w, gu, dn, dev_status=st)
    assert int(st) == 0
    ref, S = _reference(x, ids, w, gu, dn)
    assert float(S.max()) < 1e-9
    _check(got, ref, S)
