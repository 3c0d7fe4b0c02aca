"""NaN among a token's logits: its ids stay in range, and the other tokens get the
router's ids and weights and their own rows, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(12, 3), (8, 8), (200, 32)])
@pytest.mark.parametrize("bits", [0x7FC00000, 0xFFC00000, 0xFFFFFFFF, 0x7F800001])
def test_nan_logits(lib, E, k, bits):
    import torch
    from test_gpu_few import _inputs
    M, d, m = 6, 256, 64
    x, logits, gu, dn = _inputs(M, d, m, E, k, seed=2)
    ids, w = lib.w4_moe_route(logits, k)
    want = lib.w4_moe_layer_few(x, ids, w, gu, dn)
    bad = logits.clone()
    nan = torch.tensor([bits], dtype=torch.int64).to(torch.int32).cuda() if bits < 1 << 31 else \
        torch.tensor([bits - (1 << 32)], dtype=torch.int32, device="cuda")
    raw = bad.view(torch.int32)
    raw[1, E // 2] = nan
    raw[4] = nan                              # every logit of a token
    assert bool(bad[1].isnan().any()) and bool(bad[4].isnan().all())
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, ids2, w2 = lib.w4_moe_layer_few_from_logits(x, bad, k, gu, dn, dev_status=st)
    assert bool((ids2 >= 0).all()) and bool((ids2 < E).all())
    rest = [0, 2, 3, 5]
    assert torch.equal(ids2[rest], ids[rest]) and torch.equal(w2[rest], w[rest])
    assert torch.equal(out[rest], want[rest])
    assert int(st) & ~lib.W4_DEV_FP16_RANGE == 0
