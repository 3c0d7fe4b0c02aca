"""The few-token layer's status word is int32, as attention's and the cache's."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "int64", "uint8", "int16"])
def test_a_status_of_another_type_is_refused(lib, dtype):
    import torch
    from test_gpu_few import _inputs
    x, logits, gu, dn = _inputs(3, 256, 128, 8, 2)
    ids, w = lib.w4_moe_route(logits, 2)
    st = torch.zeros(1, dtype=getattr(torch, dtype), device="cuda")
    with pytest.raises(ValueError):
        lib.w4_moe_layer_few(x, ids, w, gu, dn, dev_status=st)
    with pytest.raises(ValueError):
        lib.w4_moe_layer_few_from_logits(x, logits, 2, gu, dn, dev_status=st)
    with pytest.raises(ValueError):
        lib.w4_moe_layer_few(x, ids, w, gu, dn, dev_status=torch.zeros(1, dtype=torch.int32))
