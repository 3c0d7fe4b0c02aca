"""w4_attn_shared_prefix on tensors of a GPU that is not the current one: refused on the
host, where the kernels would read the other's pointers."""
import pytest

pytestmark = pytest.mark.gpu


def test_another_current_device_is_refused(lib):
    import torch
    from test_gpu_attention import _build
    from w4a16_moe_expert_sync_gb300 import _lib
    c = _build([126, 43, 60], [6, 3, 1], [2], [32], 8, 2, 64, 16, "bfloat16", seed=1)
    kw = dict(group_offsets=c["group_offsets"], shared_lens=c["shared"], max_q=6)

    def call(**more):
        return lib.w4_attn_shared_prefix(c["q"], c["cache"][0], c["cache"][1], c["table"], c["lens"],
                                         c["q_offsets"], **dict(kw, **more))
    want = call()
    given = [dict(), dict(out=torch.empty_like(want)), dict(group_offsets=None, shared_lens=None),
             dict(dev_status=torch.zeros(1, dtype=torch.int32, device="cuda"))]
    _lib._calls().pretend_device(1)
    try:
        for more in given:
            with pytest.raises(ValueError, match="current device"):
                call(**more)
    finally:
        _lib._calls().pretend_device(-1)
    for more in given[:2]:
        assert torch.equal(call(**more), want)
