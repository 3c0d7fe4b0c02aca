"""Arguments of a step's calls that no GPU is needed to refuse: their kinds, their places."""
import pytest
import torch

import w4a16_moe_expert_sync_gb300 as w4


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _i(*values):
    return torch.tensor(values, dtype=torch.int32)


def _calls():
    q, k, pages = _t(3, 4, 64), _t(3, 2, 64), _t(5, 16, 2, 64)
    table, lens, offsets = torch.zeros((1, 4), dtype=torch.int32), _i(3), _i(0, 3)
    steps = w4.w4_rope_steps(64, device="cpu")
    return {
        w4.w4_w4a16_linear_few: [_t(2, 128), _t(8, 64, dtype=torch.uint8),
                                 _t(8, 1, dtype=torch.float16), _t(8, 1, dtype=torch.float16)],
        w4.w4_qk_norm_rope: [q, k, _i(0, 1, 2), steps],
        w4.w4_kv_append_rope: [pages, pages, table, lens, q, k, k, offsets, steps],
        w4.w4_kv_keep: [_t(1, 2, 5, 16, 2, 64), table, lens, _i(1, 1, 1, 1, 1), offsets, _i(0),
                        _i(0, 1)],
        w4.w4_attn_shared_prefix: [q, pages, pages, table, lens, offsets],
        w4.w4_attn_tree: [q, pages, pages, table, lens, offsets, _i(1, 1, 1)[:, None]],
    }


@pytest.mark.parametrize("call", list(_calls()), ids=lambda f: f.__name__)
def test_tensors_are_asked_for(call):
    args = _calls()[call]
    with pytest.raises(ValueError, match="live on the GPU"):
        call(*args)
    for i in range(len(args)):
        for other in (3, "x", [1.0], object()):
            with pytest.raises(TypeError, match="expected a tensor"):
                call(*args[:i], other, *args[i + 1:])
        if not (call is w4.w4_qk_norm_rope and i == 2 or call is w4.w4_attn_tree and i == 6):
            with pytest.raises(TypeError, match="not None"):
                call(*args[:i], None, *args[i + 1:])
        else:
            with pytest.raises(ValueError):
                call(*args[:i], None, *args[i + 1:])


def test_numbers_are_asked_for():
    calls = _calls()
    q, k, positions, steps = calls[w4.w4_qk_norm_rope]
    linear, attn = calls[w4.w4_w4a16_linear_few], calls[w4.w4_attn_shared_prefix]
    with pytest.raises(TypeError):
        w4.w4_w4a16_linear_few(*linear, group="128")
    with pytest.raises(TypeError):
        w4.w4_w4a16_linear_few(*linear, group=64.0)
    for group in (1 << 40, -1 << 40, 0, -128):
        with pytest.raises(ValueError):
            w4.w4_w4a16_linear_few(*linear, group=group)
    with pytest.raises(OverflowError):
        w4.w4_w4a16_linear_few(*linear, group=1 << 80)
    with pytest.raises(TypeError):
        w4.w4_attn_shared_prefix(*attn, max_q=1.5)
    with pytest.raises(ValueError):
        w4.w4_attn_shared_prefix(*attn, max_q=1 << 40)


def test_shapes_come_before_places():
    """What does not fit is named, wherever it lies."""
    x, q, s, z = _calls()[w4.w4_w4a16_linear_few]
    for bad in ((x[0], q, s, z), (x, q[:, 0], s, z), (x, q, s[:7], z), (x, q, s, z.float()),
                (x.half(), q, s, z), (x, q.to(torch.int8), s, z), (x, q, s[..., None], z)):
        with pytest.raises(ValueError, match=r"\[M, K\]"):
            w4.w4_w4a16_linear_few(*bad)
    with pytest.raises(ValueError, match="contiguous"):
        w4.w4_w4a16_linear_few(_t(128, 2).t(), q, s, z)
    q, k, positions, steps = _calls()[w4.w4_qk_norm_rope]
    for bad in (dict(k=k.half()), dict(q=q.float(), k=k.float()), dict(k=k[:2]), dict(k=k[..., :32]),
                dict(q=q[0]), dict(q=q.transpose(1, 2)), dict(steps=steps.int()),
                dict(positions=positions.long()), dict(positions=positions[:2]),
                dict(q_weight=_t(32)), dict(k_weight=_t(64).half()), dict(q_weight=_t(128)[::2])):
        with pytest.raises(ValueError, match="must be"):
            w4.w4_qk_norm_rope(**dict(dict(q=q, k=k, positions=positions, steps=steps), **bad))
