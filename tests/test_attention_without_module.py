"""w4_attn_shared_prefix where the module of the calls in C++ has not been built for the
installed torch: the same checks and, on a GPU, the same bits; the calls that are the
module's alone say what is missing."""
import pytest
import torch

import w4a16_moe_expert_sync_gb300 as w4
from w4a16_moe_expert_sync_gb300 import _lib


@pytest.fixture
def no_module(monkeypatch, tmp_path):
    monkeypatch.setattr(_lib, "_calls_module", None)
    monkeypatch.setattr(_lib, "_calls_file", None, raising=False)
    monkeypatch.setattr(_lib, "calls_path", lambda: str(tmp_path / "none.so"))


def _on_cpu():
    pages, ints = torch.zeros((5, 16, 2, 64), dtype=torch.bfloat16), dict(dtype=torch.int32)
    return [torch.zeros((3, 4, 64), dtype=torch.bfloat16), pages, pages,
            torch.zeros((1, 4), **ints), torch.tensor([3], **ints), torch.tensor([0, 3], **ints)]


def test_arguments_are_checked(no_module):
    args = _on_cpu()
    with pytest.raises(ValueError, match="live on the GPU"):
        w4.w4_attn_shared_prefix(*args)


def test_the_others_say_what_is_missing(no_module):
    args = _on_cpu()
    for call in (lambda: w4.w4_attn_tree(*args, torch.ones((3, 1), dtype=torch.int32)),
                 lambda: w4.w4_w4a16_linear_few(args[0], args[0], args[0], args[0])):
        with pytest.raises(RuntimeError, match="build the CUDA library"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,causal", [("bfloat16", True), ("float16", False)])
def test_the_same_bits(lib, monkeypatch, tmp_path, dtype, causal):
    from test_gpu_attention import _build
    c = _build([126, 43, 60], [6, 3, 1], [2], [32], 8, 2, 64, 16, dtype, seed=2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [c["q"], c["cache"][0], c["cache"][1], c["table"], c["lens"], c["q_offsets"],
            c["group_offsets"], c["shared"]]

    def both(**kw):
        with_module = lib.w4_attn_shared_prefix(*args, max_q=6, causal=causal, **kw).clone()
        with monkeypatch.context() as m:
            m.setattr(_lib, "_calls_module", None)
            m.setattr(_lib, "_calls_file", str(tmp_path / "none.so"))
            return with_module, lib.w4_attn_shared_prefix(*args, max_q=6, causal=causal, **kw)
    out = torch.empty_like(c["q"])
    ws = torch.empty(lib.w4_attn_shared_prefix_workspace_size(10, 3, 1, 6, 8, 2, 64),
                     dtype=torch.uint8, device="cuda")
    want = None
    for kw in (dict(), dict(scale=64 ** -0.5), dict(out=out, workspace=ws, dev_status=status),
               dict(stream=torch.cuda.Stream())):
        torch.cuda.synchronize()
        a, b = both(**kw)
        torch.cuda.synchronize()
        want = a if want is None else want
        assert torch.equal(a, want) and torch.equal(b, want) and int(status) == 0
    with monkeypatch.context() as m:
        m.setattr(_lib, "_calls_module", None)
        m.setattr(_lib, "_calls_file", str(tmp_path / "none.so"))
        m.setattr(torch.cuda, "current_device", lambda: 1)
        with pytest.raises(ValueError, match="current device"):
            lib.w4_attn_shared_prefix(*args, max_q=6)
        m.undo()
    assert torch.equal(lib.w4_attn_shared_prefix(*args, max_q=6, causal=causal), want)
