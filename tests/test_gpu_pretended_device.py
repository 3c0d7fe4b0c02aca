"""The hook that lets a test stand in for the current device is its thread's own: calls of
other threads go on."""
import threading

import pytest

pytestmark = pytest.mark.gpu


def test_other_threads_do_not_see_it(lib):
    import torch
    from test_gpu_linear_few import _inputs
    from w4a16_moe_expert_sync_gb300 import _lib
    args = _inputs(2, 256, 64, 128)
    want = lib.w4_w4a16_linear_few(*args)
    torch.cuda.synchronize()
    set_, done, seen = threading.Event(), threading.Event(), []

    def pretend():
        _lib._calls().pretend_device(1)
        try:
            with pytest.raises(ValueError, match="current device"):
                lib.w4_w4a16_linear_few(*args)
            set_.set()
            done.wait(60)
        finally:
            _lib._calls().pretend_device(-1)
            set_.set()
        seen.append(True)
    t = threading.Thread(target=pretend)
    t.start()
    assert set_.wait(60)
    try:
        got = lib.w4_w4a16_linear_few(*args)
    finally:
        done.set()
        t.join()
    assert seen and torch.equal(got, want)
