"""The bounded waits of the decoding step's kernels, made to run out through the
library's test hook: each CTA (or warp) never counts its first copy as landed, the
wait for it gives up after 2 ms, the kernel sets W4_DEV_PIPELINE_TIMEOUT, gives
what it has under way its time to land and ends.  Nothing faults or hangs: every wait is bounded, and the
context then gives the normal result bit for bit."""
import time

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture
def hooks(lib):
    clib = lib.load_library()
    yield clib
    clib.w4_test_pipeline_hooks(0, 0)


def _times_out(lib, hooks, call):
    """The call's result without the hooks, with a short limit alone, and after a
    call whose first copies never count as landed: the same bits, and status words of 0,
    0 and a timeout."""
    import torch
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = call(st)
    torch.cuda.synchronize()
    assert int(st) == 0
    hooks.w4_test_pipeline_hooks(50_000_000, 0)
    assert torch.equal(call(st), want) and int(st) == 0
    hooks.w4_test_pipeline_hooks(2_000_000, 1)
    t0 = time.perf_counter()
    call(st)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert int(st) & lib.W4_DEV_PIPELINE_TIMEOUT
    hooks.w4_test_pipeline_hooks(0, 0)
    st.zero_()
    for _ in range(3):
        assert torch.equal(call(st), want)
    assert int(st) == 0


@pytest.mark.parametrize("lens,nqs,groups,shared,Hq,Hkv,D,page", [
    ([40, 33], [1, 1], [], [], 2, 1, 64, 16),                         # single items, few tiles
    ([3000] * 40, [1] * 40, [40], [2500], 8, 4, 128, 64),             # both streams of a CTA, long
    ([1700, 1703], [200, 180], [2], [1500], 4, 2, 128, 16),           # pairs, ends cleared by both
    ([5000, 900, 17], [1, 300, 5], [2], [777], 6, 2, 64, 32)])        # pairs and single items
def test_attention(lib, hooks, lens, nqs, groups, shared, Hq, Hkv, D, page):
    from test_gpu_attention import _build, _run
    c = _build(lens, nqs, groups, shared, Hq, Hkv, D, page, "bfloat16", seed=7)
    _times_out(lib, hooks, lambda st: _run(lib, c, True, dev_status=st))


@pytest.mark.parametrize("M,d,m,E,k", [(1, 128, 64, 1, 1), (7, 2816, 704, 16, 8), (32, 384, 192, 12, 8),
                                       (3, 6144, 64, 4, 2)])
def test_few_token_layer(lib, hooks, M, d, m, E, k):
    from test_gpu_few import _inputs
    x, logits, gu, dn = _inputs(M, d, m, E, k)
    _times_out(lib, hooks,
               lambda st: lib.w4_moe_layer_few_from_logits(x, logits, k, gu, dn, dev_status=st)[0])


@pytest.mark.parametrize("planes,page,Hkv,D", [(1, 4, 1, 8), (2, 16, 2, 64), (6, 64, 8, 128)])
def test_page_copies(lib, hooks, planes, page, Hkv, D):
    import torch
    P = 900
    pool = torch.randn((planes, P, page, Hkv, D), device="cuda").bfloat16()
    perm = torch.randperm(P, device="cuda").int()
    refs = (torch.rand(P, device="cuda") < 0.4).int()
    table = torch.where(refs > 0, torch.arange(P, device="cuda").int(), -1)[None]

    def copy(st):
        out = pool.clone()
        lib.w4_kv_copy_pages(out, perm[:400].contiguous(), perm[400:800].contiguous(), dev_status=st)
        return out

    def compact(st):
        out = pool.clone()
        lib.w4_kv_compact(out, table.clone(), refs.clone(), dev_status=st)
        return out
    _times_out(lib, hooks, copy)
    _times_out(lib, hooks, compact)
