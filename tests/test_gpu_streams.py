"""Calls with a stream of their own and no workspace: the temporaries belong to
that stream, so that nothing on the current stream can take them while the
kernels run, and the results are not memory that earlier work of the current
stream still writes."""
import pytest

pytestmark = pytest.mark.gpu


def _calls():
    """name -> (call(lib, **kw) returning a tensor or tensors, or None)."""
    import torch
    from test_gpu_attention import _build, _run
    from test_gpu_few import _inputs
    x, logits, gu, dn = _inputs(6, 384, 192, 12, 3, seed=4)
    ids = logits.topk(3, 1).indices.int().contiguous()
    w = torch.full((6, 3), 1 / 3, device="cuda")
    c = _build([450, 500, 470], [2, 1, 3], [3], [430], 8, 4, 128, 32, "bfloat16", seed=4)
    pool = torch.randn((2, 2, 40, 8, 2, 16), device="cuda").bfloat16()
    ints = dict(dtype=torch.int32, device="cuda")
    table = torch.full((4, 8), -1, **ints)
    table[0, :4] = torch.tensor([30, 7, 12, 39], **ints)
    refs = torch.zeros(40, **ints)
    refs[table[0, :4].long()] = 1
    lens = torch.tensor([29, 0, 0, 0], **ints)
    parents, children = torch.tensor([0, 0], **ints), torch.tensor([1, 3], **ints)
    vocab = torch.randn((7, 5003), device="cuda")
    linear = tuple(t[0] for t in gu)
    calls = {
        "few": lambda lib, **kw: lib.w4_moe_layer_few(x, ids, w, gu, dn, **kw),
        "few_from_logits": lambda lib, **kw: lib.w4_moe_layer_few_from_logits(x, logits, 3, gu, dn,
                                                                              **kw),
        "attention": lambda lib, **kw: _run(lib, c, True, **kw),
        "layer": lambda lib, **kw: lib.w4_moe_layer(x, ids, w, gu, dn, **kw),
        "layer_from_logits": lambda lib, **kw: lib.w4_moe_layer_from_logits(x, logits, 3, gu, dn,
                                                                            **kw),
        "linear": lambda lib, **kw: lib.w4_w4a16_linear(x, *linear, **kw),
        "sampler": lambda lib, **kw: lib.w4_sample_logits(vocab, 5, **kw),
        "route": lambda lib, **kw: lib.w4_moe_route(logits, 3, **kw),
    }

    def fork(lib, **kw):
        state = [t.clone() for t in (pool, table, lens, refs)]
        torch.cuda.synchronize()
        lib.w4_kv_fork(*state, parents, children, **kw)
        return state

    def compact(lib, **kw):
        state = [t.clone() for t in (pool, table, refs)]
        torch.cuda.synchronize()
        lib.w4_kv_compact(*state, **kw)
        return state
    calls.update(fork=fork, compact=compact)
    return calls


NAMES = ["few", "few_from_logits", "attention", "layer", "layer_from_logits", "linear", "sampler",
         "route", "fork", "compact"]


def _list(out):
    return list(out) if isinstance(out, (tuple, list)) else [out]


@pytest.mark.parametrize("name", NAMES)
def test_temporaries_and_results_belong_to_the_stream(lib, monkeypatch, name):
    import torch
    from w4a16_moe_expert_sync_gb300 import _lib
    call = _calls()[name]
    want = _list(call(lib))
    torch.cuda.synchronize()
    # what the call allocates: (address, bytes), and whether it is let go at its end
    seen = []
    own = torch.empty

    def spy(*a, **kw):
        t = own(*a, **kw)
        seen.append((t.data_ptr(), t.nbytes, torch.cuda.current_stream().cuda_stream))
        return t
    s = torch.cuda.Stream()
    monkeypatch.setattr(torch, "empty", spy)
    got = _list(call(lib, stream=s))
    monkeypatch.undo()
    seen = [x for x in seen if x[1] > 0]
    kept = {t.data_ptr() for t in got}
    scratch = [x for x in seen if x[0] not in kept]
    if name != "route":
        assert scratch
    assert all(x[2] == s.cuda_stream for x in seen)
    # nothing on the current stream gets that memory
    for at, size, _ in scratch:
        blocks = [own(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(b.data_ptr() + size <= at or at + size <= b.data_ptr() for b in blocks)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(got) == len(want)
    assert _lib._scratch(16, torch.uint8, "cuda", None).shape == (16,)


@pytest.mark.parametrize("name", ["few", "few_from_logits", "attention", "layer", "linear", "sampler",
                                  "route"])
def test_results_are_not_what_earlier_work_still_writes(lib, name):
    """Memory that the current stream let go of, with a write to it still queued
    there, is not handed out as a result on the other stream."""
    import torch
    call = _calls()[name]
    want = _list(call(lib))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    held = [torch.empty_like(t) for t in want for _ in range(3)]
    for t in held:
        t.fill_(77)
    del held, t
    got = _list(call(lib, stream=s))
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_outlive_the_current_streams_use(lib):
    """A result let go while the current stream still has work on it is not handed
    out again before that has run."""
    import torch
    call = _calls()["few"]
    want = call(lib)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(lib, stream=s)
    s.synchronize()
    at = got.data_ptr()
    torch.cuda._sleep(100_000_000)
    copy = got.clone()
    del got
    with torch.cuda.stream(s):
        blocks = [torch.empty_like(want).fill_(77) for _ in range(4)]
    assert at not in [b.data_ptr() for b in blocks]
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
