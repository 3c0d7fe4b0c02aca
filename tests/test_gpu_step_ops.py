"""What the verifying step's operators have in common: nothing is allocated where outputs
and workspaces are given, temporaries and results belong to a call's stream, tensors of
another device are refused, two graphs share a workspace."""
import pytest

pytestmark = pytest.mark.gpu


def _setup():
    import torch
    from test_gpu_attention import _build
    from test_gpu_attn_tree import _tree, _words
    from test_gpu_linear_few import _inputs
    nodes = [6, 3]
    c = _build([126, 43], nodes, [], [], 8, 2, 64, 16, "bfloat16", seed=1)
    tree = _words([b for n in nodes for b in _tree(list(range(-1, n - 1)))], 1)
    ints = dict(dtype=torch.int32, device="cuda")
    x, q, s, z = _inputs(9, 1024, 12 * 64, 128, 1)
    d = dict(c=c, tree=tree, x=x, q=q, s=s, z=z,
             wide=_inputs(12, 512, 39000, 128, 2),
             lengths=torch.empty(2, **ints), refs=torch.ones(c["cache"].shape[1], **ints),
             kept=torch.tensor([0, 3, 5, 1], **ints), kept_offsets=torch.tensor([0, 3, 4], **ints),
             pos=torch.arange(9, **ints), status=torch.zeros(1, **ints),
             w=torch.ones(64, device="cuda").bfloat16())
    return d


def _calls(lib, d, **kw):
    """name -> call that returns its results."""
    c = d["c"]
    steps = lib.w4_rope_steps(64)
    kv = lib.w4_w4a16_linear_few(d["x"], d["q"], d["s"], d["z"]).view(9, 12, 64)
    q, k, v = kv[:, :8], kv[:, 8:10], kv[:, 10:]
    kp, vp = c["cache"][0], c["cache"][1]
    pool = c["cache"][None]
    return {
        "linear": lambda **o: lib.w4_w4a16_linear_few(d["x"], d["q"], d["s"], d["z"], **o),
        "wide": lambda **o: lib.w4_w4a16_linear_few(*d["wide"], **o),
        "rope": lambda **o: lib.w4_qk_norm_rope(q, k, d["pos"], steps, q_weight=d["w"], **o),
        "append": lambda **o: lib.w4_kv_append_rope(kp, vp, c["table"], c["lens"], q, k, v,
                                                    c["q_offsets"], steps, k_weight=d["w"], **o),
        "tree": lambda **o: lib.w4_attn_tree(c["q"], kp, vp, c["table"], c["lens"], c["q_offsets"],
                                             d["tree"], max_q=6, **o),
        "keep": lambda **o: lib.w4_kv_keep(pool, c["table"], c["lens"], d["refs"], c["q_offsets"],
                                           d["kept"], d["kept_offsets"],
                                           **dict(dict(lens_out=d["lengths"]), **o)),
    }


def _list(out):
    return list(out) if isinstance(out, (tuple, list)) else [out]


def test_nothing_is_allocated(lib):
    import torch
    d = _setup()
    calls = _calls(lib, d)
    held = {n: [torch.empty_like(t) for t in _list(calls[n]())] for n in ("linear", "wide", "rope",
                                                                         "append", "tree")}
    ws = torch.empty(lib.w4_attn_shared_prefix_workspace_size(9, 2, 0, 6, 8, 2, 64),
                     dtype=torch.uint8, device="cuda")

    def step():
        for n in ("linear", "wide", "append"):
            calls[n](**({"q_out" if n == "append" else "out": held[n][0]}))
        calls["rope"](q_out=held["rope"][0], k_out=held["rope"][1])
        calls["tree"](out=held["tree"][0], workspace=ws, dev_status=d["status"])
        calls["keep"](dev_status=d["status"])
    step()
    torch.cuda.synchronize()
    count = torch.cuda.memory_stats()["allocation.all.allocated"]
    for _ in range(3):
        step()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == count
    torch.cuda.synchronize()
    assert int(d["status"]) == 0


@pytest.mark.parametrize("name", ["linear", "wide", "rope", "append", "tree"])
def test_results_belong_to_the_stream(lib, monkeypatch, name):
    """What a call on a stream of its own takes is that stream's memory, and not what
    earlier work of the current one still writes."""
    import torch
    d = _setup()
    call = _calls(lib, d)[name]
    want = _list(call())
    torch.cuda.synchronize()
    seen, own = [], torch.empty

    def spy(*a, **kw):
        t = own(*a, **kw)
        seen.append(torch.cuda.current_stream().cuda_stream)
        return t
    s = torch.cuda.Stream()
    torch.cuda._sleep(50_000_000)
    held = [torch.empty_like(t) for t in want for _ in range(3)]
    for t in held:
        t.fill_(77)
    del held, t
    monkeypatch.setattr(torch, "empty", spy)
    got = _list(call(stream=s))
    monkeypatch.undo()
    s.synchronize()
    torch.cuda.synchronize()
    assert seen and all(x == s.cuda_stream for x in seen)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["linear", "rope", "append", "tree", "keep"])
def test_another_current_device_is_refused(lib, name):
    from w4a16_moe_expert_sync_gb300 import _lib
    d = _setup()
    call = _calls(lib, d)[name]
    call()
    _lib._calls().pretend_device(1)
    try:
        with pytest.raises(ValueError, match="current device"):
            call()
    finally:
        _lib._calls().pretend_device(-1)
    call()


def test_two_graphs_share_a_workspace(lib):
    """Captured with one workspace, replayed in turn: each its own results."""
    import torch
    d = _setup()
    calls = _calls(lib, d)
    ws = torch.empty(lib.w4_attn_shared_prefix_workspace_size(9, 2, 0, 6, 8, 2, 64),
                     dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(d["c"]["q"]) for _ in range(2)]
    want = calls["tree"]()
    graphs = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls["tree"](out=out, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_results_do_not_depend_on_what_the_workspace_held(lib):
    import torch
    d = _setup()
    calls = _calls(lib, d)
    ws = torch.full((lib.w4_attn_shared_prefix_workspace_size(9, 2, 0, 6, 8, 2, 64),), 255,
                    dtype=torch.uint8, device="cuda")
    want = calls["tree"]()
    assert torch.equal(calls["tree"](workspace=ws), want)
    ws.fill_(0)
    assert torch.equal(calls["tree"](workspace=ws), want)


def test_each_reads_what_the_one_before_wrote(lib):
    """A chain whose kernels begin while the one before still runs, over the same buffers
    with other values every time: as with a wait between all of them."""
    import torch
    d = _setup()
    c, steps = d["c"], lib.w4_rope_steps(64)
    _, w2, s2, z2 = (t.cuda() for t in d["wide"])
    kp, vp = c["cache"][0].clone(), c["cache"][1].clone()
    x, kv = torch.empty_like(d["x"]), torch.empty((9, 12, 64), dtype=torch.bfloat16, device="cuda")
    qr, o, y = torch.empty_like(c["q"]), torch.empty_like(c["q"]), []
    g = torch.Generator("cuda").manual_seed(8)
    inputs = [torch.randn(x.shape, device="cuda", generator=g).bfloat16() for _ in range(12)]
    norm = torch.ones(1024, device="cuda").bfloat16()
    ys = [torch.empty((9, 39000), dtype=torch.bfloat16, device="cuda") for _ in inputs]

    def run(wait):
        y.clear()
        for i, v in enumerate(inputs):
            lib.w4_rmsnorm(v, norm, out=x)
            wait()
            lib.w4_w4a16_linear_few(x, d["q"], d["s"], d["z"], out=kv.view(9, -1))
            wait()
            lib.w4_kv_append_rope(kp, vp, c["table"], c["lens"], kv[:, :8], kv[:, 8:10], kv[:, 10:],
                                  c["q_offsets"], steps, q_weight=d["w"], k_weight=d["w"], q_out=qr)
            wait()
            lib.w4_attn_tree(qr, kp, vp, c["table"], c["lens"], c["q_offsets"], d["tree"], max_q=6,
                             out=o)
            wait()
            lib.w4_w4a16_linear_few(o.view(9, -1), w2, s2, z2, out=ys[i])
            wait()
            y.append((qr.clone(), o.clone(), ys[i].clone()))
        torch.cuda.synchronize()
        return list(y)
    want = run(torch.cuda.synchronize)
    for _ in range(3):
        got = run(lambda: None)
        assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))


def test_from_two_threads(lib):
    """Two threads with a stream each, the same inputs: the same results as alone."""
    import threading
    import torch
    d = _setup()
    calls = _calls(lib, d)
    names = ("linear", "wide", "rope", "tree")
    want = {n: [t.clone() for t in _list(calls[n]())] for n in names}
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = {n: _list(calls[n]()) for n in names}
                    torch.cuda.current_stream().synchronize()
                    wrong.extend(n for n in names
                                 if not all(torch.equal(a, b) for a, b in zip(got[n], want[n])))
        except Exception as e:                 # noqa: BLE001 (shown by the assertion)
            wrong.append(repr(e))
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_results_are_ordinary_tensors(lib):
    """In inference mode too, and of inputs that ask for gradients (none is given)."""
    import torch
    d = _setup()
    calls = _calls(lib, d)
    want = calls["linear"]()
    assert not want.requires_grad and want.device == d["x"].device and want.is_contiguous()
    with torch.inference_mode():
        got = calls["linear"]()
        assert got.is_inference() and torch.equal(got.clone(), want)
    x = d["x"].clone().requires_grad_()
    got = lib.w4_w4a16_linear_few(x, d["q"], d["s"], d["z"])
    assert not got.requires_grad and torch.equal(got, want)
    w = torch.nn.Parameter(torch.ones(3, device="cuda", dtype=torch.bfloat16))
    (got[:, :3] * w).sum().backward()
    assert w.grad is not None
    with pytest.raises(lib.W4Error, match="M <= 32"):
        lib.w4_w4a16_linear_few(torch.zeros((33, 1024), device="cuda").bfloat16(), d["q"], d["s"],
                                d["z"])
