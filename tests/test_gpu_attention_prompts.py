"""Attention and appending on batches that a server forms: a causal prompt of some
thousand tokens, and one prompt among many single tokens; and the router's choices in
the decoding example, exactly."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,nqs,groups,shared,Hq,Hkv,D,page,dtype", [
    ([2048], [2048], [], [], 4, 2, 128, 64, "bfloat16"),
    ([2500], [2048], [], [], 6, 2, 64, 16, "float16"),                  # behind 452 cached tokens
    ([2048, 1999], [2048, 99], [2], [1900], 4, 2, 128, 16, "bfloat16"),
    ([2048] + [100 + 7 * i for i in range(200)], [2048] + [1] * 200, [], [], 4, 2, 64, 32,
     "bfloat16"),
    ([40 + i for i in range(100)] + [1500] + [300] * 100, [1] * 100 + [1500] + [1] * 100, [100],
     [33], 4, 1, 128, 16, "float16")])
def test_prompts(lib, lens, nqs, groups, shared, Hq, Hkv, D, page, dtype):
    import torch
    from test_gpu_attention import _build, _check, _run
    c = _build(lens, nqs, groups, shared, Hq, Hkv, D, page, dtype, seed=len(lens))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run(lib, c, True, dev_status=st)
    assert int(st) == 0
    _check(got, c, True)
    assert torch.equal(_run(lib, c, True), got)


@pytest.mark.parametrize("B,prompt,at", [(256, 2048, 255), (256, 2048, 0), (40, 333, 7), (256, 1, 3)])
def test_appending_a_mixed_batch(lib, B, prompt, at):
    """Sequence `at` brings a prompt, every other one token."""
    import torch
    page, Hkv, D = 16, 2, 64
    ints = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(B)
    lens = torch.randint(1, 90, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[at] = prompt
    need = (lens + page - 1) // page
    W, P = int(need.max()), int(need.sum()) + 3
    perm = torch.randperm(P, generator=g, device="cuda").int()
    table, start = torch.full((B, W), -1, **ints), 0
    for b, n in enumerate(need.tolist()):
        table[b, :n] = perm[start:start + n]
        start += n
    nq = torch.ones(B, **ints)
    nq[at] = prompt
    offs = torch.zeros(B + 1, **ints)
    offs[1:] = nq.cumsum(0)
    kv = torch.randn((int(offs[-1]), 2, Hkv, D), generator=g, device="cuda").bfloat16()
    cache = torch.zeros((2, P, page, Hkv, D), device="cuda").bfloat16()
    want = cache.clone()
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), nq.long())
    pos = (lens[seq] - (offs[1:][seq] - torch.arange(len(seq), device="cuda"))).long()
    where = table[seq, pos // page].long()
    for i in range(2):
        want[i, where, pos % page] = kv[:, i]
    st = torch.zeros(1, **ints)
    lib.w4_kv_append(cache[0], cache[1], table, lens, kv[:, 0], kv[:, 1], offs, dev_status=st)
    assert int(st) == 0 and torch.equal(cache, want)


def test_the_examples_choices_are_the_routers(lib, monkeypatch):
    """Every expert choice and weight in the decoding example is w4_moe_route's for the
    same logits, bit for bit, and each call's output that of the layer with them."""
    import torch
    from test_gpu_decode_example import _example
    ex = _example()
    model = ex.Model()
    own, calls = ex.w4.w4_moe_layer_few_from_logits, []

    def routed(x, logits, k, gu, dn, **kw):
        out, ids, w = own(x, logits, k, gu, dn, **kw)
        want_ids, want_w = lib.w4_moe_route(logits, k)
        assert torch.equal(ids, want_ids) and torch.equal(w, want_w)
        assert torch.equal(out, lib.w4_moe_layer_few(x, ids, w, gu, dn))
        calls.append(x.shape[0])
        return out, ids, w
    monkeypatch.setattr(ex.w4, "w4_moe_layer_few_from_logits", routed)
    prompt = torch.randint(0, ex.VOCAB, (75,), generator=torch.Generator().manual_seed(3)).tolist()
    ex.decode(model, prompt, 4, 3)
    assert len(calls) == ex.LAYERS * (3 + 3)     # three parts of the prompt, three steps
