"""The decoding example: drafts that share their prompt's pages give the logits
that they give alone, and the cache's accounts come out even."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location(
        "decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.gpu
@pytest.mark.parametrize("length,drafts,steps", [(37, 5, 6), (32, 1, 3), (301, 9, 20)])
def test_drafts_share_and_agree(lib, monkeypatch, length, drafts, steps):
    import torch
    ex = _example()
    model = ex.Model()
    prompt = torch.randint(0, ex.VOCAB, (length,),
                           generator=torch.Generator().manual_seed(length)).tolist()
    # The choice of experts is discrete: two runs that differ by rounding may
    # choose differently where two logits nearly tie, and then differ by an
    # expert's whole output.  The second run takes the first's choices, weighted by
    # its own logits, and its own choice may differ only at such a tie.
    own, chosen, ties = ex.w4.w4_moe_layer_few_from_logits, [], []

    def record(x, logits, k, *a, **kw):
        out = own(x, logits, k, *a, **kw)
        chosen.append(out[1])
        return out

    def replay(x, logits, k, gu, dn, **kw):
        ids = chosen[len(ties)]
        at = logits.gather(1, ids.long())
        best = logits.topk(k, dim=1).values
        ties.append(float((best.sort(1).values - at.sort(1).values).max()))
        return (ex.w4.w4_moe_layer_few(x, ids, torch.softmax(at, 1), gu, dn, **kw),)

    monkeypatch.setattr(ex.w4, "w4_moe_layer_few_from_logits", record)
    tokens, shared, cache = ex.decode(model, prompt, drafts, steps)
    monkeypatch.setattr(ex.w4, "w4_moe_layer_few_from_logits", replay)
    _, alone, _ = ex.decode(model, prompt, drafts, steps, share=False, forced=tokens)
    print("largest gap of a choice that differs:", max(ties), "difference:",
          float((shared - alone).abs().max()))
    assert len(ties) == len(chosen) and max(ties) <= 0.15
    # the two differ in where the prefix's partial sums are cut: rounding that the
    # later layers' bf16 steps can amplify a little; logits have an rms near 1
    assert float((shared - alone).abs().max()) <= 0.15 * float(alone.pow(2).mean().sqrt())
    assert int(cache.status) == 0
    # the first step: every draft sees the same, so gives the same
    assert torch.equal(shared[0], shared[0, :1].expand_as(shared[0]))
    full = length // ex.PAGE
    assert cache.refs[cache.table[1, :full].long()].tolist() == [drafts + 1] * full
    keep = drafts
    before = cache.pool[:, :, cache.table[keep, :-(-(length + steps) // ex.PAGE)].long()].clone()
    cache.free(ex.ints([s for s in range(drafts + 1) if s != keep]))
    cache.compact()
    kept = -(-(length + steps) // ex.PAGE)
    assert cache.refs.tolist() == [1] * kept + [0] * (cache.refs.numel() - kept)
    assert torch.equal(cache.pool[:, :, cache.table[keep, :kept].long()], before)
    cache.free(ex.ints([keep]))
    assert int(cache.refs.abs().sum()) == 0 and int(cache.lens.sum()) == 0
