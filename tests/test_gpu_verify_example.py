"""The verifying step's operators together, as examples/verify_tree.py runs them."""
import os
import random
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_trees_and_one_by_one(lib):
    """Every token that verifying keeps is one that decoding token by token may choose at
    that place: its logit there is the best one's or within what bf16 activations leave open
    (the two paths round alike values in other sums; a logit is off by well below 1/8 of the
    logits' spread), as long as the answers so far are the same."""
    import torch
    import verify_tree as ex
    model, r = ex.Model(), random.Random(5)
    prompts = [[r.randrange(ex.base.VOCAB) for _ in range(n)] for n in (70, 33, 5)]
    text, logits = ex.greedy(model, prompts, 16)
    answers, steps, chosen, cache = ex.verify(model, prompts, 16, ex.guesses(text, r))
    assert int(cache.status) == 0 and steps < 15
    compared = 0
    for i, (a, b) in enumerate(zip(text, answers)):
        assert a[0] == b[0]
        for t in range(1, 16):
            one, tree = logits[t - 1, i], chosen[i][t - 1]
            assert float((one - tree).abs().max()) < 0.125 * float(one.std())
            assert float(one.max() - one[b[t]]) < 0.25 * float(one.std())
            compared += 1
            if a[t] != b[t]:
                break
    assert compared >= 16
    # what the cache holds counts: the prompt and all answered tokens but the last
    assert cache.lens.tolist() == [len(p) + len(b) - 1 for p, b in zip(prompts, answers)]


def test_nothing_guessed_right(lib):
    """Trees of one node, and trees whose every guess is wrong, are decoding step by step."""
    import verify_tree as ex
    model = ex.Model()
    prompts = [[3, 1, 4, 1, 5, 9, 2, 6], [7] * 40]
    alone = ex.verify(model, prompts, 6, lambda i, a: ([a[-1]], [-1]))
    assert alone[1] == 5 and [len(a) for a in alone[0]] == [6, 6]
    assert alone[3].lens.tolist() == [13, 45] and int(alone[3].status) == 0
