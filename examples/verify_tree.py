"""Trees of drafted tokens verified for a few answers, on a small random model.

Prompts are admitted into a paged cache.  Then every step takes a tree of guesses
for each answer: the projections for a few tokens, the norms of queries and keys
with the rotation on the way into the cache (a guess stands at its depth), attention
that sees a guess's ancestors, and the routed experts for a few tokens, all guesses at
once; the longest path that the model itself would have chosen is kept, the rest is
taken back.

    python examples/verify_tree.py [--answers 3] [--tokens 24] [--prompt 70]
"""
from __future__ import annotations

import argparse
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import decode_step as base  # noqa: E402
from decode_step import Cache, ints, w4  # noqa: E402

HQ, HKV, HEAD, TOP_K = base.HQ, base.HKV, base.HEAD, base.TOP_K


class Model(base.Model):
    """The other example's model with norms of queries and keys and a rotation."""

    def __init__(self, seed: int = 0, device: str = "cuda"):
        super().__init__(seed, device)
        g = torch.Generator(device=device).manual_seed(seed + 1)
        for layer in self.layers:
            for name in ("q_norm", "k_norm"):
                layer[name] = (1 + 0.1 * torch.randn(HEAD, generator=g, device=device)).bfloat16()
        self.steps = w4.w4_rope_steps(HEAD, device=device)


def project(x, weight, status):
    """Rows of x through a W4A16 weight, by the path that their number asks for."""
    if x.shape[0] <= 32:
        return w4.w4_w4a16_linear_few(x, *weight, dev_status=status)
    return w4.w4_w4a16_linear(x, *weight, dev_status=status)


def forward(model, cache, tokens, rows, q_offsets, max_q, positions=None, tree=None):
    """Logits [T, VOCAB] of `tokens`, appended to the cache's slots `rows` (a slice),
    whose lengths already count them; with a tree's bits, or causal without."""
    table, lens, st = cache.table[rows], cache.lens[rows], cache.status
    x = model.embed[tokens]
    for i, layer in enumerate(model.layers):
        qkv = project(w4.w4_rmsnorm(x, layer["norm1"]), layer["qkv"], st)
        q, k, v = qkv.view(-1, HQ + 2 * HKV, HEAD).split((HQ, HKV, HKV), dim=1)
        pages = cache.pool[i]
        q = w4.w4_kv_append_rope(pages[0], pages[1], table, lens, q, k, v, q_offsets, model.steps,
                                 positions=positions, q_weight=layer["q_norm"],
                                 k_weight=layer["k_norm"], dev_status=st)
        if tree is None:
            a = w4.w4_attn_shared_prefix(q, pages[0], pages[1], table, lens, q_offsets, max_q=max_q,
                                         dev_status=st)
        else:
            a = w4.w4_attn_tree(q, pages[0], pages[1], table, lens, q_offsets, tree, max_q=max_q,
                                dev_status=st)
        x = x + project(a.flatten(1), layer["out"], st)
        y = w4.w4_rmsnorm(x, layer["norm2"])
        out = []
        for part in y.split(32):                 # the few-token layer takes up to 32
            logits = (part.float() @ layer["router"].T).contiguous()
            out.append(w4.w4_moe_layer_few_from_logits(part.contiguous(), logits, TOP_K,
                                                       layer["gate_up"], layer["down"],
                                                       dev_status=st)[0])
        x = x + torch.cat(out)
    return project(x, model.head, st).float()


def admit(model, prompts, room: int):
    """A cache with the prompts, and the token that the model chooses after each."""
    n, longest = len(prompts), max(len(p) for p in prompts)
    width = (longest + room) // base.PAGE + 2
    cache = Cache(n, n * width, width)
    cache.grow(ints(range(n)), ints([len(p) for p in prompts]))
    offsets = [0]
    for p in prompts:
        offsets.append(offsets[-1] + len(p))
    logits = forward(model, cache, torch.tensor(sum(prompts, []), device="cuda"), slice(0, n),
                     ints(offsets), longest)
    return cache, logits[[o - 1 for o in offsets[1:]]].argmax(1).tolist()


def greedy(model, prompts, tokens: int):
    """The answers, token by token, and the logits that chose them [tokens, answers, VOCAB]."""
    cache, last = admit(model, prompts, tokens)
    n = len(prompts)
    answers, logits = [[t] for t in last], []
    for _ in range(tokens - 1):
        cache.grow(ints(range(n)), cache.lens + 1)
        out = forward(model, cache, torch.tensor(last, device="cuda"), slice(0, n),
                      ints(range(n + 1)), 1)
        logits.append(out)
        last = out.argmax(1).tolist()
        for a, t in zip(answers, last):
            a.append(t)
    return answers, torch.stack(logits)


def verify(model, prompts, tokens: int, guess):
    """The answers by verifying trees: guess(answer, so far) gives a tree's tokens and the
    parents of its nodes; node 0 is the last token taken.  Returns (answers, steps, the
    logits that chose each token after the first, the cache)."""
    cache, last = admit(model, prompts, tokens + 33)
    n, steps = len(prompts), 0
    answers, logits = [[t] for t in last], [[] for _ in last]
    slots = ints(range(n))
    while min(len(a) for a in answers) < tokens:
        trees = [guess(i, a) for i, a in enumerate(answers)]
        sizes = [len(t) for t, _ in trees]
        offsets, depths, bits, most = [0], [], [], max(sizes)
        for nodes, parents in trees:
            offsets.append(offsets[-1] + len(nodes))
            seen, depth = [], []
            for i, p in enumerate(parents):
                seen.append((seen[p] if i else 0) | (1 << i))
                depth.append(depth[p] + 1 if i else 0)
            depths.append(depth)
            bits += [[b >> 32 * w & 0xFFFFFFFF for w in range(-(-most // 32))] for b in seen]
        before = cache.lens.tolist()
        cache.grow(slots, cache.lens + ints(sizes))
        out = forward(model, cache, torch.tensor(sum((t for t, _ in trees), []), device="cuda"),
                      slice(0, n), ints(offsets), most,
                      positions=ints([b + d for b, ds in zip(before, depths) for d in ds]),
                      tree=torch.tensor(bits, device="cuda").to(torch.int32))
        best = out.argmax(1).tolist()
        kept, kept_offsets = [], [0]
        for i, (nodes, parents) in enumerate(trees):
            at, path = 0, [0]
            while True:                          # down to the child that the model chose
                chosen = best[offsets[i] + at]
                answers[i].append(chosen)
                logits[i].append(out[offsets[i] + at])
                child = [c for c in range(at + 1, len(nodes)) if parents[c] == at and
                         nodes[c] == chosen]
                if not child:
                    break
                at = child[0]
                path.append(at)
            kept += path
            kept_offsets.append(len(kept))
        w4.w4_kv_keep(cache.pool, cache.table, cache.lens, cache.refs, ints(offsets), ints(kept),
                      ints(kept_offsets), dev_status=cache.status)
        steps += 1
    return answers, steps, logits, cache


def guesses(text, r, right: float = 0.8):
    """A drafter that knows the answers and errs: the next tokens, each wrong with some
    probability, and beside each a wrong sibling with a child."""
    def guess(i, so_far):
        ahead = text[i][len(so_far):len(so_far) + 4]
        nodes, parents, at = [so_far[-1]], [-1], 0
        for t in ahead:
            nodes += [t if r.random() < right else r.randrange(base.VOCAB), r.randrange(base.VOCAB)]
            parents += [at, at]
            nodes.append(r.randrange(base.VOCAB))
            parents.append(len(nodes) - 2)
            at = len(nodes) - 3
        return nodes, parents
    return guess


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--answers", type=int, default=3)
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--prompt", type=int, default=70)
    a = ap.parse_args()
    model, r = Model(), random.Random(2)
    prompts = [[r.randrange(base.VOCAB) for _ in range(a.prompt + 9 * i)] for i in range(a.answers)]
    text, _ = greedy(model, prompts, a.tokens)
    answers, steps, _, cache = verify(model, prompts, a.tokens, guesses(text, r))
    alike = sum(x == y for t, u in zip(text, answers) for x, y in zip(t, u))
    print(f"{a.answers} answers of {a.tokens} tokens in {steps} steps instead of {a.tokens - 1}; "
          f"{alike} of {a.answers * a.tokens} tokens as one by one, status {int(cache.status)}")


if __name__ == "__main__":
    main()
