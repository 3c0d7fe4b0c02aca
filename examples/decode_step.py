"""A decoding step for a few drafts of one prompt, on a small random model.

One prompt is admitted into a paged cache and forked into several drafts, which
share its pages.  Every step of every layer is then the library's: RMSNorm, the
W4A16 projections, appending to the cache, attention that reads the shared
prompt once for all drafts, and the routed experts for a few tokens; tokens are
drawn by the one-pass sampler.  At the end all drafts but one are freed and the
pool is compacted.

    python examples/decode_step.py [--drafts 6] [--steps 8] [--prompt 300]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a16_moe_expert_sync_gb300 as w4  # noqa: E402

LAYERS, D_MODEL, M_EXPERT, EXPERTS, TOP_K = 2, 256, 128, 8, 2
HQ, HKV, HEAD, PAGE, VOCAB = 4, 2, 64, 16, 512


class Model:
    """Random weights of a decoder with W4A16 projections and routed experts."""

    def __init__(self, seed: int = 0, device: str = "cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device=device) * scale

        def linear(n, k):
            q, s, z = w4.w4_quantize(rand(n, k, scale=k ** -0.5), 128)
            return q[0], s[0], z[0]

        def experts(n, k, group):
            return w4.w4_quantize(rand(EXPERTS, n, k, scale=k ** -0.5), group)

        self.embed = rand(VOCAB, D_MODEL).bfloat16()
        self.head = linear(VOCAB, D_MODEL)
        self.layers = [dict(
            norm1=(1 + rand(D_MODEL, scale=0.1)).bfloat16(),
            norm2=(1 + rand(D_MODEL, scale=0.1)).bfloat16(),
            qkv=linear((HQ + 2 * HKV) * HEAD, D_MODEL), out=linear(D_MODEL, HQ * HEAD),
            router=rand(EXPERTS, D_MODEL, scale=D_MODEL ** -0.5),
            gate_up=experts(2 * M_EXPERT, D_MODEL, 128), down=experts(D_MODEL, M_EXPERT, 64))
            for _ in range(LAYERS)]


class Cache:
    """A paged cache: the pool and its state on the device."""

    def __init__(self, slots: int, pages: int, width: int, device: str = "cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.pool = torch.zeros((LAYERS, 2, pages, PAGE, HKV, HEAD), dtype=torch.bfloat16,
                                device=device)
        self.table = torch.full((slots, width), -1, **i32)
        self.lens = torch.zeros(slots, **i32)
        self.refs = torch.zeros(pages, **i32)
        self.status = torch.zeros(1, **i32)

    def grow(self, slots, lens):
        w4.w4_kv_reserve(self.table, self.lens, self.refs, slots, lens, PAGE,
                         dev_status=self.status)

    def fork(self, parents, children):
        w4.w4_kv_fork(self.pool, self.table, self.lens, self.refs, parents, children,
                      dev_status=self.status)

    def free(self, slots):
        w4.w4_kv_free(self.table, self.lens, self.refs, slots, dev_status=self.status)

    def compact(self):
        w4.w4_kv_compact(self.pool, self.table, self.refs, dev_status=self.status)


def forward(model, cache, tokens, rows, q_offsets, group_offsets, shared, max_q):
    """Logits [T, VOCAB] of `tokens` [T], appended to the cache's slots `rows`
    (a slice), whose lengths already count them."""
    table, lens, st = cache.table[rows], cache.lens[rows], cache.status
    x = model.embed[tokens]
    for i, layer in enumerate(model.layers):
        qkv = w4.w4_w4a16_linear(w4.w4_rmsnorm(x, layer["norm1"]), *layer["qkv"], dev_status=st)
        q, k, v = qkv.view(-1, HQ + 2 * HKV, HEAD).split((HQ, HKV, HKV), dim=1)
        pages = cache.pool[i]
        w4.w4_kv_append(pages[0], pages[1], table, lens, k, v, q_offsets, dev_status=st)
        a = w4.w4_attn_shared_prefix(q, pages[0], pages[1], table, lens, q_offsets, group_offsets,
                                     shared, max_q=max_q, causal=True, dev_status=st)
        x = x + w4.w4_w4a16_linear(a.flatten(1), *layer["out"], dev_status=st)
        y = w4.w4_rmsnorm(x, layer["norm2"])
        out = []
        for part in y.split(32):                 # the few-token layer takes up to 32
            logits = (part.float() @ layer["router"].T).contiguous()
            out.append(w4.w4_moe_layer_few_from_logits(part.contiguous(), logits, TOP_K,
                                                       layer["gate_up"], layer["down"],
                                                       dev_status=st)[0])
        x = x + torch.cat(out)
    return w4.w4_w4a16_linear(x, *model.head, dev_status=st).float()


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def decode(model, prompt, drafts: int, steps: int, share: bool = True, seed: int = 1, forced=None):
    """Draws `steps` tokens for each of `drafts` continuations of the prompt (or
    takes forced [drafts, steps]).  Returns (tokens, logits [steps, drafts,
    VOCAB], cache); the drafts are slots 1 .. drafts."""
    n = len(prompt)
    cache = Cache(drafts + 1, (n + steps) // PAGE * (drafts + 1) + 2 * drafts + 4,
                  (n + steps) // PAGE + 2)
    cache.grow(ints([0]), ints([n]))
    forward(model, cache, torch.tensor(prompt, device="cuda"), slice(0, 1), ints([0, n]), None,
            None, n)
    cache.fork(ints([0] * drafts), ints(range(1, drafts + 1)))
    rows = slice(1, drafts + 1)
    slots = ints(range(1, drafts + 1))
    offsets = ints(range(drafts + 1))
    # the drafts are one group: the prompt's tokens, wherever its last page ends
    groups, shared = (ints([0, drafts]), ints([n])) if share else (None, None)
    last = torch.tensor([prompt[-1]] * drafts, device="cuda")
    tokens, logits = [], []
    for t in range(steps):
        cache.grow(slots, cache.lens[rows] + 1)
        out = forward(model, cache, last, rows, offsets, groups, shared, 1)
        if forced is None:
            last = w4.w4_gumbel_argmax_sample(out.contiguous(), seed, t)[0]
        else:
            last = forced[:, t]
        tokens.append(last)
        logits.append(out)
    return torch.stack(tokens, 1), torch.stack(logits), cache


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--drafts", type=int, default=6)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=300)
    a = ap.parse_args()
    model = Model()
    g = torch.Generator().manual_seed(2)
    prompt = torch.randint(0, VOCAB, (a.prompt,), generator=g).tolist()
    tokens, logits, cache = decode(model, prompt, a.drafts, a.steps)
    used = int((cache.refs > 0).sum())
    alone = (a.drafts + 1) * -(-(a.prompt + a.steps) // PAGE)
    print(f"{a.drafts} drafts of {a.steps} tokens after {a.prompt}: {used} pages in use "
          f"({alone} without sharing)")
    print(tokens.tolist())
    best = int(torch.log_softmax(logits, -1).gather(
        2, tokens.T[..., None]).sum((0, 2)).argmax()) + 1
    cache.free(ints([s for s in range(a.drafts + 1) if s != best]))
    cache.compact()
    kept = int((cache.refs > 0).sum())
    print(f"draft {best - 1} kept: {kept} pages, the pool's first: "
          f"{bool((cache.refs[:kept] > 0).all())}, status {int(cache.status)}")


if __name__ == "__main__":
    main()
