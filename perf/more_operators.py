"""Timed cases of a decoding step that verifies drafted tokens: W4A16
projections for a few tokens, the norms of queries and keys with the position
rotation, the same on the way into a paged cache, attention for a tree of
drafted tokens over that cache, and keeping the accepted ones.

Each case runs either in its plain form (elementary torch operations in 32
bits, angles in 64, rounded once at the end) or, with ``own`` set, through the
library's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _linear(name, M, K, N, group):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "group": group}


def _rope(name, T, Hq, Hkv, D, rot, interleaved, norm, scaled, far, dtype):
    return {"name": name, "op": "rope", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "interleaved": interleaved, "norm": norm, "scaled": scaled, "far": far, "dtype": dtype}


def _append(name, seqs, new_lo, new_hi, before, Hq, Hkv, D, rot, page, drafted, dtype, pattern):
    return {"name": name, "op": "append", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi,
            "before": before, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "page": page,
            "drafted": drafted, "dtype": dtype, "pattern": pattern}


def _tree(name, groups, members, shared, tail, nodes_lo, nodes_hi, Hq, Hkv, D, page, dtype, pattern):
    return {"name": name, "op": "tree", "groups": groups, "members": members, "shared": shared,
            "tail": tail, "nodes_lo": nodes_lo, "nodes_hi": nodes_hi, "Hq": Hq, "Hkv": Hkv, "D": D,
            "page": page, "dtype": dtype, "pattern": pattern}


def _keep(name, seqs, before, nodes, kept_lo, kept_hi, layers, Hkv, D, page, pattern):
    return {"name": name, "op": "keep", "seqs": seqs, "before": before, "nodes": nodes,
            "kept_lo": kept_lo, "kept_hi": kept_hi, "layers": layers, "Hkv": Hkv, "D": D,
            "page": page, "pattern": pattern}


def listed():
    return [
        # one user's queries, keys and values: latency counts
        _linear("linear_1", 1, 2816, 4096, 128),
        # the down projection of a narrow MLP for a small tree, groups of 64, an odd output
        _linear("linear_11", 11, 704, 2815, 64),
        # the logits of as many tokens as count as few, over a large vocabulary
        _linear("linear_32", 32, 2816, 262144, 128),
        # one token's queries and keys
        _rope("rope_1", 1, 16, 8, 128, 128, False, True, False, 5000, "bf16"),
        # a long prompt far behind the trained length: half of each head rotated in
        # neighbouring pairs with scaled frequencies, no norm
        _rope("rope_long", 16387, 32, 4, 128, 64, True, False, True, 1000000, "fp16"),
        # a decoding step of 64 conversations, one token each
        _append("append_step", 64, 1, 1, 2000, 16, 8, 128, 128, 64, False, "bf16", 1),
        # a batch of prompts admitted
        _append("append_prompts", 48, 700, 1900, 0, 16, 8, 128, 128, 16, False, "bf16", 2),
        # one answer, a small tree of drafts
        _tree("tree_1", 1, 1, 0, 1511, 25, 25, 16, 8, 128, 16, "bf16", 3),
        # a chat server: 32 conversations behind one system prompt, trees of many sizes
        _tree("tree_chat", 1, 32, 8192, 800, 9, 60, 32, 4, 128, 64, "bf16", 4),
        # long documents of their own, large trees, narrow heads
        _tree("tree_long", 4, 1, 0, 50000, 64, 100, 24, 4, 64, 16, "fp16", 5),
        # one answer's accepted tokens in every layer
        _keep("keep_1", 1, 900, 25, 4, 4, 30, 8, 128, 16, 6),
        # the same for a server's batch
        _keep("keep_64", 64, 40, 48, 2, 9, 30, 8, 128, 64, 7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["linear", "linear", "linear", "rope", "rope", "append", "append", "tree",
                     "tree", "tree", "keep"])
    if op == "linear":
        group = rng.choice([64, 128, 128])
        M, K = _log_int(rng, 1, 32), group * _log_int(rng, 2, 128 * 64 // group)
        c = _linear("", M, K, _log_int(rng, 16, min(260000, 2816 * 262144 // K)), group)
    elif op == "rope":
        D = rng.choice([64, 80, 96, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        c = _rope("", _log_int(rng, 1, 6000), Hkv * rng.choice([1, 2, 4, 5]), Hkv, D,
                  rng.choice([D, D // 32 * 16]), rng.random() < 0.5, rng.random() < 0.5,
                  rng.random() < 0.5, _log_int(rng, 6000, 1000000), rng.choice(["bf16", "fp16"]))
    elif op == "append":
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        seqs = _log_int(rng, 1, 100)
        hi = _log_int(rng, 1, max(1, 30000 // seqs))
        c = _append("", seqs, max(1, hi // 3), hi, _log_int(rng, 1, 60000 // seqs),
                    Hkv * rng.choice([1, 2, 3, 8]), Hkv, D, rng.choice([D, D // 2]),
                    rng.choice([16, 32, 64, 128]), rng.random() < 0.4,
                    rng.choice(["bf16", "fp16"]), rng.randint(0, 10 ** 6))
    elif op == "tree":
        groups = rng.choice([1, 1, 2, 7])
        members = _log_int(rng, 1, max(1, 48 // groups))
        Hkv = rng.choice([1, 2, 4, 8])
        hi = _log_int(rng, 1, 128)
        shared = rng.choice([0, _log_int(rng, 1, 30000 // groups)])
        c = _tree("", groups, members, shared, _log_int(rng, 1, max(2, 60000 // (groups * members))),
                  max(1, hi // 4), hi, Hkv * rng.choice([1, 2, 4, 6]), Hkv, rng.choice([64, 128]),
                  rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "fp16"]),
                  rng.randint(0, 10 ** 6))
        while work(c)["flops"] > 1.2e11:        # no more than the largest listed case
            c["nodes_lo"], c["nodes_hi"] = _ceil(c["nodes_lo"], 2), _ceil(c["nodes_hi"], 2)
    else:
        seqs, nodes = _log_int(rng, 1, 64), rng.randint(2, 64)
        lo = rng.randint(1, max(1, nodes // 4))
        c = _keep("", seqs, _log_int(rng, 1, 300), nodes, lo, rng.randint(lo, max(lo, nodes // 3)),
                  rng.randint(1, 24), rng.choice([1, 4, 8]), rng.choice([64, 128]),
                  rng.choice([16, 32, 64]), rng.randint(0, 10 ** 6))
    del c["name"]
    return c


# --------------------------------------------------------------------------
# shapes that follow from a case alone
# --------------------------------------------------------------------------
def _ceil(a, b):
    return -(-a // b)


def _append_lengths(case):
    """(tokens before, new tokens) of each sequence."""
    r = random.Random(case["pattern"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    return [r.randint(case["before"] // 2, case["before"]) for _ in new], new


def _trees(case):
    """(length before its tree, parents of its nodes) of each sequence, members
    and shared length of each group."""
    r = random.Random(case["pattern"])
    seqs, sizes, shared = [], [], []
    for _ in range(case["groups"]):
        ragged = case["groups"] > 1 and case["members"] > 1
        n = r.randint(max(1, case["members"] // 2), case["members"]) if ragged else case["members"]
        s = r.randint(case["shared"] // 2, case["shared"])
        sizes.append(n)
        shared.append(s)
        for _ in range(n):
            nodes = r.randint(case["nodes_lo"], case["nodes_hi"])
            # the root is the last token taken; drafts hang mostly on recent ones
            parents = [-1] + [r.randint(max(0, i - 12), i - 1) for i in range(1, nodes)]
            seqs.append((s + r.randint((case["tail"] + 1) // 2, case["tail"]), parents))
    return seqs, sizes, shared


def _ancestors(parents):
    """Each node's ancestors and itself as a number's bits."""
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else 0) | (1 << i))
    return seen


def _kept(case):
    """(length before its tree, kept nodes) of each sequence.  A path starts with
    nodes that stand in their place already and goes on behind the number of kept
    ones, so that no node is moved over another one that is kept and a pass can be
    run again."""
    r = random.Random(case["pattern"])
    out = []
    for _ in range(case["seqs"]):
        n = r.randint(case["kept_lo"], case["kept_hi"])
        stay = r.randint(1, max(1, n // 2))
        stay = stay if case["nodes"] - n >= n - stay else n
        out.append((r.randint((case["before"] + 1) // 2, case["before"]),
                    list(range(stay)) + sorted(r.sample(range(n, case["nodes"]), n - stay))))
    return out


def work(case):
    op = case["op"]
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": N * (K // 2) + 4 * N * (K // case["group"]) + 2 * M * (K + N),
                "flops": 2.0 * M * N * K}
    if op == "rope":
        rows = case["T"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 4 * rows * case["D"] + 4 * case["T"], "flops": 0}
    if op == "append":
        T = sum(_append_lengths(case)[1])
        return {"bytes": 4 * T * (case["Hq"] + 2 * case["Hkv"]) * case["D"], "flops": 0}
    if op == "tree":
        seqs, sizes, shared = _trees(case)
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        keys, pairs, T, i = 0, 0, 0, 0
        for n, s in zip(sizes, shared):
            keys += s
            for before, parents in seqs[i:i + n]:
                keys += before - s + len(parents)
                pairs += before * len(parents) + sum(bin(a).count("1") for a in _ancestors(parents))
                T += len(parents)
            i += n
        return {"bytes": 4 * keys * Hkv * D + 4 * T * Hq * D, "flops": 4.0 * pairs * Hq * D}
    row = 2 * case["Hkv"] * case["D"] * 2 * case["layers"]
    moved = sum(sum(i != k for i, k in enumerate(kept)) for _, kept in _kept(case))
    return {"bytes": 2 * moved * row + 8 * case["seqs"], "flops": 0}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _randn_(t, g):
    for c in t.view(-1).split(1 << 26):
        c.copy_(torch.randn(c.shape, generator=g, device=DEV))
    return t


def _prepare_linear(case, seed):
    g = _gen(seed)
    M, K, N, group = (case[x] for x in ("M", "K", "N", "group"))
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=DEV)
    for c in q.view(-1).split(1 << 26):
        lo, hi = (torch.randn(c.shape, generator=g, device=DEV).mul_(2.6).add_(7.5).round_()
                  .clamp_(0, 15).to(torch.uint8) for _ in range(2))
        c.copy_(lo | (hi << 4))
    sh = (N, K // group)
    s = ((torch.rand(sh, generator=g, device=DEV) * 0.3 + 0.85) * (0.02 / 2.6)).half()
    z = (torch.rand(sh, generator=g, device=DEV) + 7.0).half()
    x = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
    return {"case": case, "x": x, "q": q, "s": s, "z": z}


# Frequencies of the rotation's pairs: base^(-2 i / rot), where scaled those that turn
# seldom within the trained length divided by the factor, those that turn often kept,
# the ones between a mixture by their number of turns.
BASE, FACTOR, TRAINED, LOW, HIGH, AMPLITUDE = 10000.0, 16.0, 8192, 1.0, 32.0, 1.2


def _frequencies(rot, scaled):
    f = [BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaled:
        for i, x in enumerate(f):
            keep = min(1.0, max(0.0, (TRAINED * x / (2 * math.pi) - LOW) / (HIGH - LOW)))
            f[i] = x * keep + x / FACTOR * (1.0 - keep)
    return f


def _steps(st, rot, scaled):
    """The rotation's frequencies as either side keeps them."""
    if own:
        import w4a16_moe_expert_sync_gb300 as w4
        if scaled:
            st["steps"] = w4.w4_rope_steps(rot, BASE, method="parts", factor=FACTOR,
                                           trained_len=TRAINED, low=LOW, high=HIGH, device=DEV)
        else:
            st["steps"] = w4.w4_rope_steps(rot, BASE, device=DEV)
    else:
        st["freq"] = torch.tensor(_frequencies(rot, scaled), dtype=torch.float64, device=DEV)
    st["amplitude"] = AMPLITUDE if scaled else 1.0


def _head_weights(g, D, dt):
    return [(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt) for _ in range(2)]


def _prepare_rope(case, seed):
    g = _gen(seed)
    T, Hq, Hkv, D = (case[x] for x in ("T", "Hq", "Hkv", "D"))
    dt = DTYPES[case["dtype"]]
    # queries, keys and values as one projection leaves them
    qkv = _randn_(torch.empty((T, Hq + 2 * Hkv, D), dtype=dt, device=DEV), g)
    first = random.Random(seed).randint(0, case["far"] - T) if case["far"] > T else 0
    st = {"case": case, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv],
          "positions": torch.arange(first, first + T, dtype=torch.int32, device=DEV),
          "weights": _head_weights(g, D, dt) if case["norm"] else [None, None]}
    _steps(st, case["rot"], case["scaled"])
    return st


def _pages(lens, page, seed):
    """A table [B, W] of random pages for these lengths, and their number."""
    need = [_ceil(n, page) for n in lens]
    P = sum(need) + sum(need) // 8 + 8
    perm = list(range(P))
    random.Random(seed).shuffle(perm)
    W, rows, at = max(need) + 2, [], 0
    for n in need:
        rows.append(perm[at:at + n] + [-1] * (W - n))
        at += n
    return _i32(rows), P


def _offsets(sizes):
    out = [0]
    for n in sizes:
        out.append(out[-1] + n)
    return out


def _prepare_append(case, seed):
    g = _gen(seed)
    before, new = _append_lengths(case)
    Hq, Hkv, D, page = (case[x] for x in ("Hq", "Hkv", "D", "page"))
    dt = DTYPES[case["dtype"]]
    lens = [a + b for a, b in zip(before, new)]
    table, P = _pages(lens, page, seed)
    T = sum(new)
    qkv = _randn_(torch.empty((T, Hq + 2 * Hkv, D), dtype=dt, device=DEV), g)
    cache = _randn_(torch.empty((2, P, page, Hkv, D), dtype=dt, device=DEV), g)
    r = random.Random(seed)
    st = {"case": case, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "v": qkv[:, Hq + Hkv:],
          "cache": cache, "table": table, "lens": _i32(lens), "q_offsets": _i32(_offsets(new)),
          "weights": _head_weights(g, D, dt), "positions": None}
    if case["drafted"]:
        # drafts of a tree stand at their depth, not at their place in the cache
        st["positions"] = _i32([a + r.randint(0, i) for a, n in zip(before, new) for i in range(n)])
    _steps(st, case["rot"], False)
    return st


def _prepare_tree(case, seed):
    g = _gen(seed)
    seqs, sizes, shared = _trees(case)
    page, Hq, Hkv, D = (case[x] for x in ("page", "Hq", "Hkv", "D"))
    lens = [before + len(parents) for before, parents in seqs]
    rows, used, copies, b = [], 0, [], 0
    for n, s in zip(sizes, shared):
        full = s // page
        first = list(range(used, used + full))
        used += full
        head = None
        for _ in range(n):
            mine = _ceil(lens[b], page) - full
            ids = list(range(used, used + mine))
            used += mine
            if s % page:                        # the prefix ends inside a page: one copy each
                if head is None:
                    head = ids[0]
                else:
                    copies.append((head, ids[0], s % page))
            rows.append(first + ids)
            b += 1
    P = used + used // 8 + 8
    perm = list(range(P))
    random.Random(seed).shuffle(perm)
    W = max(len(x) for x in rows) + 3
    dt = DTYPES[case["dtype"]]
    cache = _randn_(torch.empty((2, P, page, Hkv, D), dtype=dt, device=DEV), g)
    for a, c, t in copies:
        cache[:, perm[c], :t] = cache[:, perm[a], :t]
    nodes = [len(parents) for _, parents in seqs]
    T, max_q = sum(nodes), max(nodes)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV)
    qkv[:, :Hq] *= 1.5
    bits = []
    for _, parents in seqs:
        for a in _ancestors(parents):
            words = [(a >> (32 * i)) & 0xFFFFFFFF for i in range(_ceil(max_q, 32))]
            bits.append([w - (1 << 32) if w >> 31 else w for w in words])
    st = {"case": case, "q": qkv.to(dt)[:, :Hq], "k": cache[0], "v": cache[1],
          "table": _i32([[perm[p] for p in x] + [-1] * (W - len(x)) for x in rows]),
          "lens": _i32(lens), "q_offsets": _i32(_offsets(nodes)), "tree": _i32(bits),
          "group_offsets": _i32(_offsets(sizes)), "shared": _i32(shared), "lengths": lens,
          "nodes": nodes, "max_q": max_q}
    if own:
        import w4a16_moe_expert_sync_gb300 as w4
        need = w4.w4_attn_shared_prefix_workspace_size(T, len(lens), len(sizes), max_q, Hq, Hkv, D)
        st["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return st


def _prepare_keep(case, seed):
    g = _gen(seed)
    paths = _kept(case)
    lens = [before + case["nodes"] for before, _ in paths]
    table, P = _pages(lens, case["page"], seed)
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[table[table >= 0].long()] = 1
    pool = _randn_(torch.empty((case["layers"], 2, P, case["page"], case["Hkv"], case["D"]),
                               dtype=torch.bfloat16, device=DEV), g)
    return {"case": case, "pool": pool, "table": table, "lens": _i32(lens), "refs": refs,
            "q_offsets": _i32([i * case["nodes"] for i in range(len(lens) + 1)]),
            "kept": _i32([k for _, kept in paths for k in kept]),
            "kept_offsets": _i32(_offsets([len(kept) for _, kept in paths])),
            "lens_out": torch.empty(len(lens), dtype=torch.int32, device=DEV)}


_prepare = {"linear": _prepare_linear, "rope": _prepare_rope, "append": _prepare_append,
            "tree": _prepare_tree, "keep": _prepare_keep}


def prepare(case, seed):
    return _prepare[case["op"]](case, seed)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _own_linear(st):
    import w4a16_moe_expert_sync_gb300 as w4
    return w4.w4_w4a16_linear_few(st["x"], st["q"], st["s"], st["z"], st["case"]["group"])


def _own_rope(st):
    import w4a16_moe_expert_sync_gb300 as w4
    return w4.w4_qk_norm_rope(st["q"], st["k"], st["positions"], st["steps"],
                              q_weight=st["weights"][0], k_weight=st["weights"][1], eps=EPS,
                              interleaved=st["case"]["interleaved"], amplitude=st["amplitude"])


def _own_append(st):
    import w4a16_moe_expert_sync_gb300 as w4
    q = w4.w4_kv_append_rope(st["cache"][0], st["cache"][1], st["table"], st["lens"], st["q"],
                             st["k"], st["v"], st["q_offsets"], st["steps"],
                             positions=st["positions"], q_weight=st["weights"][0],
                             k_weight=st["weights"][1], eps=EPS)
    return q, st["cache"]


def _own_tree(st):
    import w4a16_moe_expert_sync_gb300 as w4
    return w4.w4_attn_tree(st["q"], st["k"], st["v"], st["table"], st["lens"], st["q_offsets"],
                           st["tree"], st["group_offsets"], st["shared"], max_q=st["max_q"],
                           workspace=st["ws"])


def _own_keep(st):
    import w4a16_moe_expert_sync_gb300 as w4
    w4.w4_kv_keep(st["pool"], st["table"], st["lens"], st["refs"], st["q_offsets"], st["kept"],
                  st["kept_offsets"], lens_out=st["lens_out"])
    return st["lens_out"], st["pool"]


_own = {"linear": _own_linear, "rope": _own_rope, "append": _own_append, "tree": _own_tree,
        "keep": _own_keep}


def _plain_linear(st):
    group, K = st["case"]["group"], st["case"]["K"]
    x, out = st["x"].float(), []
    for q, s, z in zip(*(st[n].split(max(1, (1 << 28) // K)) for n in ("q", "s", "z"))):
        c = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).float()
        w = (c - z.float().repeat_interleave(group, -1)) * s.float().repeat_interleave(group, -1)
        out.append(x @ w.T)
    return torch.cat(out, dim=1).to(torch.bfloat16)


def _turn(st, x, weight, positions, rot, interleaved):
    """x [T, H, D] normalised and rotated, in fp32."""
    u = x.float()
    if weight is not None:
        u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + EPS) * weight.float()
    angle = positions.double()[:, None] * st["freq"]
    cos, sin = (t.float()[:, None] * st["amplitude"] for t in (torch.cos(angle), torch.sin(angle)))
    if interleaved:
        a, b = u[..., 0:rot:2], u[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = u[..., :rot // 2], u[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, u[..., rot:]), dim=-1).to(x.dtype)


def _plain_rope(st):
    case = st["case"]
    return tuple(_turn(st, x, w, st["positions"], case["rot"], case["interleaved"])
                 for x, w in ((st["q"], st["weights"][0]), (st["k"], st["weights"][1])))


def _plain_append(st):
    page, rot = st["case"]["page"], st["case"]["rot"]
    start, end = st["q_offsets"][:-1].long(), st["q_offsets"][1:].long()
    t = torch.arange(st["q"].shape[0], device=DEV)
    seq = torch.searchsorted(end, t, right=True)
    at = t - end[seq] + st["lens"].long()[seq]
    pos = at if st["positions"] is None else st["positions"]
    where = st["table"][seq, at // page].long()
    st["cache"][0][where, at % page] = _turn(st, st["k"], st["weights"][1], pos, rot, False)
    st["cache"][1][where, at % page] = st["v"]
    return _turn(st, st["q"], st["weights"][0], pos, rot, False), st["cache"]


def _visible(st, b, L, n):
    """Which of its L keys each of sequence b's n queries sees, [n, L]."""
    words = st["tree"][st["q_offsets"][b]:st["q_offsets"][b + 1]]
    j = torch.arange(n, device=DEV)
    own_bits = (words[:, j // 32] >> (j % 32)) & 1
    return torch.cat((torch.ones((n, L - n), dtype=torch.bool, device=DEV), own_bits > 0), dim=1)


def _plain_tree(st):
    case = st["case"]
    page, D = case["page"], case["D"]
    rep = case["Hq"] // case["Hkv"]
    out = torch.empty(st["q"].shape, dtype=st["q"].dtype, device=DEV)
    at = 0
    for b, (L, n) in enumerate(zip(st["lengths"], st["nodes"])):
        pages = st["table"][b, :_ceil(L, page)].long()
        k = st["k"][pages].flatten(0, 1)[:L].float()
        v = st["v"][pages].flatten(0, 1)[:L].float()
        q = st["q"][at:at + n].float().unflatten(1, (case["Hkv"], rep))
        s = torch.einsum("thrd,lhd->hrtl", q, k) * (1.0 / math.sqrt(D))
        s = s.masked_fill(~_visible(st, b, L, n), float("-inf"))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.einsum("hrtl,lhd->thrd", p, v)
        o = o / p.sum(-1).permute(2, 0, 1)[..., None]
        out[at:at + n] = o.flatten(1, 2).to(out.dtype)
        at += n
    return out


def _plain_keep(st):
    page = st["case"]["page"]
    start = st["kept_offsets"].long()
    base = st["lens"].long() - (st["q_offsets"][1:] - st["q_offsets"][:-1]).long()
    i = torch.arange(st["kept"].numel(), device=DEV)
    seq = torch.searchsorted(start[1:], i, right=True)
    src, dst = base[seq] + st["kept"].long(), base[seq] + i - start[seq]
    sp, dp = st["table"][seq, src // page].long(), st["table"][seq, dst // page].long()
    for layer in st["pool"]:
        layer[:, dp, dst % page] = layer[:, sp, src % page]
    st["lens_out"].copy_(base + start[1:] - start[:-1])
    return st["lens_out"], st["pool"]


_plain = {"linear": _plain_linear, "rope": _plain_rope, "append": _plain_append,
          "tree": _plain_tree, "keep": _plain_keep}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    return _exact[case["op"]](case, seed) if case["op"] in _exact else None


def _exact_linear(case, seed):
    st = _prepare_linear(case, seed)
    M, K, N, group = (case[x] for x in ("M", "K", "N", "group"))
    x = st["x"].double().view(M, K // group, group)
    out = torch.empty((M, N), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 27) // K)
    for n in range(0, N, step):
        q = st["q"][n:n + step]
        w = torch.empty((q.shape[0], K), dtype=torch.float64, device=DEV)
        w[:, 0::2], w[:, 1::2] = (q % 16).double(), (q // 16).double()
        w = w.view(q.shape[0], K // group, group) - st["z"][n:n + step].double()[..., None]
        w *= st["s"][n:n + step].double()[..., None]
        out[:, n:n + step] = x.flatten(1) @ w.flatten(1).T
    return out


def _exact_turn(x, weight, positions, rot, interleaved, scaled):
    u = x.double()
    if weight is not None:
        u = u * (u.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight.double()
    f = torch.tensor(_frequencies(rot, scaled), dtype=torch.float64, device=DEV)
    # a pair of values is a complex number, turned by its position
    turn = torch.polar(torch.full((), AMPLITUDE if scaled else 1.0, dtype=torch.float64,
                                  device=DEV), positions.double()[:, None, None] * f)
    out = u.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    c = torch.complex(u[..., first], u[..., second]) * turn
    out[..., first], out[..., second] = c.real, c.imag
    return out


def _exact_rope(case, seed):
    st = _prepare_rope(case, seed)
    return tuple(_exact_turn(x, w, st["positions"], case["rot"], case["interleaved"], case["scaled"])
                 for x, w in ((st["q"], st["weights"][0]), (st["k"], st["weights"][1])))


def _exact_append(case, seed):
    st = _prepare_append(case, seed)
    before, new = _append_lengths(case)
    page = case["page"]
    places = [(b, a + i) for b, (a, n) in enumerate(zip(before, new)) for i in range(n)]
    seq = torch.tensor([b for b, _ in places], device=DEV)
    at = torch.tensor([i for _, i in places], device=DEV)
    pos = at if st["positions"] is None else st["positions"]
    row = st["table"].long()[seq, at // page] * page + at % page
    cache = st["cache"].double()
    flat = cache.flatten(1, 2)
    flat[0].index_copy_(0, row, _exact_turn(st["k"], st["weights"][1], pos, case["rot"], False,
                                            False))
    flat[1].index_copy_(0, row, st["v"].double())
    return _exact_turn(st["q"], st["weights"][0], pos, case["rot"], False, False), cache


def _exact_tree(case, seed):
    st = _prepare_tree(case, seed)
    seqs, _, _ = _trees(case)
    page, D, Hkv = case["page"], case["D"], case["Hkv"]
    rep = case["Hq"] // Hkv
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    t0 = 0
    for b, (before, parents) in enumerate(seqs):
        n = len(parents)
        L = before + n
        seen = torch.zeros((n, L), dtype=torch.bool)
        seen[:, :before] = True
        for i in range(n):
            j = i
            while j >= 0:                       # up to the root
                seen[i, before + j] = True
                j = parents[j]
        seen = seen.to(DEV).repeat_interleave(rep, 0)
        at = torch.arange(L, device=DEV)
        where = st["table"][b].long()[at // page] * page + at % page
        for h in range(Hkv):
            k = st["k"].flatten(0, 1)[where, h].double()
            v = st["v"].flatten(0, 1)[where, h].double()
            q = st["q"][t0:t0 + n, h * rep:(h + 1) * rep].double().reshape(-1, D)
            s = torch.where(seen, (q @ k.T) / D ** 0.5, -torch.inf)
            o = torch.softmax(s, dim=1) @ v
            out[t0:t0 + n, h * rep:(h + 1) * rep] = o.view(n, rep, D)
        t0 += n
    return out


# what is kept is moved, nothing is computed
_exact = {"linear": _exact_linear, "rope": _exact_rope, "append": _exact_append,
          "tree": _exact_tree}
