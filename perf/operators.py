"""Timed cases of the decode-step operators: the routed mixture-of-experts
layer for a few tokens, attention over a paged cache whose sequences share a
prefix, and the cache's page operations.

Each case runs either in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, with ``own`` set, through the library's
entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _moe(name, M, d, m, E, k, logits):
    return {"name": name, "op": "moe", "M": M, "d": d, "m": m, "E": E, "k": k, "logits": logits}


def _attn(name, groups, members, shared, tail_lo, tail_hi, nq, causal, Hq, Hkv, D, page, dtype,
          pattern):
    return {"name": name, "op": "attn", "groups": groups, "members": members, "shared": shared,
            "tail_lo": tail_lo, "tail_hi": tail_hi, "nq": nq, "causal": causal, "Hq": Hq,
            "Hkv": Hkv, "D": D, "page": page, "dtype": dtype, "pattern": pattern}


def _pages(name, op, slots, length, children, layers, Hkv, D, page, pattern):
    return {"name": name, "op": op, "slots": slots, "length": length, "children": children,
            "layers": layers, "Hkv": Hkv, "D": D, "page": page, "pattern": pattern}


def listed():
    return [
        # one user, one token a step: latency counts
        _moe("moe_1", 1, 2816, 704, 128, 8, True),
        # a handful of users, an odd count, routing already at hand
        _moe("moe_7", 7, 2816, 704, 128, 8, False),
        # the largest batch that still counts as a few tokens
        _moe("moe_32", 32, 2816, 704, 128, 8, True),
        # two answers drafted from one short prompt
        _attn("attn_pair", 1, 2, 203, 1, 40, 1, True, 16, 8, 128, 16, "bf16", 1),
        # a chat server: 64 conversations behind one system prompt
        _attn("attn_chat", 1, 64, 8192, 33, 1500, 1, True, 16, 8, 128, 64, "bf16", 2),
        # questions about one long document
        _attn("attn_document", 1, 32, 120000, 5, 300, 1, True, 32, 4, 128, 128, "bf16", 3),
        # four 256-token canvases denoised over one prompt, no causal mask
        _attn("attn_canvas", 1, 4, 4096, 256, 256, 256, False, 16, 8, 128, 32, "bf16", 4),
        # several prompts with ragged groups, a few speculative tokens each
        _attn("attn_ragged", 9, 7, 1777, 9, 700, 5, True, 24, 4, 64, 16, "fp16", 5),
        # admitting a batch of prompts: release, reserve and fill their pages
        _pages("pages_admit", "admit", 48, 1900, 0, 1, 8, 128, 16, 6),
        # re-drafting: children released and forked again from their prompts
        _pages("pages_fork", "fork", 4, 9000, 96, 8, 8, 128, 64, 7),
        # copying finished pages into the pages of another place in the pool
        _pages("pages_copy", "copy", 16, 2000, 0, 8, 8, 128, 32, 8),
        # half of the sequences have left: the rest moves to the pool's front
        _pages("pages_compact", "compact", 64, 3000, 0, 8, 8, 128, 64, 9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["moe", "moe", "attn", "attn", "attn", "admit", "fork", "copy", "compact"])
    if op == "moe":
        d, m, E, k = rng.choice([(2816, 704, 128, 8), (2816, 704, 128, 8), (384, 192, 12, 3),
                                 (256, 128, 8, 2), (2048, 512, 64, 6), (1152, 320, 40, 4)])
        c = _moe("", _log_int(rng, 1, 32), d, m, E, k, rng.random() < 0.5)
    elif op == "attn":
        groups = rng.choice([1, 1, 2, 5, 11])
        members = _log_int(rng, 1, max(1, 64 // groups))
        D = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        budget = 120000 * 32 * 32 // (groups * members * Hq)
        shared = _log_int(rng, 1, max(2, min(65000 // groups, budget)))
        nq = rng.choice([1, 1, 1, 4, 33])
        if groups * members * nq * Hq * shared > 120000 * 32 * 32:
            nq = 1
        lo = rng.randint(nq, nq + 50)
        c = _attn("", groups, members, shared, lo, lo + _log_int(rng, 1, 1000), nq,
                  rng.random() < 0.6, Hq, Hkv, D, rng.choice([16, 32, 64, 128]),
                  rng.choice(["bf16", "fp16"]), rng.randint(0, 10 ** 6))
    else:
        page = rng.choice([16, 32, 64])
        slots = _log_int(rng, 2, 48)
        c = _pages("", op, slots, _log_int(rng, 10, 2500),
                   slots * rng.randint(1, 4) if op == "fork" else 0,
                   1 if op == "admit" else rng.randint(1, 6), rng.choice([1, 4, 8]),
                   rng.choice([64, 128]), page, rng.randint(0, 10 ** 6))
    del c["name"]
    return c


# --------------------------------------------------------------------------
# shapes that follow from a case alone
# --------------------------------------------------------------------------
def _attn_lengths(case):
    """(lengths of the sequences, members of each group, shared lengths)."""
    r = random.Random(case["pattern"])
    sizes, shared, lens = [], [], []
    for g in range(case["groups"]):
        ragged = case["groups"] > 1
        n = r.randint(max(1, case["members"] // 2), case["members"]) if ragged else case["members"]
        s = r.randint(max(0, case["shared"] // 3), case["shared"]) if ragged else case["shared"]
        sizes.append(n)
        shared.append(s)
        lens += [s + r.randint(case["tail_lo"], case["tail_hi"]) for _ in range(n)]
    return lens, sizes, shared


def _page_lengths(case):
    """Lengths of the sequences of a page-operation case."""
    r = random.Random(case["pattern"])
    return [r.randint(max(1, case["length"] // 2), case["length"]) for _ in range(case["slots"])]


def _ceil(a, b):
    return -(-a // b)


def _copy_pairs(case):
    return sum(_ceil(n, case["page"]) for n in _page_lengths(case))


def _fork_parents(case):
    return [i % case["slots"] for i in range(case["children"])]


def _keep(case):
    """Whether each sequence of a compaction case is still there."""
    r = random.Random(case["pattern"] + 1)
    return [r.random() < 0.5 for _ in range(case["slots"])]


def work(case):
    if case["op"] == "moe":
        M, d, m, E, k = (case[x] for x in ("M", "d", "m", "E", "k"))
        touched = E * (1.0 - (1.0 - k / E) ** M)       # experts of M independent tokens
        per = (3 * m * d) // 2 + 4 * (2 * m * (d // 128) + d * (m // 64))
        route = 4 * M * E + 8 * M * k if case["logits"] else 8 * M * k
        return {"bytes": touched * per + 4 * M * d + route, "flops": 6.0 * M * k * m * d}
    if case["op"] == "attn":
        lens, sizes, shared = _attn_lengths(case)
        Hq, Hkv, D, nq = case["Hq"], case["Hkv"], case["D"], case["nq"]
        keys, pairs, i = 0, 0, 0
        for n, s in zip(sizes, shared):
            keys += s
            for L in lens[i:i + n]:
                keys += L - s
                pairs += nq * L - (nq * (nq - 1) // 2 if case["causal"] else 0)
            i += n
        return {"bytes": 4 * keys * Hkv * D + 4 * len(lens) * nq * Hq * D,
                "flops": 4.0 * pairs * Hq * D}
    lens = _page_lengths(case)
    page, row = case["page"], 2 * case["Hkv"] * case["D"] * 2 * case["layers"]
    if case["op"] == "admit":
        return {"bytes": 2 * sum(lens) * row + 4 * sum(_ceil(n, page) for n in lens), "flops": 0}
    if case["op"] == "fork":
        p = _fork_parents(case)
        return {"bytes": sum(2 * (lens[a] % page) * row + 8 * _ceil(lens[a], page) for a in p),
                "flops": 0}
    if case["op"] == "copy":
        return {"bytes": 2 * _copy_pairs(case) * page * row, "flops": 0}
    own_pages = [_ceil(n, page) for n in lens]
    live = sum(p for p, keep in zip(own_pages, _keep(case)) if keep)
    total = sum(own_pages)
    # of the live pages, those behind the first `live` pages of the pool move;
    # the pages lie at random, so about (1 - live / pool) of them
    moved = live * (1.0 - live / _pool_pages(case, total))
    return {"bytes": 2 * moved * page * row + 8 * total, "flops": 0}


def _pool_pages(case, used):
    return used + used // 8 + 8


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _packed(g, E, N, K, group, std):
    """A packed expert weight: 4-bit codes with a scale and zero per group."""
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        c = torch.randn((n, N, K // 2, 2), generator=g, device=DEV).mul_(2.6).add_(7.5)
        c = c.round_().clamp_(0, 15).to(torch.uint8)
        q[e:e + n] = c[..., 0] | (c[..., 1] << 4)
    sh = (E, N, K // group)
    s = (torch.rand(sh, generator=g, device=DEV) * 0.3 + 0.85) * (std / 2.6)
    z = torch.rand(sh, generator=g, device=DEV) + 7.0
    return q, s.half(), z.half()


def _prepare_moe(case, seed):
    g = _gen(seed)
    M, d, m, E, k = (case[x] for x in ("M", "d", "m", "E", "k"))
    st = {"case": case, "gu": _packed(g, E, 2 * m, d, 128, 0.02),
          "dn": _packed(g, E, d, m, 64, 0.02),
          "x": torch.randn((M, d), generator=g, device=DEV).to(torch.bfloat16),
          "logits": torch.randn((M, E), generator=g, device=DEV)}
    v, ids = st["logits"].topk(k, dim=1)
    st["ids"] = ids.to(torch.int32).contiguous()
    st["w"] = torch.softmax(v, dim=1).contiguous()
    if own:
        import w4a16_moe_expert_sync_gb300 as w4
        need = w4.w4_moe_layer_few_workspace_size(M, d, m, E, k)
        st["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return st


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _prepare_attn(case, seed):
    g = _gen(seed)
    r = random.Random(seed)
    lens, sizes, shared = _attn_lengths(case)
    page, Hq, Hkv, D, nq = (case[x] for x in ("page", "Hq", "Hkv", "D", "nq"))
    rows, used, copies, b = [], 0, [], 0
    for n, s in zip(sizes, shared):
        full = s // page
        first = list(range(used, used + full))
        used += full
        head = None
        for i in range(n):
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
    P = _pool_pages(case, used)
    perm = list(range(P))
    r.shuffle(perm)
    W = max(len(x) for x in rows) + 3
    table = _i32([[perm[p] for p in x] + [-1] * (W - len(x)) for x in rows])
    dt = DTYPES[case["dtype"]]
    cache = torch.empty((2, P, page, Hkv, D), dtype=dt, device=DEV)
    for c in cache.view(-1).split(1 << 26):
        c.copy_(torch.randn(c.shape, generator=g, device=DEV))
    for a, c, t in copies:
        cache[:, perm[c], :t] = cache[:, perm[a], :t]
    T = len(lens) * nq
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV)
    qkv[:, :Hq * D] *= 1.5
    qkv = qkv.to(dt)
    offs = [0]
    for n in sizes:
        offs.append(offs[-1] + n)
    st = {"case": case, "q": qkv[:, :Hq * D].view(T, Hq, D), "qkv": qkv, "k": cache[0],
          "v": cache[1], "table": table, "lens": _i32(lens),
          "q_offsets": _i32([i * nq for i in range(len(lens) + 1)]),
          "group_offsets": _i32(offs), "shared": _i32(shared), "lengths": lens}
    if own:
        import w4a16_moe_expert_sync_gb300 as w4
        need = w4.w4_attn_shared_prefix_workspace_size(T, len(lens), len(sizes), nq, Hq, Hkv, D)
        st["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return st


def _prepare_pages(case, seed):
    g = _gen(seed)
    r = random.Random(seed)
    lens = _page_lengths(case)
    op, page, Hkv, D = case["op"], case["page"], case["Hkv"], case["D"]
    need = [_ceil(n, page) for n in lens]
    used = sum(need)
    children = case["children"]
    P = _pool_pages(case, 2 * used if op == "copy" else used + children)
    perm = list(range(P))
    r.shuffle(perm)
    W = max(need) + 2
    B = len(lens) + children
    rows, at = [], 0
    for n in need:
        rows.append(perm[at:at + n] + [-1] * (W - n))
        at += n
    rows += [[-1] * W for _ in range(children)]
    lengths = lens + [0] * children
    gone = [not x for x in _keep(case)] if op == "compact" else [False] * len(lens)
    refs = [0] * P
    for i in range(len(lens)):
        if gone[i]:
            rows[i], lengths[i] = [-1] * W, 0
        for p in rows[i]:
            if p >= 0:
                refs[p] = 1
    cache = torch.empty((case["layers"], 2, P, page, Hkv, D), dtype=torch.bfloat16, device=DEV)
    for c in cache.view(-1).split(1 << 26):
        c.copy_(torch.randn(c.shape, generator=g, device=DEV))
    st = {"case": case, "cache": cache, "table": _i32(rows), "lens": _i32(lengths),
          "refs": _i32(refs), "slots": _i32(list(range(len(lens))))}
    if op == "admit":
        T = sum(lens)
        qkv = torch.randn((T, 4, Hkv, D), generator=g, device=DEV).to(torch.bfloat16)
        offs = [0]
        for n in lens:
            offs.append(offs[-1] + n)
        st.update(new_lens=_i32(lens), k=qkv[:, 2], v=qkv[:, 3], q_offsets=_i32(offs))
    if op == "fork":
        st.update(parents=_i32(_fork_parents(case)),
                  children=_i32(list(range(len(lens), len(lens) + children))))
    if op == "copy":
        n = _copy_pairs(case)
        st.update(src=_i32(perm[:n]), dst=_i32(perm[n:2 * n]))
    if op == "compact":
        st.update(table_out=torch.empty_like(st["table"]), refs_out=torch.empty_like(st["refs"]))
    if own and op in ("fork", "compact"):
        import w4a16_moe_expert_sync_gb300 as w4
        need = w4.w4_kv_workspace_size(P, max(children, 1))
        st["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return st


def prepare(case, seed):
    if case["op"] == "moe":
        return _prepare_moe(case, seed)
    if case["op"] == "attn":
        return _prepare_attn(case, seed)
    return _prepare_pages(case, seed)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(st):
    op = st["case"]["op"]
    return (_own if own else _plain)[op](st)


def _own_moe(st):
    import w4a16_moe_expert_sync_gb300 as w4
    if st["case"]["logits"]:
        return w4.w4_moe_layer_few_from_logits(st["x"], st["logits"], st["case"]["k"], st["gu"],
                                               st["dn"], workspace=st["ws"])
    return w4.w4_moe_layer_few(st["x"], st["ids"], st["w"], st["gu"], st["dn"],
                               workspace=st["ws"])


def _own_attn(st):
    import w4a16_moe_expert_sync_gb300 as w4
    return w4.w4_attn_shared_prefix(st["q"], st["k"], st["v"], st["table"], st["lens"],
                                    st["q_offsets"], st["group_offsets"], st["shared"],
                                    max_q=st["case"]["nq"], causal=st["case"]["causal"],
                                    workspace=st["ws"])


def _own_admit(st):
    import w4a16_moe_expert_sync_gb300 as w4
    w4.w4_kv_free(st["table"], st["lens"], st["refs"], st["slots"])
    w4.w4_kv_reserve(st["table"], st["lens"], st["refs"], st["slots"], st["new_lens"],
                     st["case"]["page"])
    w4.w4_kv_append(st["cache"][0, 0], st["cache"][0, 1], st["table"], st["lens"], st["k"],
                    st["v"], st["q_offsets"])
    return st["table"], st["lens"], st["refs"], st["cache"]


def _own_fork(st):
    import w4a16_moe_expert_sync_gb300 as w4
    w4.w4_kv_free(st["table"], st["lens"], st["refs"], st["children"])
    w4.w4_kv_fork(st["cache"], st["table"], st["lens"], st["refs"], st["parents"],
                  st["children"], workspace=st["ws"])
    return st["table"], st["lens"], st["refs"], st["cache"]


def _own_copy(st):
    import w4a16_moe_expert_sync_gb300 as w4
    w4.w4_kv_copy_pages(st["cache"], st["src"], st["dst"])
    return st["cache"]


def _own_compact(st):
    import w4a16_moe_expert_sync_gb300 as w4
    w4.w4_kv_compact(st["cache"], st["table"], st["refs"], table_out=st["table_out"],
                     refs_out=st["refs_out"], workspace=st["ws"])
    return st["table_out"], st["refs_out"], st["cache"]


_own = {"moe": _own_moe, "attn": _own_attn, "admit": _own_admit, "fork": _own_fork,
        "copy": _own_copy, "compact": _own_compact}


def _dequant(w, e, group):
    q, s, z = w[0][e], w[1][e].float(), w[2][e].float()
    c = torch.stack((q & 15, q >> 4), dim=-1).flatten(-2).float()
    return (c - z.repeat_interleave(group, -1)) * s.repeat_interleave(group, -1)


def _plain_moe(st):
    case = st["case"]
    k, m = case["k"], case["m"]
    if case["logits"]:
        order = torch.sort(st["logits"], dim=1, descending=True, stable=True)
        ids = order.indices[:, :k].to(torch.int32)
        p = torch.exp(order.values[:, :k] - order.values[:, :1])
        wts = p / p.sum(1, keepdim=True)
    else:
        ids, wts = st["ids"], st["w"]
    out = []
    for t in range(case["M"]):
        e = ids[t].long()
        x = st["x"][t].float()
        gu = (_dequant(st["gu"], e, 128) * x).sum(-1)
        gate, up = gu[:, :m], gu[:, m:]
        u = math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate ** 3)
        h = 0.5 * gate * (1.0 + torch.tanh(u)) * up
        y = (_dequant(st["dn"], e, 64) * h[:, None, :]).sum(-1)
        out.append((wts[t][:, None] * y).sum(0))
    out = torch.stack(out).to(torch.bfloat16)
    return (out, ids, wts) if case["logits"] else out


def _plain_attn(st):
    case = st["case"]
    page, nq, D = case["page"], case["nq"], case["D"]
    rep = case["Hq"] // case["Hkv"]
    out = torch.empty(st["q"].shape, dtype=st["q"].dtype, device=DEV)
    for b, L in enumerate(st["lengths"]):
        pages = st["table"][b, :_ceil(L, page)].long()
        k = st["k"][pages].flatten(0, 1)[:L].float()
        v = st["v"][pages].flatten(0, 1)[:L].float()
        q = st["q"][b * nq:(b + 1) * nq].float().unflatten(1, (case["Hkv"], rep))
        s = torch.einsum("thrd,lhd->hrtl", q, k) * (1.0 / math.sqrt(D))
        if case["causal"] and nq > 1:
            pos = torch.arange(L, device=DEV)
            last = torch.arange(L - nq, L, device=DEV)
            s = s.masked_fill(pos[None, :] > last[:, None], float("-inf"))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = torch.einsum("hrtl,lhd->thrd", p, v)
        o = o / p.sum(-1).permute(2, 0, 1)[..., None]
        out[b * nq:(b + 1) * nq] = o.flatten(1, 2).to(out.dtype)
    return out


def _plain_release(st, slots):
    rows = st["table"][slots]
    held = rows[rows >= 0].long()
    st["refs"].scatter_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    st["table"][slots] = -1
    st["lens"][slots] = 0


def _plain_admit(st):
    page = st["case"]["page"]
    slots = st["slots"].long()
    _plain_release(st, slots)
    need = (st["new_lens"] + page - 1) // page
    W = st["table"].shape[1]
    hole = torch.arange(W, device=DEV)[None, :] < need[:, None]
    free = torch.nonzero(st["refs"] == 0).flatten()
    rows = torch.full((len(slots), W), -1, dtype=torch.int32, device=DEV)
    rank = torch.cumsum(hole.flatten(), 0).view(hole.shape) - 1
    rows = torch.where(hole, free[rank.clamp(min=0)].to(torch.int32), rows)
    st["table"][slots] = rows
    st["refs"][rows[hole].long()] = 1
    st["lens"][slots] = st["new_lens"]
    start = st["q_offsets"][:-1].long()
    t = torch.arange(st["k"].shape[0], device=DEV)
    seq = torch.searchsorted(st["q_offsets"][1:].long(), t, right=True)
    pos = t - start[seq] + (st["lens"].long()[seq] - (st["q_offsets"][1:].long() - start)[seq])
    at = st["table"][seq, pos // page].long()
    st["cache"][0, 0][at, pos % page] = st["k"]
    st["cache"][0, 1][at, pos % page] = st["v"]
    return st["table"], st["lens"], st["refs"], st["cache"]


def _plain_fork(st):
    page = st["case"]["page"]
    parents, children = st["parents"].long(), st["children"].long()
    _plain_release(st, children)
    n = st["lens"][parents].long()
    full, tail = n // page, n % page
    W = st["table"].shape[1]
    col = torch.arange(W, device=DEV)[None, :]
    rows = torch.where(col < full[:, None], st["table"][parents], -1)
    shared = rows[rows >= 0].long()
    st["refs"].scatter_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    free = torch.nonzero(st["refs"] == 0).flatten()
    new = free[(torch.cumsum(tail > 0, 0) - 1).clamp(min=0)]
    cut = torch.nonzero(tail > 0).flatten()
    old = st["table"][parents[cut], full[cut]].long()
    rows[cut, full[cut]] = new[cut].to(torch.int32)
    st["refs"][new[cut]] = 1
    st["table"][children] = rows
    st["lens"][children] = n.to(torch.int32)
    held = torch.arange(page, device=DEV)[None, :] < tail[cut][:, None]
    i, j = torch.nonzero(held, as_tuple=True)
    for layer in st["cache"]:
        layer[:, new[cut][i], j] = layer[:, old[i], j]
    return st["table"], st["lens"], st["refs"], st["cache"]


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    for layer in st["cache"]:
        layer[:, dst] = layer[:, src]
    return st["cache"]


def _plain_compact(st):
    refs = st["refs"]
    P = refs.numel()
    live = (refs > 0).sum()
    at = torch.arange(P, device=DEV)
    dst = at[(refs == 0) & (at < live)]
    src = at[(refs > 0) & (at >= live)]
    move = at.clone()
    move[src] = dst
    held = st["table"] >= 0
    st["table_out"].copy_(torch.where(held, move[st["table"].clamp(min=0).long()].to(torch.int32),
                                      st["table"]))
    st["refs_out"].copy_(refs)
    st["refs_out"][dst] = refs[src]
    st["refs_out"][src] = 0
    for layer in st["cache"]:
        layer[:, dst] = layer[:, src]
    return st["table_out"], st["refs_out"], st["cache"]


_plain = {"moe": _plain_moe, "attn": _plain_attn, "admit": _plain_admit, "fork": _plain_fork,
          "copy": _plain_copy, "compact": _plain_compact}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "moe":
        return _exact_moe(case, seed)
    if case["op"] == "attn":
        return _exact_attn(case, seed)
    return None                                  # pages are moved, nothing is computed


def _exact_weight(w, e, group):
    lo, hi = (w[0][e] & 15).double(), (w[0][e] >> 4).double()
    full = torch.empty((lo.shape[0], 2 * lo.shape[1]), dtype=torch.float64, device=DEV)
    full[:, 0::2], full[:, 1::2] = lo, hi
    full = full.view(lo.shape[0], -1, group)
    return ((full - w[2][e].double()[..., None]) * w[1][e].double()[..., None]).flatten(1)


def _exact_moe(case, seed):
    st = _prepare_moe(case, seed)
    M, k, m = case["M"], case["k"], case["m"]
    if case["logits"]:
        l = st["logits"].double().cpu()
        ids = torch.empty((M, k), dtype=torch.int32)
        for t in range(M):
            row = l[t].tolist()
            ids[t] = torch.tensor(sorted(range(len(row)), key=lambda e: (-row[e], e))[:k])
        top = torch.gather(l, 1, ids.long())
        wts = torch.softmax(top, dim=1).to(DEV)
        ids = ids.to(DEV)
    else:
        ids, wts = st["ids"], st["w"].double()
    out = torch.zeros((M, case["d"]), dtype=torch.float64, device=DEV)
    x = st["x"].double()
    for e in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        g = x[t] @ _exact_weight(st["gu"], e, 128).T
        h = torch.nn.functional.gelu(g[:, :m], approximate="tanh") * g[:, m:]
        out.index_add_(0, t, wts[t, j][:, None] * (h @ _exact_weight(st["dn"], e, 64).T))
    return (out, ids, wts) if case["logits"] else out


def _exact_attn(case, seed):
    st = _prepare_attn(case, seed)
    page, nq, D, Hkv = case["page"], case["nq"], case["D"], case["Hkv"]
    rep = case["Hq"] // Hkv
    if sum(st["lengths"]) * nq * case["Hq"] * D > 4e12:
        return None
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    for b, L in enumerate(st["lengths"]):
        at = torch.arange(L, device=DEV)
        where = st["table"][b].long()[at // page] * page + at % page
        lim = torch.full((nq,), L, device=DEV)
        if case["causal"]:
            lim = L - nq + 1 + torch.arange(nq, device=DEV)
        seen = (at[None, :] < lim[:, None]).repeat_interleave(rep, 0)
        for h in range(Hkv):
            k = st["k"].flatten(0, 1)[where, h].double()
            v = st["v"].flatten(0, 1)[where, h].double()
            q = st["q"][b * nq:(b + 1) * nq, h * rep:(h + 1) * rep].double().reshape(-1, D)
            s = torch.where(seen, (q @ k.T) / D ** 0.5, -torch.inf)
            o = torch.softmax(s, dim=1) @ v
            out[b * nq:(b + 1) * nq, h * rep:(h + 1) * rep] = o.view(nq, rep, D)
    return out
