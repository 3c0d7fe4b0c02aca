"""fp16 attention where one key outweighs all others by far: the weights' small end.

Tolerance, derived beforehand, as in test_gpu_attention.py (u = 2^-11, A = sum_l p_l
|v_l|: u (|ref| + A) for the weights' and the result's rounding, 2^-14 A for fp32),
with the absolute term of weights below fp16's normal range: they are rounded to
multiples of 2^-24 of a weight of at least 2^7, so each is off by at most 2^-32 of the
largest: 2^-32 sum_l |v_l| in all, with the denominator at least that largest weight."""
import pytest

pytestmark = pytest.mark.gpu


def _cache(lens, page, Hkv, D, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need) + 2
    perm = torch.randperm(P, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return torch.zeros((2, P, page, Hkv, D), device="cuda"), table


def _put(cache, table, b, pos, k, v):
    page = cache.shape[2]
    where = table[b, pos // page].long()
    cache[0, where, pos % page] = k
    cache[1, where, pos % page] = v


@pytest.mark.parametrize("n,page,D", [(3000, 64, 128), (120000, 64, 64), (40000, 16, 128)])
@pytest.mark.parametrize("sink", ["first", "middle", "last"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("nats", [6.0, 12.0, 18.0])
def test_a_key_that_outweighs_the_rest(lib, n, page, D, sink, shared, nats):
    import torch
    g = torch.Generator(device="cuda").manual_seed(n)
    B, Hq, Hkv = 2, 4, 2
    lens = [n, n + 5]
    cache, table = _cache(lens, page, Hkv, D, n)
    if shared:
        table[1, :n // page] = table[0, :n // page]
    for b, L in enumerate(lens):
        pos = torch.arange(L, device="cuda")
        if shared and b:
            pos = pos[n // page * page:]
        k = torch.zeros((len(pos), Hkv, D), device="cuda")
        k[..., 0] = torch.rand((len(pos), Hkv), generator=g, device="cuda")
        v = torch.rand((len(pos), Hkv, D), generator=g, device="cuda") + 0.5
        _put(cache, table, b, pos, k, v)
    if shared:                               # the tokens before the last page's end are alike
        part = n - n // page * page
        cache[:, table[1, n // page].long(), :part] = cache[:, table[0, n // page].long(), :part]
    for b in range(B):
        at = torch.tensor([{"first": 0, "middle": n // 2, "last": n - 1}[sink]], device="cuda")
        k = torch.zeros((1, Hkv, D), device="cuda")
        k[..., 0] = nats + 1.0
        _put(cache, table, b, at, k, torch.zeros((1, Hkv, D), device="cuda"))
    cache = cache.half()
    q = torch.zeros((B, Hq, D), device="cuda")
    q[..., 0] = D ** 0.5                     # a key's score is its first value
    q = q.half()
    ints = dict(dtype=torch.int32, device="cuda")
    kw = dict(group_offsets=torch.tensor([0, 2], **ints),
              shared_lens=torch.tensor([n], **ints)) if shared else {}
    got = lib.w4_attn_shared_prefix(q, cache[0], cache[1], table, torch.tensor(lens, **ints),
                                    torch.tensor([0, 1, 2], **ints), **kw).double()
    for b, L in enumerate(lens):
        ids = table[b, :-(-L // page)].long()
        k, v = (c[ids].flatten(0, 1)[:L].double().repeat_interleave(Hq // Hkv, 1) for c in cache)
        s = torch.einsum("hd,lhd->hl", q[b].double(), k) * D ** -0.5
        p = torch.softmax(s, 1)
        ref = torch.einsum("hl,lhd->hd", p, v)
        A, small = torch.einsum("hl,lhd->hd", p, v.abs()), v.abs().sum(0)
        tol = 2.0 ** -11 * (ref.abs() + A) * (1 + 2.0 ** -6) + 2.0 ** -14 * A + 2.0 ** -32 * small
        assert bool(((got[b] - ref).abs() <= tol).all())
