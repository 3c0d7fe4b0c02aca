"""A pool whose pages lie past 2^31 elements (and 2^32 bytes) from its start:
the cache's operations and attention address them in 64 bits."""
import pytest


@pytest.mark.gpu
def test_pages_past_32_bit_offsets(lib):
    import torch
    P, page, Hkv, D, Hq = 36000, 64, 8, 128, 16
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs a pool of 9.4 GB")
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = torch.empty((2, P, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    assert pool[0].numel() > 1 << 31
    table = torch.full((4, 8), -1, **i32)
    lens, refs, st = (torch.zeros(n, **i32) for n in (4, P, 1))
    refs[:P - 40] = 1                        # only the last pages are free
    slots = torch.tensor([0, 1], **i32)
    new = torch.tensor([200, 130], **i32)
    lib.w4_kv_reserve(table, lens, refs, slots, new, page, dev_status=st)
    assert table[0, :4].tolist() == [P - 40, P - 39, P - 38, P - 37]
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn((330, Hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    offs = torch.tensor([0, 200, 330], **i32)
    lib.w4_kv_append(pool[0], pool[1], table, lens, k, v, offs, dev_status=st)
    lib.w4_kv_fork(pool, table, lens, refs, torch.tensor([0], **i32), torch.tensor([2], **i32),
                   dev_status=st)
    for p, x in ((pool[0], k), (pool[1], v)):
        for slot, lo, n in ((0, 0, 200), (1, 200, 130), (2, 0, 200)):
            ids = table[slot, :-(-n // page)].long()
            assert torch.equal(p[ids].flatten(0, 1)[:n], x[lo:lo + n])
    q = torch.randn((3, Hq, D), generator=g, device="cuda").bfloat16()
    out = lib.w4_attn_shared_prefix(q, pool[0], pool[1], table, lens,
                                    torch.tensor([0, 1, 2, 3], **i32), dev_status=st)
    for b, (lo, n) in enumerate(((0, 200), (200, 130), (0, 200))):
        kk, vv = (x[lo:lo + n].double().repeat_interleave(2, 1) for x in (k, v))
        p = torch.softmax(torch.einsum("hd,lhd->hl", q[b].double(), kk) * D ** -0.5, 1)
        ref, A = (torch.einsum("hl,lhd->hd", p, x) for x in (vv, vv.abs()))
        # the result's rounding, the weights' and fp32 sums
        assert bool(((out[b].double() - ref).abs()
                     <= 2.0 ** -8 * (ref.abs() + A) * (1 + 2.0 ** -6) + 2.0 ** -14 * A).all())
    src, dst = table[0, :2].clone(), torch.tensor([P - 3, P - 2], **i32)
    lib.w4_kv_copy_pages(pool, src, dst, dev_status=st)
    # as bits: what no token filled may be NaN
    bits = pool.view(torch.int16)
    assert torch.equal(bits[:, dst.long()], bits[:, src.long()])
    refs[:P - 40] = 0                        # the rest leaves: the last pages move to the front
    before = bits[:, table[1, :3].long()].clone()
    lib.w4_kv_compact(pool, table, refs, dev_status=st)
    assert int(table.max()) < 10 and torch.equal(bits[:, table[1, :3].long()], before)
    assert int(st) == 0
