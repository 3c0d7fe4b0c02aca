"""With their outputs and workspaces given, the decoding step's operators allocate
nothing: neither from torch's pool nor on the device."""
import pytest

pytestmark = pytest.mark.gpu


def test_nothing_is_allocated(lib):
    import torch
    from test_gpu_attention import _build
    from test_gpu_few import _inputs
    M, d, m, E, k = 6, 384, 192, 12, 3
    x, logits, gu, dn = _inputs(M, d, m, E, k, seed=4)
    ids, w = lib.w4_moe_route(logits, k)
    out = torch.empty_like(x)
    ws = torch.empty(lib.w4_moe_layer_few_workspace_size(M, d, m, E, k), dtype=torch.uint8,
                     device="cuda")
    c = _build([450, 500, 470], [2, 1, 3], [3], [430], 8, 4, 128, 32, "bfloat16", seed=4)
    att_out = torch.empty_like(c["q"])
    att_ws = torch.empty(lib.w4_attn_shared_prefix_workspace_size(6, 3, 1, 3, 8, 4, 128),
                         dtype=torch.uint8, device="cuda")
    ints = dict(dtype=torch.int32, device="cuda")
    pool = torch.randn((2, 2, 40, 8, 2, 16), device="cuda").bfloat16()
    table, refs, lens = torch.full((4, 8), -1, **ints), torch.zeros(40, **ints), torch.zeros(4, **ints)
    one, n, two = (torch.tensor([i], **ints) for i in (0, 29, 2))
    both, pages = torch.tensor([0, 2], **ints), torch.tensor([30, 31], **ints)
    first = torch.tensor([0, 1], **ints)
    kv = torch.randn((29, 2, 2, 16), device="cuda").bfloat16()
    k_rows, v_rows, kp, vp = kv[:, 0], kv[:, 1], pool[0, 0], pool[0, 1]
    offs, row, row_len = torch.tensor([0, 29], **ints), table[:1], lens[:1]
    kv_ws = torch.empty(lib.w4_kv_workspace_size(40, 2), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, **ints)

    def step():
        lib.w4_moe_layer_few(x, ids, w, gu, dn, workspace=ws, out=out, dev_status=st)
        lib.w4_moe_layer_few_from_logits(x, logits, k, gu, dn, workspace=ws, out=out, ids=ids,
                                         weights=w, dev_status=st)
        lib.w4_attn_shared_prefix(c["q"], c["cache"][0], c["cache"][1], c["table"], c["lens"],
                                  c["q_offsets"], c["group_offsets"], c["shared"], max_q=3,
                                  workspace=att_ws, out=att_out, dev_status=st)
        lib.w4_kv_reserve(table, lens, refs, one, n, 8, dev_status=st)
        lib.w4_kv_append(kp, vp, row, row_len, k_rows, v_rows, offs, dev_status=st)
        lib.w4_kv_fork(pool, table, lens, refs, one, two, workspace=kv_ws, dev_status=st)
        lib.w4_kv_copy_pages(pool, first, pages, dev_status=st)
        lib.w4_kv_compact(pool, table, refs, workspace=kv_ws, dev_status=st)
        lib.w4_kv_free(table, lens, refs, both, dev_status=st)
    step()
    torch.cuda.synchronize()
    count = torch.cuda.memory_stats()["allocation.all.allocated"]
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        step()
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == count
    torch.cuda.synchronize()
    # (what little another process may take apart)
    assert free - torch.cuda.mem_get_info()[0] < 1 << 20
    assert int(st) == 0
