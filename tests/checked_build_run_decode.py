"""Runs the decoding step's operators with the library given on the command line (the
W4_CHECK_BOUNDS build) and saves their results and status words to an .npz: a child
process of test_gpu_check_bounds_decode.py, which runs the normal build itself."""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def run(lib_path, out_path):
    import torch
    import w4a16_moe_expert_sync_gb300 as w4
    w4.load_library(lib_path)
    from test_gpu_attention import CASES, _build, _run
    from test_gpu_few import _inputs
    res, words = {}, {}

    def status(name):
        words[name] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return words[name]

    def keep(name, t):
        res[name] = t.view(torch.int16).cpu().numpy() if t.element_size() == 2 else t.cpu().numpy()

    for M, d, m, E, k in [(1, 256, 128, 8, 2), (17, 384, 192, 12, 8), (3, 6144, 64, 4, 2),
                          (32, 2816, 704, 16, 8)]:
        x, logits, gu, dn = _inputs(M, d, m, E, k)
        name = f"few_{M}_{d}"
        out, ids, w = w4.w4_moe_layer_few_from_logits(x, logits, k, gu, dn, dev_status=status(name))
        keep(name, out)
        keep(name + "_ids", ids)
        keep(name + "_w", w)
        ids[0, 0] = E                                    # one that is none
        keep(name + "_bad", w4.w4_moe_layer_few(x, ids, w, gu, dn, dev_status=status(name + "_bad")))
    for i, case in enumerate(CASES):
        *shape, causal = case
        c = _build(*shape, seed=len(shape[0]))
        keep(f"attn_{i}", _run(w4, c, causal, dev_status=status(f"attn_{i}")))

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for page, P, W in ((4, 40, 12), (16, 3000, 200)):
        name = f"kv_{page}"
        st = status(name)
        pool = torch.randn((2, 2, P, page, 2, 16), generator=g, device="cuda").bfloat16()
        table, lens = torch.full((6, W), -1, dtype=torch.int32, device="cuda"), ints([0] * 6)
        refs = torch.zeros(P, dtype=torch.int32, device="cuda")
        state = (table, lens, refs)
        n = [page * W // 2 - 1, page * 3, 2, 0, 0, 0]
        w4.w4_kv_reserve(*state, ints([2, 0, 1]), ints([n[2], n[0], n[1]]), page, dev_status=st)
        kv = torch.randn((n[0] + 5, 2, 2, 16), generator=g, device="cuda").bfloat16()
        w4.w4_kv_append(pool[0, 0], pool[0, 1], table, lens, kv[:, 0], kv[:, 1],
                        ints([0, n[0], n[0] + 3, n[0] + 5, n[0] + 5, n[0] + 5, n[0] + 5]),
                        dev_status=st)
        w4.w4_kv_fork(pool, *state, ints([0, 0, 2]), ints([3, 4, 5]), dev_status=st)
        w4.w4_kv_free(*state, ints([0, 2]), dev_status=st)
        w4.w4_kv_reserve(*state, ints([5, 0, 3]), ints([page * 2, page * W, n[0] + 2]), page,
                         dev_status=st)                  # the small pool runs out
        w4.w4_kv_copy_pages(pool, table[3, :2].contiguous(), ints([P - 1, P - 2]), dev_status=st)
        for slots in ([3], [1]):
            w4.w4_kv_free(*state, ints(slots), dev_status=st)
            w4.w4_kv_compact(pool, table, refs, dev_status=st)
        for what, t in (("pool", pool), ("table", table), ("lens", lens), ("refs", refs)):
            keep(f"{name}_{what}", t)
    torch.cuda.synchronize()
    res["status_names"] = np.array(list(words))
    res["status"] = np.array([int(t) for t in words.values()])
    np.savez(out_path, **res)


if __name__ == "__main__":
    run(sys.argv[1], sys.argv[2])
