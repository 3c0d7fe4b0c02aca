"""Runs the verifying step's operators with the library given on the command line (the
W4_CHECK_BOUNDS build) and saves their results and status words to an .npz: a child
process of test_gpu_check_bounds_verify.py, which runs the normal build itself."""
import os
import random
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def run(lib_path, out_path):
    import torch
    import w4a16_moe_expert_sync_gb300 as w4
    w4.load_library(lib_path)
    import test_gpu_attn_tree as trees
    import test_gpu_kv_keep as keeping
    import test_gpu_linear_few as linear
    import test_gpu_rope as rope
    res, words = {}, {}

    def status(name):
        words[name] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return words[name]

    def keep(name, t):
        res[name] = t.view(torch.int16).cpu().numpy() if t.element_size() == 2 else t.cpu().numpy()

    for M, K, N, group in [(1, 384, 4097, 128), (11, 704, 2815, 64), (13, 2816, 39041, 128),
                           (32, 2816, 40000, 128)]:
        name = f"linear_{M}"
        x, q, s, z = linear._inputs(M, K, N, group, M)
        keep(name, w4.w4_w4a16_linear_few(x, q, s, z, group, dev_status=status(name)))
    for i, case in enumerate(trees.CASES):
        befores, nodes, *shape = case
        r = random.Random(i)
        c = trees._build([a + n for a, n in zip(befores, nodes)], nodes, *shape, seed=i)
        tree = trees._words([b for n in nodes if n for b in trees._random_tree(r, n)],
                            -(-max(nodes) // 32))
        keep(f"tree_{i}", trees._run(w4, c, tree, dev_status=status(f"tree_{i}")))
    for i, (news, befores, page, bad) in enumerate([([3, 0, 40, 1], [0, 9, 30, 63], 16, False),
                                                    ([12] * 70, list(range(70)), 32, True)]):
        name = f"append_{i}"
        T = sum(news)
        q, k, v, (wq, wk) = rope._inputs(T, 6, 2, 128, "bfloat16", T)
        c = rope._sequences(news, befores, page, 2, 128, "bfloat16", T)
        if bad:                                          # pages and lengths that are none
            c["table"][5, 0], c["table"][6, 0], c["lens"][7] = -1, 1 << 30, 3
        keep(name, w4.w4_kv_append_rope(c["kp"], c["vp"], c["table"], c["lens"], q, k, v,
                                        c["q_offsets"], w4.w4_rope_steps(128), q_weight=wq,
                                        k_weight=wk, dev_status=status(name)))
        keep(name + "_pool", c["pool"])
    for i, (befores, news, bad) in enumerate([([40, 3, 7, 100], [25, 2, 64, 30], False),
                                              ([7] * 90, [33] * 90, True)]):
        name = f"keep_{i}"
        r = random.Random(i)
        c = keeping._build(befores, news, [sorted(r.sample(range(n), r.randint(0, n))) for n in news],
                           3, 16, 2, 64, i)
        if bad:
            c["table"][4, 1], c["table"][5, 2], c["kept_offsets"][9] = 1 << 30, -7, 1 << 29
        keep(name, keeping._call(w4, c, dev_status=status(name)))
        keep(name + "_pool", c["pool"])
    torch.cuda.synchronize()
    res["status_names"] = np.array(list(words))
    res["status"] = np.array([int(t) for t in words.values()])
    np.savez(out_path, **res)


if __name__ == "__main__":
    run(sys.argv[1], sys.argv[2])
