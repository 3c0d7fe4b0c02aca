"""Runs the few-token linear with the library given on the command line (the W4_CHECK_BOUNDS
build) and saves its results and status words to an .npz: a child process of
test_gpu_check_bounds_linear.py, which runs the normal build itself."""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

# (tokens, K, rows, group): odd rows and single ones, a unit of one group of 64, tasks that
# cross warps, each layout of the activations, and the path for many rows with 16 and 32
# tokens, in parts, with groups of 128 and of 64
CASES = [(1, 128, 1, 128), (2, 64, 3, 64), (1, 384, 4097, 128), (11, 704, 2815, 64),
         (8, 640, 5001, 128), (31, 8192, 130, 64), (17, 11264, 9999, 128), (9, 5632, 9728, 64),
         (13, 2816, 39041, 128), (32, 2816, 40000, 128), (30, 5632, 38913, 128),
         (12, 1024, 77825, 64), (27, 2816, 38915, 64), (32, 5760, 19459, 64)]


def run(lib_path, out_path):
    import torch
    import w4a16_moe_expert_sync_gb300 as w4
    w4.load_library(lib_path)
    from test_gpu_linear_few import _inputs
    res, words = {}, []
    for i, (M, K, N, group) in enumerate(CASES):
        x, q, s, z = _inputs(M, K, N, group, i)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = w4.w4_w4a16_linear_few(x, q, s, z, group, dev_status=status)
        res[f"y_{i}"] = y.view(torch.int16).cpu().numpy()
        words.append(int(status))
    res["status"] = np.array(words)
    np.savez(out_path, **res)


if __name__ == "__main__":
    run(sys.argv[1], sys.argv[2])
