"""The W4_CHECK_BOUNDS build on the few-token linear (results, staged activations, the
places of scales): no check fails, and the results are the normal build's bit for bit."""
import os
import subprocess
import sys

import numpy as np
import pytest


@pytest.mark.gpu
def test_checked_build_matches_and_finds_nothing(lib, tmp_path):
    from w4a16_moe_expert_sync_gb300 import build
    checked = build.build_checked(str(tmp_path))
    here = os.path.dirname(os.path.abspath(__file__))
    out, ref = str(tmp_path / "checked.npz"), str(tmp_path / "normal.npz")
    r = subprocess.run([sys.executable, os.path.join(here, "checked_build_run_linear.py"), checked,
                        out], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    import checked_build_run_linear
    checked_build_run_linear.run(build.LIB, ref)
    got, want = np.load(out), np.load(ref)
    assert sorted(got.files) == sorted(want.files)
    assert not got["status"].any(), list(zip(checked_build_run_linear.CASES, got["status"]))
    for name in want.files:
        assert np.array_equal(got[name], want[name]), name


def test_the_kernels_check_their_stores():
    from w4a16_moe_expert_sync_gb300 import build
    for name, least in (("linear_few.cu", 4), ("linear_few_wide.cu", 4)):
        with open(os.path.join(build.CSRC, name)) as f:
            text = f.read()
        assert text.count("W4_IN_BOUNDS(") >= least and '#include "checks.cuh"' in text, name
