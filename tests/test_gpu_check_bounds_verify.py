"""The W4_CHECK_BOUNDS build on the verifying step's operators (the tokens' places in
their pages, where kept ones go, the trees' pieces and output): no check fails, whatever
tables, lengths and lists say, and the results are the normal build's bit for bit."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def test_checked_build_matches_and_finds_nothing(lib, tmp_path):
    from w4a16_moe_expert_sync_gb300 import build
    checked = build.build_checked(str(tmp_path))
    here = os.path.dirname(os.path.abspath(__file__))
    out, ref = str(tmp_path / "checked.npz"), str(tmp_path / "normal.npz")
    r = subprocess.run([sys.executable, os.path.join(here, "checked_build_run_verify.py"), checked,
                        out], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    import checked_build_run_verify
    checked_build_run_verify.run(build.LIB, ref)
    got, want = np.load(out), np.load(ref)
    for name, word in zip(got["status_names"], got["status"]):
        assert not word & lib.W4_DEV_OUT_OF_BOUNDS, (name, word)
        if name in ("append_1", "keep_1"):
            assert word & (lib.W4_DEV_BAD_PAGE | lib.W4_DEV_BAD_SLOT), name
        else:
            assert word == 0, (name, word)
    assert sorted(got.files) == sorted(want.files)
    for name in want.files:
        assert np.array_equal(got[name], want[name]), name


def test_the_operators_check_their_stores():
    from w4a16_moe_expert_sync_gb300 import build
    for name, least in (("rope.cu", 1), ("kv.cu", 9)):
        with open(os.path.join(build.CSRC, name)) as f:
            assert f.read().count("W4_IN_BOUNDS(") >= least, name
