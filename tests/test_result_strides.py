"""Results of the rotation whose tokens and heads share memory are refused, by the library
and by the binding, and no others are: csrc/strides.h against every pair of rows."""
import ctypes
import itertools
import os
import random
import shutil
import subprocess

import pytest

import w4a16_moe_expert_sync_gb300 as w4
from w4a16_moe_expert_sync_gb300 import build

AT = 0x10000                                   # an address that nobody reads
# (tokens, heads, strides of tokens and heads) of rows of 64
OVERLAPPING = [(2, 2, 64, 64), (4, 2, 64, 64), (3, 3, 128, 64), (4, 3, 128, 64), (4, 2, 64, 128),
               (5, 4, 256, 64 + 8), (2, 2, -64, 64), (5, 4, 192, 256), (4, 5, 256, 192)]
APART = [(2, 2, 128, 64), (2, 3, 64, 128), (4, 2, 64, 256), (2, 2, 192, 128), (2, 2, 128, 192),
         (3, 2, 128, 320), (2, 3, 192, 128), (1, 3, 0, 64), (3, 1, 64, 0), (3, 3, -192, 64),
         (4, 3, 192, 128), (3, 4, 128, 192)]


def _refused(rc):
    return rc == 1 and b"overlap" in w4.load_library().w4_last_error_detail()


def _rope(T, H, tok, head, of_keys):
    far = (1 << 20, 64)
    q_out, k_out = (far, (tok, head)) if of_keys else ((tok, head), far)
    return w4.load_library().w4_qk_norm_rope(
        AT, 1 << 20, 64, AT, 1 << 20, 64, AT, AT, None, None, T, H, H, 64, 64, 0, 0, 1e-6, 1.0, AT,
        *q_out, AT, *k_out, None)


def _append(T, H, tok, head):
    return w4.load_library().w4_kv_append_rope(
        AT, AT, 2048, 128, 64, 8, 16, AT, 1, 4, AT, AT, 1 << 20, 64, AT, 128, 64, AT, 128, 64, AT,
        None, AT, None, None, T, H, 2, 64, 64, 0, 0, ctypes.c_float(1e-6), ctypes.c_float(1.0), AT,
        tok, head, None, None)


@pytest.mark.parametrize("T,H,tok,head", OVERLAPPING)
def test_the_library_refuses_them(T, H, tok, head):
    assert _refused(_rope(T, H, tok, head, False))
    assert _refused(_rope(T, H, tok, head, True))
    assert _refused(_append(T, H, tok, head))


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("strides")
    (d / "s.cpp").write_text('#include "strides.h"\nextern "C" int overlap(long long T, long long H, '
                             'long long D, long long a, long long b)\n'
                             '{ return w4::rows_overlap(T, H, D, a, b); }\n')
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC,
                    str(d / "s.cpp"), "-o", str(d / "s.so")], check=True)
    f = ctypes.CDLL(str(d / "s.so")).overlap
    f.argtypes = [ctypes.c_longlong] * 5
    return f


def _by_pairs(T, H, D, tok, head):
    at = [t * tok + h * head for t in range(T) for h in range(H)]
    return any(abs(a - b) < D for a, b in itertools.combinations(at, 2))


def test_against_every_pair_of_rows(overlap):
    for case in OVERLAPPING:
        assert overlap(*case[:2], 64, *case[2:]) and _by_pairs(*case[:2], 64, *case[2:]), case
    for case in APART:
        assert not overlap(*case[:2], 64, *case[2:]) and not _by_pairs(*case[:2], 64, *case[2:]), case
    r = random.Random(1)
    found = [0, 0]
    for _ in range(20000):
        T, H, D = r.randint(0, 6), r.randint(0, 6), r.choice([1, 3, 8])
        a, b = (r.choice([1, 1, -1]) * r.randint(0, r.choice([9, 30, 60])) for _ in range(2))
        want = _by_pairs(T, H, D, a, b)
        assert bool(overlap(T, H, D, a, b)) == want, (T, H, D, a, b)
        found[want] += 1
    assert min(found) > 2000
    # large ones are answered without a comparison of rows
    assert not overlap(2 ** 31 - 1, 65535, 256, 65535 * 256, 256)
    assert not overlap(2 ** 31 - 1, 65535, 256, 256, (2 ** 31 - 1) * 256)


@pytest.mark.gpu
def test_the_binding_refuses_them(lib):
    import torch
    from test_gpu_rope import _inputs, _sequences
    for T, H, tok, head in OVERLAPPING:
        if tok < 0:
            continue                           # no tensor has such strides
        q, k, v, _ = _inputs(T, H, H, 64, "bfloat16", 3)
        pos, steps = torch.zeros(T, dtype=torch.int32, device="cuda"), lib.w4_rope_steps(64)
        bad = torch.zeros(1 << 14, dtype=torch.bfloat16, device="cuda").as_strided((T, H, 64),
                                                                                   (tok, head, 1))
        c = _sequences([T], [0], 16, H, 64, "bfloat16", 1)
        for call in (lambda: lib.w4_qk_norm_rope(q, k, pos, steps, q_out=bad),
                     lambda: lib.w4_qk_norm_rope(q, k, pos, steps, k_out=bad),
                     lambda: lib.w4_kv_append_rope(c["kp"], c["vp"], c["table"], c["lens"], q, k, v,
                                                   c["q_offsets"], steps, q_out=bad)):
            with pytest.raises(ValueError, match="overlap"):
                call()


@pytest.mark.gpu
def test_rows_apart_are_taken(lib):
    import torch
    from test_gpu_rope import _inputs
    for T, H, tok, head in APART:
        if tok < 0:
            continue
        q, k, _, _ = _inputs(T, H, H, 64, "bfloat16", 4)
        pos, steps = torch.arange(T, dtype=torch.int32, device="cuda"), lib.w4_rope_steps(64)
        want = lib.w4_qk_norm_rope(q, k, pos, steps)
        outs = [torch.zeros(1 << 14, dtype=torch.bfloat16, device="cuda").as_strided((T, H, 64),
                                                                                     (tok, head, 1))
                for _ in range(2)]
        lib.w4_qk_norm_rope(q, k, pos, steps, q_out=outs[0], k_out=outs[1])
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
