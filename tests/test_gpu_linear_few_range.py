"""w4_w4a16_linear_few at the ends of the activations' range, on both of its paths.

Up to 2^57 results are as test_gpu_linear_few.py says (its tolerance).  Beyond, an output
is that or not finite, and never finite and wrong: scaled activations, sums of activations
and a group's sum before its scale may leave fp32's range.  Downwards the tensor-memory
path loses nothing.  The other one holds a group's sums times 2^-63, so fp32's steps of
2^-149 are steps of 2^-86: at most half of one for each of a group's 8 MMAs and, times the
zero (below 16), for its activations' sum, and once more with the scale (below 1) for the
sum of all groups: together (8 / 2 + 16 / 2 + 1 / 2) 2^-86 a group."""
import math

import pytest

pytestmark = pytest.mark.gpu

MAX = 2.0 ** 127 * (2 - 2.0 ** -7)             # bf16's largest value
LARGE = [2.0 ** 58, 2.0 ** 61, 2.0 ** 90, 2.0 ** 125, 2.0 ** 126, 1.75 * 2.0 ** 126, 2.0 ** 127, MAX,
         -MAX]
# (tokens, K, rows, group): the path for many rows and the other one
SHAPES = [(12, 1024, 39000, 128), (30, 1024, 39000, 128), (12, 2816, 38912, 64), (30, 384, 300, 128),
          (12, 320, 300, 64)]


def _expect(x, q, s, z, group):
    from test_gpu_linear_few import _reference
    ref, S = _reference(x, q, s, z, group)
    return ref, 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + 2.0 ** -15 * S


@pytest.mark.parametrize("M,K,N,group", SHAPES)
def test_large_activations_are_right_or_not_finite(lib, M, K, N, group):
    import torch
    from test_gpu_linear_few import _inputs
    x, q, s, z = _inputs(M, K, N, group, 7)
    want = lib.w4_w4a16_linear_few(x, q, s, z, group)
    tokens = [t for t in range(1, M)][:len(LARGE)]
    for at in (5, K - 2):                      # a code in either half of a byte, two groups
        for alone in (True, False):
            big = x.clone()
            for t, v in zip(tokens, LARGE):
                if alone:
                    big[t] = 0.0
                big[t, at] = v
            got = lib.w4_w4a16_linear_few(big, q, s, z, group)
            ref, tol = _expect(big, q, s, z, group)
            wrong = got.isfinite() & ~((got.double() - ref).abs() <= tol)
            assert not bool(wrong.any()), wrong.nonzero()[:5].tolist()
            rest = [t for t in range(M) if t not in tokens]
            assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("M,K,N,group", SHAPES)
def test_up_to_2_57_nothing_is_lost(lib, M, K, N, group):
    from test_gpu_linear_few import _check, _inputs
    x, q, s, z = _inputs(M, K, N, group, 8)
    x[1] = x[1].sign() * 2.0 ** 57
    x[2] *= 2.0 ** 54
    x[3, 7] = -(2.0 ** 57)
    y = lib.w4_w4a16_linear_few(x, q, s, z, group)
    assert bool(y.isfinite().all())
    _check(y, x, q, s, z, group)


@pytest.mark.parametrize("M,K,N,group", SHAPES)
def test_small_activations(lib, M, K, N, group):
    from test_gpu_linear_few import _inputs
    x, q, s, z = _inputs(M, K, N, group, 9)
    for t in range(M):
        x[t] *= 2.0 ** (-50 - 7 * (t % 12))    # down to bf16's subnormals
    x[4] = 2.0 ** -133
    y = lib.w4_w4a16_linear_few(x, q, s, z, group)
    ref, tol = _expect(x, q, s, z, group)
    # (a result below bf16's normal ones is rounded to a step of 2^-133)
    tol = tol + 2.0 ** -134 + (0.0 if N > 10000 else K / group * 12.5 * 2.0 ** -86)
    assert bool(((y.double() - ref).abs() <= tol).all())
    assert N > 10000 or (float(s.max()) < 1.0 and float(z.max()) < 16.0)


@pytest.mark.parametrize("M,K,N,group", SHAPES)
def test_what_is_not_finite_stays_so(lib, M, K, N, group):
    import torch
    from test_gpu_linear_few import _inputs
    x, q, s, z = _inputs(M, K, N, group, 10)
    s[3], z[4] = 0.0, 0.0
    want = lib.w4_w4a16_linear_few(x, q, s, z, group)
    x[1, 0], x[2, K - 1], x[5, 9] = math.inf, -math.inf, math.nan
    got = lib.w4_w4a16_linear_few(x, q, s, z, group)
    assert not bool(got[[1, 2, 5]].isfinite().any())
    rest = [t for t in range(M) if t not in (1, 2, 5)]
    assert torch.equal(got[rest], want[rest])
