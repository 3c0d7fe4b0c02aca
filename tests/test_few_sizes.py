"""The few-token layer refuses widths whose rows do not fit shared memory, however
large: their sizes are not worked out in wrapped 32-bit arithmetic."""
import ctypes
import random

import pytest

import w4a16_moe_expert_sync_gb300 as w4


@pytest.fixture(scope="module")
def call():
    from w4a16_moe_expert_sync_gb300 import build as w4build
    w4build.build()
    lib = w4.load_library()
    fake = ctypes.c_void_p(0x10000)

    def few(d, m):
        return lib.w4_moe_layer_few(fake, fake, fake, 1, d, m, 1, 1, fake, fake, fake, 128, fake,
                                    fake, fake, 64, None, 0, fake, None, None)
    return few


# without a workspace nothing is launched, whatever the shape
UNSUPPORTED, NO_WORKSPACE = 2, 6


def test_widths_that_once_wrapped(call):
    for d in (1041205888, 1 << 30, 2114444928, (1 << 31) - 128):
        assert call(d, 64) == UNSUPPORTED
    for m in (67125056, 1 << 30, 2103657472, (1 << 31) - 64):
        assert call(128, m) == UNSUPPORTED


def test_no_larger_width_is_accepted(call):
    r = random.Random(1)
    for _ in range(20000):
        wide = int(2 ** r.uniform(13.1, 30.99))
        assert call(wide // 128 * 128, r.choice([64, 704, 2560])) == UNSUPPORTED
        assert call(r.choice([128, 2816, 6144]), wide // 64 * 64) == UNSUPPORTED


def test_the_documented_widths_are(call):
    for d, m in ((6144, 64), (128, 2560), (2816, 704), (128, 64)):
        assert call(d, m) == NO_WORKSPACE
