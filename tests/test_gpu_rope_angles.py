"""How exact the rotation's angles are.  Near a half turn a sine is as small as the angle's
distance from it, so a 16-bit result shows angles far below its own step of a half turn.

Tolerance.  pos * step modulo 2^64 is the angle's definition; its upper 32 bits drop less
than 2^-32 of a turn, and fp32 rounds them by at most 2^6 of 2^-32, 2^-26 of a turn: together
below 2^-25, times 2 pi a unit of the first value.  sincospif is within 2^-22 of its value,
the result's rounding within a half step of its type."""
import math

import pytest

pytestmark = pytest.mark.gpu


def _near_half(step, span):
    """Positions up to 2^26 at which a pair's angle is nearest to a half turn, and by how much
    (in turns)."""
    import numpy as np
    pos = np.arange(1, 1 << 26, dtype=np.uint64)
    far = (pos * np.uint64(step) + np.uint64(1 << 63)).astype(np.int64)    # modulo 2^64
    near = np.abs(far.astype(np.float64)) < span * 2.0 ** 64
    return pos[near].astype(np.int64), far[near]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_near_a_half_turn(lib, dtype, interleaved):
    import numpy as np
    import torch
    u = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}[dtype]
    steps = lib.w4_rope_steps(64)
    for pair in (0, 3):
        step = int(steps[pair]) % 2 ** 64
        pos, far = _near_half(step, 2.0 ** -15)
        assert len(pos) > 500
        pos, far = np.concatenate((pos, -pos)), np.concatenate((far, -far))
        q = torch.zeros((len(pos), 1, 64), dtype=getattr(torch, dtype), device="cuda")
        first, second = (2 * pair, 2 * pair + 1) if interleaved else (pair, pair + 32)
        q[:, :, first] = 1.0
        got = lib.w4_qk_norm_rope(q, q[:, :0], torch.from_numpy(pos.astype(np.int32)).cuda(), steps,
                                  interleaved=interleaved)[0][:, 0].double().cpu().numpy()
        # sin(2 pi (1/2 + d)) = -sin(2 pi d)
        want = -np.sin(2 * math.pi * far.astype(np.float64) * 2.0 ** -64)
        bound = 2 * math.pi * 2.0 ** -25 + (u + 2.0 ** -22) * np.abs(want) + 2.0 ** -25 * u
        if dtype == "float16":
            bound = bound + 2.0 ** -25         # half a step of its subnormals
        assert (np.abs(got[:, second] - want) <= bound).all()
        assert (got[:, first] == -1.0).all()
