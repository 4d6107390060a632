"""Rotary positions near 2^31, where the frequency's last bits decide: positions
are picked at which the angle is all but a whole number of turns, so that the
sine shows the angle's absolute error.

Bound of a sine s of (a, b) = (1, 0): the angle to 2^-31 turns (the header's
statement), 2^-21 |s| for fp32 (as in tests/test_gpu_rotary.py), then one
rounding to bf16. The oracle is in integers: 1 / 2 pi to 300 bits.
"""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from exact_attention_forward_tiled_gb300 import api
from exact_attention_forward_tiled_gb300 import build as fa_build

pytestmark = pytest.mark.gpu
BITS = 300


def _one_over_2pi():
    """floor(2^BITS / 2 pi) by Machin's formula, pi / 4 = 4 atan(1/5) - atan(1/239)."""
    one = 1 << (BITS + 64)

    def atan(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (-term if k & 1 else term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total
    pi = 4 * (4 * atan(5) - atan(239))          # pi * 2^(BITS + 64)
    return (1 << (2 * BITS + 64)) // (2 * pi)


def _turns(w, p, c):
    """Angle w p as a fraction of a turn in [-1/2, 1/2)."""
    x = (Fraction(w) * p * Fraction(c, 1 << BITS)) % 1
    return float(x - 1 if x >= Fraction(1, 2) else x)


@pytest.mark.parametrize("freq", [1.0, -1.0, 0.75, 3.3, -17.1, 1000.1, -123456.7, 2.0 ** 20 + 0.3, 10000.0 ** -0.03125])
@pytest.mark.parametrize("backward", [False, True])
def test_sine_of_far_positions(cuda_device, freq, backward):
    fa_build.build()
    c = _one_over_2pi()
    assert c >> (BITS - 53) == int(math.ldexp(1 / (2 * math.pi), 53))
    step = int((Fraction(freq) * Fraction(c, 1 << BITS)) % 1 * (1 << 64))
    far = np.concatenate([np.arange(2 ** 31 - 2 ** 23, 2 ** 31, dtype=np.int64),
                          np.arange(-2 ** 31, -2 ** 31 + 2 ** 23, dtype=np.int64)])
    near = np.abs((far.astype(np.uint64) * np.uint64(step)).astype(np.int64).astype(np.float64)) * 2.0 ** -64
    pick = far[(near > 2.0 ** -25) & (near < 2.0 ** -20)]
    pick = pick[np.linspace(0, len(pick) - 1, min(len(pick), 64)).astype(int)]
    assert len(pick) >= 4
    q = torch.zeros((len(pick), 1, 2), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    pos = torch.tensor(pick, dtype=torch.int32, device="cuda")[None].contiguous()
    plan = api.rotary_plan(2, (1,), inv_freq=(freq,))
    out, _ = (api.rotary_backward if backward else api.rotary_forward)(q, None, pos, plan)
    sign = -1.0 if backward else 1.0
    for p, s in zip(pick.tolist(), out[:, 0, 1].double().tolist()):
        want = sign * math.sin(2 * math.pi * _turns(freq, p, c))
        bound = 2 * math.pi * 2.0 ** -31 + abs(want) * 2.0 ** -21
        bound += 2.0 ** -8 * (abs(want) + bound)
        assert abs(s - want) <= bound, (p, s, want, bound)
