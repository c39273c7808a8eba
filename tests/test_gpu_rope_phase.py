"""The rotary angle at any accepted frequency and any integer position, against
whole-number arithmetic on the host.

A frequency is held as 2^64 w / (2 pi) modulo 2^64, rounded once, so position m
is off by at most |m| 2^-65 of a turn; the angle is rounded once to fp32 (2 pi
2^-26 rad), cos and sin are off by 2 steps (2^-22), and y = x0 c - x1 s takes
three fp32 roundings: 1e-6 (|x0| + |x1|) in all beside the first term."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_kv_kvq_b200 import build

    build.build()
    import mixed_precision_kv_kvq_b200 as m

    m.load()
    return m


PLACES = 300


def two_pi():
    """2 pi in units of 2^-PLACES, by Machin's formula."""
    one = 1 << (PLACES + 32)

    def arctan_inverse(x):
        term, total, n, sign = one // x, one // x, 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total

    return 8 * (4 * arctan_inverse(5) - arctan_inverse(239)) >> 32


def cos_sin(m, w, turn):
    """Of the angle m w, its whole turns taken off exactly."""
    a = Fraction(w) * m
    units = (a.numerator << PLACES) // a.denominator
    angle = Fraction(units % turn, 1 << PLACES)
    return math.cos(float(angle)), math.sin(float(angle))


FREQS = [2.0 ** 20, 1048575.3, -1048575.3, 1000.3, 6.283185307179586, -5.5, 1.0, 0.37, 1e-4, 3e-9, 1e-300, 0.0]
POSITIONS = [0, 1, -1, 7, 99991, -4097, 2 ** 31 - 1, 2 ** 31 + 5, -(2 ** 33) - 1, 2 ** 40 + 12345, -(2 ** 45) + 7, 2 ** 52 + 1]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_angles_of_fast_pairs_and_far_positions(kvq, layout):
    half, n = len(FREQS), len(POSITIONS)
    rope = kvq.Rope(2 * half, layout=layout, inv_freq=np.array(FREQS))
    x = torch.randn(1, n, 3, 128, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    got = kvq.kvq_rope(rope, torch.tensor(POSITIONS, device="cuda"), x)[0].double().cpu()
    x = x.double().cpu()
    turn = two_pi()
    for t, m in enumerate(POSITIONS):
        for p, w in enumerate(FREQS):
            i, j = (p, p + half) if layout == "half" else (2 * p, 2 * p + 1)
            c, s = cos_sin(m, w, turn)
            a, b = x[0, t, :, i], x[0, t, :, j]
            tol = (1.01e-6 + 2 * math.pi * abs(m) * 2.0 ** -65) * (a.abs() + b.abs())
            for y, want in ((got[0, t, :, i], a * c - b * s), (got[0, t, :, j], b * c + a * s)):
                assert ((y - want).abs() <= tol + 2.0 ** -24 * want.abs()).all(), (m, w)
    assert torch.equal(got[..., 2 * half:], x[..., 2 * half:])
