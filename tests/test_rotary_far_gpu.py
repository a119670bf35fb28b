"""Angles of qv_rotary at far positions, against 1 / (2 pi) in whole numbers (a product in binary64 would be off itself)."""
import math

import pytest
import torch

from gpu_util import require_gpu
from quantized_verification_gb300 import qv

pytestmark = pytest.mark.gpu
BITS = 256


def _pi(bits):
    """floor(pi 2^bits), by Machin: 16 atan(1/5) - 4 atan(1/239)."""
    def atan_inverse(x):
        t = (1 << bits + 32) // x
        s, k = t, 1
        while t:
            t, k = t // (x * x), k + 2
            s += t // k if k % 4 == 1 else -(t // k)
        return s
    return (16 * atan_inverse(5) - 4 * atan_inverse(239)) >> 32


PI = _pi(BITS)


def turn(f, p):
    """The angle p * f (f a float that binary32 holds) modulo a turn, in (-pi, pi], from whole numbers."""
    num, den = f.as_integer_ratio()
    two_pi = 2 * PI
    x = (num * p << BITS) // den % two_pi
    x = x - two_pi if x > PI else x
    return x / (1 << BITS)


@pytest.mark.parametrize("freq", [1.0, 0.8125, 6.5, 31.987, 32.0, 1000.25, 2.0 ** 20 + 0.125, 1e-5])
def test_angles_at_far_positions(freq):
    require_gpu()
    f = torch.full((8,), freq, device="cuda")
    exact = float(f[0])
    pos = [2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 7, -987654321, 131071, 1]
    x = torch.zeros(len(pos), 3 * 16, device="cuda")
    x[:, :8] = 1.0                                               # (1, 0) -> (cos, sin)
    qv.qv_rotary(x, torch.tensor(pos, dtype=torch.int32, device="cuda"), f, 1, 1)
    for row, p in zip(x.tolist(), pos):
        a = turn(exact, p)
        # documented: 2e-7 up to frequencies of 32, more in proportion above; a step of the cosine itself
        tol = 2e-7 + (1.4e-18 * abs(p * exact) if exact > 32 else 0.0) + 2.0 ** -23
        assert abs(row[0] - math.cos(a)) <= tol and abs(row[8] - math.sin(a)) <= tol, (p, row[0] - math.cos(a))
