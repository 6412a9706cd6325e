"""Rotations of far positions.

Rows of (1, 0) pairs without the norm come out as the cosine and sine themselves.  Bound of their error: the reduction's
1.01 |pos| 2^-65 turns and 2^-32 where the fraction is cut, its rounding to float32 (half turns: 2^-25 of one, 2^-26
turns), and 2 steps (2^-23) of sine and cosine, 2^-24 for the product with 1."""
from fractions import Fraction
import math

import numpy as np
import pytest
import torch

from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import la

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


def pi(bits=320):
    """pi = 16 atan(1/5) - 4 atan(1/239) in integers."""
    def atan_inv(n):
        x = s = (1 << bits) // n
        k, sign = 1, -1
        while x:
            x //= n * n
            k += 2
            s += sign * (x // k)
            sign = -sign
        return s
    return Fraction(16 * atan_inv(5) - 4 * atan_inv(239), 1 << bits)


FAR = [0, 1, 4095, -70000, 10 ** 9 + 7, -(2 ** 39) + 1, 2 ** 39, 2 ** 46 + 3, -(2 ** 50) + 1, 2 ** 50]


@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("D,inter", [(128, False), (64, True), (32, False)])
def test_far_positions(D, inter, base):
    f = [base ** (-i / (D // 2)) for i in range(D // 2)]
    turn = 2 * pi()
    # the fraction of a turn, exactly, then in float64
    angle = np.array([[float((p * Fraction(x) / turn) % 1) for x in f] for p in FAR]) * 2 * math.pi
    x = torch.zeros(1, 1, len(FAR), D)
    one, other = (slice(0, D, 2), slice(1, D, 2)) if inter else (slice(0, D // 2), slice(D // 2, D))
    x[..., one] = 1.0
    y, _ = la.qk_norm_rope_fwd(x.cuda(), x.cuda(), positions=torch.tensor(FAR)[None].cuda(),
                               inv_freq=torch.tensor(f, dtype=torch.float64).cuda(), interleaved=inter, normalize=False)
    la.get_status()
    y = y[0, 0].double().cpu().numpy()
    bound = np.array([2 * math.pi * (1.01 * abs(p) * 2.0 ** -65 + 2.0 ** -32 + 2.0 ** -26) + 2.0 ** -23 + 2.0 ** -24
                      for p in FAR])[:, None]
    assert (np.abs(y[:, one] - np.cos(angle)) <= bound).all()
    assert (np.abs(y[:, other] - np.sin(angle)) <= bound).all()
