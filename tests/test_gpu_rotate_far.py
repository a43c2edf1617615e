"""rotate at far positions against angles of fifty digits.

Tolerance: what the header states, t * 2^-54 of a turn for the frequencies, and 2^-20 for the angle as a
32-bit fraction of a turn, sine, cosine and two products in fp32 of numbers of at most 1.
"""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("base,n", [(10000.0, 128), (500000.0, 64), (12345.678, 256)])
def test_far_positions(base, n):
    getcontext().prec = 60
    pos = [0, 1, 4097, 131071, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1]
    x = torch.zeros((len(pos), 1, n), device=DEV)
    x[..., ::2] = 1.0                                           # neighbours (1, 0): cosine and sine
    y = sv.rotate(x, torch.tensor(pos, dtype=torch.int32, device=DEV), sv.Rope(n, base, interleaved=True))[0]
    y = y.double().cpu().numpy()[:, 0]
    for i in range(n // 2):
        turns = (Decimal(base).ln() * Decimal(-2 * i) / n).exp() / (2 * PI)
        for t, row in zip(pos, y):
            u = float((turns * t) % 1) * 2 * math.pi
            tol = 2 * math.pi * t * 2.0 ** -54 + 2.0 ** -20
            assert abs(row[2 * i] - math.cos(u)) <= tol and abs(row[2 * i + 1] - math.sin(u)) <= tol, (i, t)
    assert np.isfinite(y).all()
