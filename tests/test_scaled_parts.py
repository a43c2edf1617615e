"""The arithmetic by which a weight of verify_attn_scaled is split, on the CPU: every fp16 number from 0 to 2^15
is the sum of three e5m2 numbers, the second over 2^4 and the third over 2^8, and NaN stays NaN."""
import numpy as np


def upper(h):
    """Rounded to the nearest number whose lower byte is zero, by its bits."""
    return ((h.view(np.uint16).astype(np.uint32) + 0x80) & 0xff00).astype(np.uint16).view(np.float16)


def parts(h):
    sixteen = np.float16(16)
    x1 = upper(h)
    r1 = (h - x1) * sixteen
    x2 = upper(r1)
    return x1, x2, (r1 - x2) * sixteen


def test_three_parts_hold_every_weight():
    h = np.arange(0, 0x7801).astype(np.uint16).view(np.float16)      # 0 .. 2^15
    assert h[-1] == 2.0 ** 15
    x = parts(h)
    for p in x:
        assert not (p.view(np.uint16) & 0xff).any() and np.abs(p.astype(np.float64)).max() <= 57344
    total = sum(p.astype(np.float64) * 2.0 ** -s for p, s in zip(x, (0, 4, 8)))
    np.testing.assert_array_equal(total, h.astype(np.float64))


def test_nan_stays():
    assert np.isnan(parts(np.array([np.nan], np.float16))[2]).all()
