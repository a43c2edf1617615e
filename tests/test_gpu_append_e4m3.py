"""Packed append into e4m3: the stored value is the quotient x / scale on the grid, ties and
the ends of the scales' range included."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import append as oapp
from tests.test_gpu_cache_side import DEV, TYPES, dev, num

pytestmark = pytest.mark.gpu


def grid_midpoints():
    every = np.arange(127, dtype=np.uint8)                       # 0 .. 448
    v = torch.from_numpy(every).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    return (v[1:] + v[:-1]) / 2


@pytest.mark.parametrize("new", ["bf16", "f16"])
def test_append_stores_the_quotient_on_ties(new):
    """Rows that are exactly a midpoint of the grid times the scale: the quotient is the
    midpoint and goes to the even neighbour.  A rounded reciprocal misses some of them."""
    D, mids = 64, grid_midpoints()
    scales, rows, missed = [], [], 0
    for m in range(3, 128, 2):
        s = np.float32(m * 2.0 ** -10)
        x = mids * float(s)
        x = x[torch.tensor(x).to(TYPES[new]).double().numpy() == x]      # exact in the type
        x = np.concatenate([x, -x])
        missed += int((x.astype(np.float32) * (np.float32(1) / s) != x / float(s)).sum())
        scales.append(s)
        rows.append(np.resize(x, 4 * D) if len(x) else np.zeros(4 * D))
    assert missed > 0                            # the cases tell the two apart
    H = len(scales)
    x = np.ascontiguousarray(np.stack(rows).reshape(H, 4, D).transpose(1, 0, 2))
    t = torch.tensor(x).to(TYPES[new]).to(DEV)
    sc = torch.tensor(np.array(scales)).to(DEV)
    kc, vc = (torch.zeros((1, 4, H, D), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    sv.append_tokens(t, t, kc, vc, dev([0, 1, 2, 3], torch.int64), rope_base=0, k_scale=sc,
                     v_scale=sc)
    want = oapp.e4m3(x / np.array(scales, dtype=np.float64)[:, None])
    np.testing.assert_array_equal(num(kc)[0], want)
    np.testing.assert_array_equal(num(vc)[0], want)


def test_append_scales_at_the_ends_of_their_range():
    """Scales whose reciprocal is no fp32 number, or a subnormal one."""
    D, scales = 64, np.array([1e-39, 1e-45, 2.0 ** 127, 3.0e38], dtype=np.float32)
    x = torch.zeros((2, 4, D), dtype=torch.bfloat16)
    for h, s in enumerate(scales):               # zeros, and multiples of the scale in row 1
        x[1, h] = torch.tensor(np.linspace(-1.0, 1.0, D) * float(s)).bfloat16()
    x[1, 0, 5], x[1, 1, 5] = 2.0, -1e-20         # far beyond the grid
    kc, vc = (torch.ones((1, 2, 4, D), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    sc = torch.tensor(scales).to(DEV)
    sv.append_tokens(x.to(DEV), x.to(DEV), kc, vc, dev([0, 1], torch.int64), rope_base=0,
                     k_scale=sc, v_scale=sc)
    q = num(x) / scales.astype(np.float64)[:, None]
    np.testing.assert_array_equal(num(kc)[0], oapp.e4m3(q))
    np.testing.assert_array_equal(num(vc)[0], oapp.e4m3(q))
