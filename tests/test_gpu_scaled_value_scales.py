"""What verify_attn_scaled makes of scales that are not finite, at positions that only some rows see, or none."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from tests.test_gpu_scaled_attn import TYPES, dev, make_cache, num, signed

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P = 16
# heads, query rows a KV head and types of both forms that V and the weights take
SHAPES = [(64, 6, 4, "bf16"), (128, 6, 2, "bf16"), (128, 6, 4, "f16"), (128, 12, 4, "bf16"), (256, 6, 2, "f16"),
          (256, 6, 4, "bf16"), (64, 1, 4, "f16"), (128, 1, 4, "bf16"), (256, 1, 2, "bf16")]


def spoilt(cache, table, at, which, value, head=0):
    """A copy of the cache in which the scales of some positions (blocks of one token) are `value`."""
    out = [x.clone() for x in cache]
    for t in at:
        for w in which:
            out[w][table[0, t // P], t % P, head] = value
    return out


def untouched(got, clean, hit):
    """Rows that do not see it are equal, bit for bit; those that do are NaN."""
    (out, lse), (out0, lse0) = got, clean
    o, o0, l, l0 = num(out)[0], num(out0)[0], num(lse)[0], num(lse0)[0]
    assert np.isnan(o[hit]).all() and np.isnan(l[hit]).all()
    np.testing.assert_array_equal(o[~hit], o0[~hit])
    np.testing.assert_array_equal(l[~hit], l0[~hit])


@pytest.mark.parametrize("D,R,G,new", SHAPES)
@pytest.mark.parametrize("which,value", [([3], float("nan")), ([2], float("nan")), ([3], float("inf")),
                                         ([2, 3], float("nan"))])
def test_scales_in_masked_places_stay_there(D, R, G, new, which, value):
    """Scales (2: of K, 3: of V) of single positions, seen by some rows of the block, by row 0 alone (the edge
    of the window) or by none."""
    ctx, Hkv = 150, 2
    cache, _, table = make_cache([ctx + R], Hkv, D, P, 1, seed=D + R, spread=0)
    q = torch.from_numpy(np.random.default_rng(D).normal(size=(1, R, G * Hkv, D))).to(TYPES[new]).to(DEV)
    masks = [[1, 3, 5, 9, 0b10011, 0b1101] + [(1 << i | 1) for i in range(6, R)]][0][:R]
    anc = dev(signed([masks]), torch.int64)
    tab, c = dev(table), dev([ctx])
    for window in (0, 100):
        call = lambda x: sv.verify_attn_scaled(q, *x, tab, c, anc, window=window)
        clean = call(cache)
        assert torch.isfinite(clean[0]).all() and torch.isfinite(clean[1]).all()
        for j in range(min(R, 6)):             # block row j: seen as the masks say (row 5 by none)
            sees = np.array([m >> j & 1 for m in masks], bool)
            hit = np.zeros((R, G * Hkv), bool)
            hit[sees, :G] = True
            untouched(call(spoilt(cache, table, [ctx + j], which, value)), clean, hit)
        if window:
            none = np.zeros((R, G * Hkv), bool)
            untouched(call(spoilt(cache, table, [ctx - window, 3], which, value, head=1)), clean, none)
            edge = none.copy()
            edge[[bin(m).count("1") == 1 for m in masks], G:] = True
            untouched(call(spoilt(cache, table, [ctx + 1 - window], which, value, head=1)), clean, edge)
