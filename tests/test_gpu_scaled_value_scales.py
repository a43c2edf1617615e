"""What verify_attn_scaled makes of scales: NaN and infinite ones at positions that only some rows see, or none,
and value scales over the range that the header states.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import scaled as osc
from tests.test_gpu_scaled_attn import HALF, TYPES, bound, chain_masks, dev, make_cache, num, signed

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


@pytest.mark.parametrize("D,R,G,new", SHAPES)
def test_value_scales_too_large_are_loud(D, R, G, new):
    """Above 2^120 a value scale makes NaN of what sees it, as a NaN does."""
    lens = [40, 300]
    cache, _, table = make_cache(lens, 1, D, P, 16, seed=R, spread=0)
    q = torch.from_numpy(np.random.default_rng(1).normal(size=(2, R, G, D))).to(TYPES[new]).to(DEV)
    args = dev(table), dev([n - R for n in lens])
    clean = sv.verify_attn_scaled(q, *cache, *args)
    bad = [x.clone() for x in cache]
    bad[3][table[0, 0]] = 2.0 ** 127           # of the first sequence's first block
    out, lse = sv.verify_attn_scaled(q, *bad, *args)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(out[1], clean[0][1]) and torch.equal(lse[1], clean[1][1])


@pytest.mark.parametrize("D,R,G", [(64, 1, 4), (128, 1, 4), (128, 5, 4), (128, 16, 4), (256, 2, 4), (256, 5, 4)])
@pytest.mark.parametrize("lo,hi", [(-80, -80), (-80, 30), (-64, 46), (10, 120), (119, 120)])
def test_value_scales_over_their_range(D, R, G, lo, hi):
    """2^-80 to 2^120, those of a row within 2^110 of one another, in bf16.  On top of bound(): logarithms and
    references of up to 128 and 256 are rounded to fp32 three times, 3 * 2^-16 (of two, and of a row's sum)."""
    rng = np.random.default_rng((D + R + hi) % 2 ** 32)
    lens, Hkv, B = [700, 90], 2, 2
    cache, _, table = make_cache(lens, Hkv, D, P, 8, seed=D + R, spread=0)
    kc, vc, ks, vs = cache
    # values of at most 2^6 codes, so that the largest scale keeps to bf16's range
    v = torch.from_numpy(rng.uniform(-64, 64, vc.shape)).float().to(torch.float8_e4m3fn).to(DEV)
    e = rng.integers(lo, hi + 1, tuple(vs.shape))
    vs = torch.from_numpy(2.0 ** e).float().to(DEV)
    q = torch.from_numpy(rng.normal(size=(B, R, G * Hkv, D))).bfloat16().to(DEV)
    ctx = [n - R for n in lens]
    out, lse = sv.verify_attn_scaled(q, kc, v, ks, vs, dev(table), dev(ctx))
    kk, vv = osc.values(num(kc), num(ks)), osc.values(num(v), num(vs))
    ref, rl, aux = osc.attention(num(q), kk, vv, table, ctx, [chain_masks(R)] * B)
    # (in units of the least scale, so that bound()'s 2^-25 for results near zero is one of them; values that
    # small vanish in a double beside 2^-25 itself, whose neighbours are 2^-77 away)
    unit = 2.0 ** lo
    aux["mass"], aux["peak"] = aux["mass"] / unit, aux["peak"] / unit
    ob, lb = bound(ref / unit, aux, rl, D, HALF["bf16"], 0)
    ob = (ob + 2 * 3 * 2.0 ** -16 * aux["mass"]) * unit
    err = np.abs(num(out) - ref)
    assert (err <= ob).all(), (err / ob).max()
    assert (np.abs(num(lse) - rl) <= lb + 3 * 2.0 ** -16).all()


@pytest.mark.parametrize("D,R,G", [(64, 1, 4), (128, 5, 4), (256, 5, 4)])
@pytest.mark.parametrize("least", [0.0, 2.0 ** -140, 2.0 ** -81])
def test_value_scales_below_the_least(D, R, G, least):
    """They count as 2^-80: values off by less than 2^-71, weights in full."""
    lens, Hkv = [2000, 40], 1
    cache, _, table = make_cache(lens, Hkv, D, P, 8, seed=D, spread=0)
    kc, vc, ks, vs = cache
    tiny = torch.zeros(vs.shape, dtype=torch.bool, device=DEV)
    tiny[::2] = True
    vs = torch.where(tiny, torch.full_like(vs, least), vs)
    vc = torch.where(torch.isnan(vc.float()), 0.0, vc.float()).to(torch.float8_e4m3fn)
    q = torch.from_numpy(np.random.default_rng(2).normal(size=(2, R, G, D))).bfloat16().to(DEV)
    ctx = [n - R for n in lens]
    out, lse = sv.verify_attn_scaled(q, kc, vc, ks, vs, dev(table), dev(ctx))
    kk, vv = osc.values(num(kc), num(ks)), osc.values(num(vc), num(vs))
    ref, rl, aux = osc.attention(num(q), kk, vv, table, ctx, [chain_masks(R)] * 2)
    ob, lb = bound(ref, aux, rl, D, HALF["bf16"], 0)
    assert (np.abs(num(out) - ref) <= ob + 2.0 ** -71 + 2 * 3 * 2.0 ** -16 * aux["mass"]).all()
    assert (np.abs(num(lse) - rl) <= lb + 3 * 2.0 ** -16).all()
