"""One-token attention over infinite values that are seen."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import decode as odec
from tests.test_gpu_cache_side import DEV, HALF, TYPES, attention_bound, dev, make_cache, num

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "f16"])
@pytest.mark.parametrize("Hkv,G,D,lens", [(2, 4, 64, [1, 2, 300, 9000]), (1, 8, 128, [30, 40000]),
                                          (1, 4, 256, [70, 3000])])
def test_decode_attn_infinite_values_that_are_seen(cache, Hkv, G, D, lens):
    """An infinite V element makes its dimension infinite, of its sign; both signs make it
    NaN; the other dimensions do not notice.  (Every weight is far above 2^-32 of the
    largest, where one may be 0.)"""
    k, v, table, _ = make_cache(lens, Hkv, D, 16, cache, D)
    rng = np.random.default_rng(D)
    inf = float("inf")
    for b, n in enumerate(lens):
        for i in range(12):                      # dimensions 0 .. 11: +, -, and both
            for sign in ((inf,), (-inf,), (inf, -inf))[i % 3]:
                t = int(rng.integers(0, n))
                v[table[b, t // 16], t % 16, i % Hkv, i] = sign
    q = torch.randn((len(lens), G * Hkv, D),
                    generator=torch.Generator().manual_seed(D)).to(TYPES[cache])
    out, lse = sv.decode_attn(q.to(DEV), k.to(DEV), v.to(DEV), dev(table), dev(lens))
    with np.errstate(invalid="ignore"):
        ref, lref, big, mass = odec.decode_attention(num(q), num(k), num(v), table, lens)
        tol, ltol = attention_bound(ref, big, mass, lref, np.array(lens)[:, None], D,
                                    HALF[cache], cache)
    o = num(out)
    np.testing.assert_array_equal(np.isnan(o), np.isnan(ref))
    np.testing.assert_array_equal(np.isposinf(o), np.isposinf(ref))
    np.testing.assert_array_equal(np.isneginf(o), np.isneginf(ref))
    fin = np.isfinite(ref)
    assert 0 < fin.sum() < fin.size and (np.abs(o[fin] - ref[fin]) <= tol[fin]).all()
    assert (np.abs(num(lse) - lref) <= ltol).all()
