"""Attention rows whose largest weight has a value of zero, so that the result is all tail: thousands of positions
2^-12 to 2^-24 below it, with weights that no short number holds.

There are more (sequence, KV head) pairs than ranges, so whole sequences lie in one, and half of a tail is
weighed beside the large position.

Tolerance.  A weight is held in 11 bits (2^-11, on the safe side) down to 2^-22 of the row's largest, and
below that to 2^-33 of it: 2^-33 of the largest weight times sum |v|.  Scores, sums and the output's own
rounding as in test_gpu_scaled_attn.bound().
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from tests.test_gpu_scaled_attn import HALF, TYPES, dev, num

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P = 64


@pytest.mark.parametrize("D,R,G", [(64, 1, 4), (128, 1, 4), (128, 5, 4), (128, 16, 4), (256, 2, 4), (256, 5, 4)])
@pytest.mark.parametrize("new", ["bf16", "f16"])
@pytest.mark.parametrize("low", [12, 17, 20, 24])
def test_a_tail_beside_one_large_position(D, R, G, new, low):
    B, Hkv, n = 40, 4, 1500
    pages = -(-n // P)
    rng = np.random.default_rng(D + R + low)
    k = np.zeros((B * pages, P, Hkv, D))
    k[..., 0] = rng.uniform(-0.5, 0.5, k.shape[:3])
    k[::pages, 0, :, 0] = 8.0                                   # position 0 of each sequence
    v = rng.normal(size=k.shape)
    v[::pages, 0] = 0.0
    kc, vc = (torch.from_numpy(x).float().to(torch.float8_e4m3fn).to(DEV) for x in (k, v))
    one = torch.ones((B * pages, 1, Hkv), device=DEV)
    q = torch.zeros((B, R, G * Hkv, D), dtype=TYPES[new], device=DEV)
    q[..., 0] = 1.0
    scale = low * np.log(2) / 8
    table = np.arange(B * pages).reshape(B, pages)
    out, lse = sv.verify_attn_scaled(q, kc, vc, one, one, dev(table), dev([n - R] * B), scale=scale)
    # rows of a chain differ in the last positions they see; all heads of a KV head are alike
    x = num(kc)[..., 0].reshape(B, pages * P, Hkv) * float(np.float32(scale))
    vals = num(vc).reshape(B, pages * P, Hkv, D)
    for i in range(R):
        m = n - R + 1 + i
        w = np.exp(x[:, :m] - x[:, :1])                         # 1 for the large one
        z = w.sum(1)
        p = (w / z[:, None]).transpose(0, 2, 1)[:, :, None]     # [B, Hkv, 1, m]
        vv = vals[:, :m].transpose(0, 2, 1, 3)
        ref, mass = (p @ vv)[:, :, 0], (p @ np.abs(vv))[:, :, 0]
        score = 3 * D * 2.0 ** -23 * low + 2.0 ** -21 * (low + 16) + 2.0 ** -20
        sums = (m / 16 + 512) * 2.0 ** -23
        tol = HALF[new] * np.abs(ref) + (2.0 ** -11 + 2 * score + 2 * sums) * mass \
            + 2.0 ** -33 * p[..., :1].max() * np.abs(vv).sum(2) + (2.0 ** -25 if new == "f16" else 0)
        got = num(out)[:, i].reshape(B, Hkv, G, D)
        err = np.abs(got - ref[:, :, None])
        assert (err <= tol[:, :, None]).all(), (i, (err / tol[:, :, None]).max())
        le = np.abs(num(lse)[:, i].reshape(B, Hkv, G) - (x[:, 0] + np.log(z))[:, :, None])
        assert (le <= score + sums + 2.0 ** -22 * low).all()
