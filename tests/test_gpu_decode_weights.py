"""One-token attention in fp16 beside e4m3 caches: the weights are not rounded to the output's
precision."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import decode as odec
from tests.test_gpu_cache_side import DEV, dev, num

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G", [(64, 4), (64, 12), (128, 1), (128, 16), (256, 8)])
def test_weights_beside_e4m3_keep_more_than_sixteen_bits(D, G):
    """Values of both signs that nearly cancel, and queries of one nonzero element, so that a
    score is one exact product.  What is left: scaling (three roundings of a score below 2),
    the distance from the reference (2^-21 of a number below 16, with the log2 domain's), ex2
    (2^-22), sums of at most 300 weights in tiles (2^-20), P's parts (2^-22, or 2^-32 of the
    largest where subnormal): below 2^-18 of sum p |v|, and one fp16 rounding of the output."""
    rng = np.random.default_rng(D + G)
    lens, P = [2, 3, 5, 9, 64, 300], 16
    width = 19
    table = rng.permutation(len(lens) * width).reshape(len(lens), width)
    k = rng.integers(-8, 9, (len(lens) * width, P, 1, D)) / 8.0       # e4m3 numbers
    v = rng.choice([-1.0, 1.0], k.shape)
    q = np.zeros((len(lens), G, D))
    q[:, np.arange(G), rng.integers(0, D, G)] = 1.5
    t = lambda x, dt: torch.tensor(x).to(dt).to(DEV)  # noqa: E731
    f8 = torch.float8_e4m3fn
    out, lse = sv.decode_attn(t(q, torch.float16), t(k, f8), t(v, f8), dev(table), dev(lens),
                              scale=0.7)
    ref, lref, _, mass = odec.decode_attention(q, k, v, table, lens, 0.7)
    tol = 2.0 ** -11 * np.abs(ref) + 2.0 ** -18 * mass + 2.0 ** -25
    assert (np.abs(ref) < 2.0 ** -4 * mass).any()         # some outputs are nearly cancelled
    assert (np.abs(num(out) - ref) <= tol).all(), (np.abs(num(out) - ref) / tol).max()
    assert (np.abs(num(lse) - lref) <= 2.0 ** -18).all()
