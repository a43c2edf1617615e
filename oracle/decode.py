"""Oracle: attention of one new token per sequence over a paged cache.

TEST INFRASTRUCTURE ONLY (see the package docstring).

What it computes: the full softmax over the positions the token sees, in
float64.  Splitting the positions and joining the parts by their log-sum-exp
("Speculative Token Decoupling: Asynchronous Verification via Flash-Decoding",
section 03) reaches this up to rounding, so the oracle does not split.

Readings: the newest of seq_len stored tokens is the one that asks; with a
window it sees the last `window` of them; positions without a page are not
seen; a token that sees nothing gets zeros and -inf.
"""
import math

import numpy as np


def decode_attention(q, k_cache, v_cache, block_table, seq_len, scale=None, window=0):
    """q [B,Hq,D], caches [pages,P,Hkv,D] (the values they stand for) -> out, lse and, for
    error bounds, the largest |scale| sum |q_d k_d| and sum p |v| of every output."""
    q = np.asarray(q, dtype=np.float64)
    B, Hq, D = q.shape
    pages, P, Hkv, _ = k_cache.shape
    scale = scale if scale else 1.0 / math.sqrt(D)
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    big, mass = np.zeros((B, Hq)), np.zeros((B, Hq, D))
    for b in range(B):
        n = min(int(seq_len[b]), block_table.shape[1] * P)
        first = max(0, n - window) if window else 0
        rows = [(int(block_table[b][t // P]), t % P) for t in range(first, n)]
        rows = [r for r in rows if 0 <= r[0] < pages]
        if not rows:
            continue
        at = tuple(np.array(rows).T)
        k, v = k_cache[at].astype(np.float64), v_cache[at].astype(np.float64)   # [n, Hkv, D]
        for h in range(Hq):
            kh, vh = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)]
            x = kh @ q[b, h] * scale
            m = x.max()
            p = np.exp(x - m)
            out[b, h] = p @ vh / p.sum()
            lse[b, h] = m + math.log(p.sum())
            big[b, h] = (np.abs(kh) @ np.abs(q[b, h])).max() * scale
            mass[b, h] = p @ np.abs(vh) / p.sum()
    return out, lse, big, mass
