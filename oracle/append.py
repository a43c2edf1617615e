"""Oracle: rotary position at depth and the block's K/V append (next row f3).

TEST INFRASTRUCTURE ONLY (see the package docstring).

What it computes.  Before the verify attention, the target writes the K/V rows
of the proposed block into the paged cache: row j at position ctx_len + j (the
layout the verify attention reads).  Keys carry their position: "Speculative
Decoding" (atlas), "Chains, trees and visibility" -- position ids follow
depth, not flattened storage order -- so node j's key is rotated for position
ctx_len + depth(j) while it is stored at slot ctx_len + j.

Readings (the pages do not print the rotation):
  * the rotary embedding is the common split-half form: for pair index
    i < D/2, theta_i = base^(-2 i / D), the pair (x_i, x_{i + D/2}) at
    position t is rotated by the angle t * theta_i;
  * the same rotation applies to the block's queries (not stored);
  * values are stored unrotated.
"""
import numpy as np


def rope(x, pos, base: float = 10000.0):
    """x [..., D] rotated for integer positions pos (broadcast over x[..., 0])."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    if D % 2:
        raise ValueError("head_dim must be even")
    half = D // 2
    theta = base ** (-2.0 * np.arange(half) / D)
    ang = np.asarray(pos, dtype=np.float64)[..., None] * theta
    c, s = np.cos(ang), np.sin(ang)
    a, b = x[..., :half], x[..., half:]
    if a.ndim > ang.ndim:  # heads between the position axes and D
        c = c[..., None, :]
        s = s[..., None, :]
    return np.concatenate([a * c - b * s, a * s + b * c], axis=-1)


def append_block(k_cache, v_cache, block_table, ctx_len, k_new, v_new, pos_ids, page_size: int,
                 base: float = 10000.0):
    """Copies of the caches with the block written in.

    k_new, v_new [B, R, Hkv, D] (keys before rotation); pos_ids [B, R] (ctx_len
    + depth).  Row j of sequence b goes to position ctx_len[b] + j; the key is
    rotated for pos_ids[b, j]."""
    kc = np.array(k_cache, dtype=np.float64, copy=True)
    vc = np.array(v_cache, dtype=np.float64, copy=True)
    B, R = np.asarray(pos_ids).shape
    for b in range(B):
        for j in range(R):
            pos = int(ctx_len[b]) + j
            page, off = block_table[b][pos // page_size], pos % page_size
            kc[page, off] = rope(np.asarray(k_new)[b, j], int(pos_ids[b][j]), base)
            vc[page, off] = np.asarray(v_new)[b, j]
    return kc, vc


def e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even, limited to +-448): 3 fraction
    bits, exponents -6 .. 8, steps of 2^-9 below 2^-6."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(x), 448.0)
    e = np.clip(np.floor(np.log2(np.maximum(mag, 2.0 ** -6))), -6, 8)
    step = 2.0 ** (e - 3)
    return np.copysign(np.minimum(np.rint(mag / step) * step, 448.0), x)


def append_tokens(k_cache, v_cache, k_new, v_new, slots, positions, page_size: int, base=10000.0,
                  k_scale=None, v_scale=None):
    """Copies of the caches with packed rows [T, Hkv, D] at their slots, before any
    rounding (divided by the heads' scales where those are given); base 0: no rotation.
    Rows whose slot is outside the cache are skipped."""
    kc = np.array(k_cache, dtype=np.float64, copy=True)
    vc = np.array(v_cache, dtype=np.float64, copy=True)
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if not 0 <= slot < kc.shape[0] * page_size or (base and positions[t] < 0):
            continue
        at = (slot // page_size, slot % page_size)
        k = rope(np.asarray(k_new)[t], int(positions[t]), base) if base else np.asarray(k_new)[t]
        kc[at] = k if k_scale is None else k / np.asarray(k_scale)[:, None]
        vc[at] = v_new[t] if v_scale is None else v_new[t] / np.asarray(v_scale)[:, None]
    return kc, vc
