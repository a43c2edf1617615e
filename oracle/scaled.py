"""Oracle: a cache of e4m3 codes with one scale for each block of tokens and head, and the
verify attention over it.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Readings: a block's scale is the smallest power of two (2^-64 at least) that keeps the largest
finite value stored to it by a call at or below 448 codes; a block whose first token is among the
rows begins anew, another keeps the larger scale, its other codes re-expressed.  A position's
code stands for code * scale.  Attention: every committed position (with a window, the last
`window` tokens of a row's own text) and the block rows of the row's mask.
"""
import math

import numpy as np

from .append import e4m3

LEAST = 2.0 ** -64


def needed(x):
    """The scale for these values."""
    x = np.abs(np.asarray(x, dtype=np.float64)).ravel()
    x = x[np.isfinite(x)]
    big, s = (x.max() if x.size else 0.0), LEAST
    while big > 448.0 * s:
        s *= 2
    return s


def held(s):
    """What a stored scale counts as: the next power of two, 0 if it is none."""
    if not (s > 0 and np.isfinite(s)):
        return 0.0
    return 2.0 ** math.ceil(math.log2(s)) if math.log2(s) != int(math.log2(s)) else float(s)


def code(x):
    """e4m3 code values of x: infinities +-448, NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    y = e4m3(np.where(np.isnan(x), 0.0, np.clip(x, -448, 448)))
    return np.where(np.isnan(x), np.nan, y)


def append(codes, scales, rows, slots):
    """codes [pages, P, H, D] (their numbers), scales [pages, nb, H], rows [T, H, D] at
    slots -> new codes and scales."""
    codes, scales = np.array(codes, np.float64), np.array(scales, np.float64)
    pages, P, H, _ = codes.shape
    size = P // scales.shape[1]
    groups = {}
    for t, s in enumerate(np.asarray(slots).tolist()):
        if 0 <= s < pages * P:
            groups.setdefault(s // size, []).append((t, s % size))
    for blk, who in groups.items():
        page, j = blk // (P // size), blk % (P // size)
        offs = [o for _, o in who]
        for h in range(H):
            have = 0.0 if 0 in offs else held(scales[page, j, h])
            new = max(have, needed(np.stack([rows[t, h] for t, _ in who])))
            if have > 0:
                for o in range(size):
                    if o not in offs:
                        at = (page, j * size + o, h)
                        codes[at] = code(codes[at] * (scales[page, j, h] / new))
            scales[page, j, h] = new
            for t, o in who:
                codes[page, j * size + o, h] = code(rows[t, h] / new)
    return codes, scales


def values(codes, scales):
    """What the codes stand for, [pages, P, H, D]."""
    return np.asarray(codes, np.float64) * np.repeat(scales, codes.shape[1] // scales.shape[1],
                                                     axis=1)[..., None]


def commit(codes, scales, table, ctx, accepted, path):
    """A tree's accepted rows moved to the next logical prefix (one cache)."""
    P = codes.shape[1]
    vals = values(codes, scales)
    for b, a in enumerate(accepted):
        rows, slots = [], []
        for k in range(a):
            src, dst = ctx[b] + path[b][k], ctx[b] + k + 1
            rows.append(vals[table[b][src // P], src % P])
            slots.append(table[b][dst // P] * P + dst % P)
        if a:
            codes, scales = append(codes, scales, np.stack(rows), slots)
    return codes, scales


def attention(q, k, v, table, ctx_len, mask, scale=None, window=0):
    """q [B, R, Hq, D], k and v [pages, P, Hkv, D] (values), mask [B][R] ints -> out, lse, and
    for error bounds: the largest scale sum |q_d k_d|, the largest scale max|q| sum |k_d|,
    sum p |v|, the largest p |v| and the positions seen, of every row."""
    q = np.asarray(q, np.float64)
    B, R, Hq, D = q.shape
    pages, P, Hkv, _ = k.shape
    scale = scale if scale else 1.0 / math.sqrt(D)
    out, lse = np.zeros((B, R, Hq, D)), np.full((B, R, Hq), -np.inf)
    aux = dict(big=np.zeros((B, R, Hq)), edge=np.zeros((B, R, Hq)), mass=np.zeros((B, R, Hq, D)),
               peak=np.zeros((B, R, Hq)), n=np.zeros((B, R, Hq)))
    for b in range(B):
        c = int(ctx_len[b])
        if c < 0:
            continue
        for i in range(R):
            m = int(mask[b][i])
            first = max(0, c + bin(m).count("1") - window) if window else 0
            ts = list(range(first, c)) + [c + j for j in range(R) if m >> j & 1]
            ts = [t for t in ts if t < table.shape[1] * P]
            at = [(int(table[b][t // P]), t % P) for t in ts]
            at = [x for x in at if 0 <= x[0] < pages]
            if not at:
                continue
            ix = tuple(np.array(at).T)
            kk, vv = k[ix], v[ix]                                # [n, Hkv, D]
            for h in range(Hq):
                kh, vh = kk[:, h // (Hq // Hkv)], vv[:, h // (Hq // Hkv)]
                x = kh @ q[b, i, h] * scale
                top = x.max()
                p = np.exp(x - top)
                z = p.sum()
                at_ = (b, i, h)
                out[at_] = p @ vh / z
                lse[at_] = top + math.log(z)
                aux["big"][at_] = (np.abs(kh) @ np.abs(q[at_])).max() * scale
                aux["edge"][at_] = np.abs(q[at_]).max() * np.abs(kh).sum(1).max() * scale
                aux["mass"][at_] = p @ np.abs(vh) / z
                aux["peak"][at_] = (p * np.abs(vh).max(1)).max() / z
                aux["n"][at_] = len(at)
    return out, lse, aux
