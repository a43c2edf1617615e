"""GPU parity of the cache's side of a decoding step (extend_tables, release_pages,
append_tokens, decode_attn) against the float64 oracle, and a run of them together.

Tolerances.  Tables hold whole numbers: equal.  A stored element is rounded once from
an fp32 rotation: half a step of its type (bf16 2^-8, fp16 2^-11, e4m3 2^-4 of the value
or 2^-10 where its steps are 2^-9) plus 2^-21 (|a| + |b|) for the angle's, the sine's and
the rotation's fp32 rounding; values that are not rotated are equal.  Attention: see
attention_bound.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import append as oapp
from oracle import decode as odec
from oracle import sampler as osm
from oracle import tables as otab
from oracle.attention import verify_attention
from speculative_decoding_verification_76_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn,
         "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4, "f32": 2.0 ** -24}


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).to(DEV)


def num(t):
    return t.detach().float().cpu().double().numpy() if t.is_floating_point() \
        else t.cpu().numpy()


# ------------------------------------------------------------------ tables
def check_extend(ctx, add, table, lst, count, P, cap):
    t = dev(table)
    e = sv.extend_tables(dev(ctx), dev(add), t, dev(lst), dev([count]), P, cap)
    ref = otab.extend(ctx, add, table, lst, count, P, cap)
    np.testing.assert_array_equal(num(t), ref["block_table"])
    for k in ("slot_map", "positions", "cu_len", "new_len", "status"):
        np.testing.assert_array_equal(num(e[k]), ref[k], err_msg=k)
    assert e["free_count"].tolist() == [ref["free_count"]]
    return t, e, ref


def random_pool(rng, ctx, P, width, spare):
    """Tables whose first ceil(ctx / P) entries hold pages, and a list of the others."""
    had = [-(-c // P) for c in ctx]
    perm = rng.permutation(sum(had) + spare)
    table, at = np.full((len(ctx), width), -1), 0
    for b, n in enumerate(had):
        table[b, :n] = perm[at:at + n]
        at += n
    lst = np.full(len(perm), -1)
    lst[:spare] = perm[at:]
    return table, lst


@pytest.mark.parametrize("B", [1, 2, 31, 257, 1000])
@pytest.mark.parametrize("P", [1, 5, 16, 128])
def test_tables_match_oracle(B, P):
    rng = np.random.default_rng(B * 1000 + P)
    ctx = rng.integers(0, 300, B)
    add = rng.integers(0, 40, B)
    add[rng.random(B) < 0.3] = 0
    add[0] = 700                                         # more pages than a warp writes
    width = -(-1000 // P)
    need = sum(-(-(c + a) // P) - -(-c // P) for c, a in zip(ctx, add))
    for spare in (need + 3, max(1, need // 2), 1):       # enough, half, almost none
        table, lst = random_pool(rng, ctx, P, width, spare)
        t, e, ref = check_extend(ctx, add, table, lst, spare, P, int(add.sum()) + 7)
        keep = np.array([-(-c // P) for c in ctx])
        keep[rng.random(B) < 0.2] = 0
        keep[B // 2] = 10 ** 6 if B > 2 else keep[0]     # past what is held: refused
        dl = dev(lst)
        n, st = sv.release_pages(t, e["new_len"], dev(keep), dl, e["free_count"], P)
        lref, nref, sref = otab.release(ref["block_table"], ref["new_len"], keep, lst,
                                        ref["free_count"], P)
        np.testing.assert_array_equal(num(dl), lref)
        assert n.tolist() == [nref]
        np.testing.assert_array_equal(num(st), sref)


def test_tables_bad_lengths_pages_and_counts():
    P = 4
    ctx, add = [3, -1, 0, 8, 5, 2, 2 ** 31 - 1], [2, 2, -3, 30, 4, 1, 2 ** 31 - 1]
    table = np.array([[9, -1, -1], [0, 0, 0], [0, 0, 0], [0, 1, -1], [-1, 2, -1], [77, 0, 0],
                      [0, 0, 0]])
    lst = [5, 99, 6, 7, -1, -1, -1, -1, -1, -1]
    for cap in (0, 1, 7, 45, 64):
        for count in (-5, 0, 1, 2, 4, 1000):
            check_extend(ctx, add, table, lst, count, P, cap)
    check_extend([], [], np.zeros((0, 3)), lst, 4, P, 5)      # no sequence: slots are -1
    check_extend([0, 0], [0, 0], np.full((2, 1), -1), lst, 4, P, 0)
    # releases: bad lengths, a table entry that is no page, a list without room
    for count in (-1, 0, 7, 9, 10):
        dl, tab = dev(lst), dev(table)
        args = ([3, -1, 9, 12, 13, 0, 4], [0, 0, 2, 1, 0, 1, 0])
        n, st = sv.release_pages(tab, dev(args[0]), dev(args[1]), dl, dev([count]), P)
        lref, nref, sref = otab.release(table, *args, lst, count, P)
        np.testing.assert_array_equal(num(dl), lref)
        assert n.tolist() == [nref]
        np.testing.assert_array_equal(num(st), sref)


def test_tables_largest_batch_and_many_tokens():
    rng = np.random.default_rng(5)
    B, P = 8192, 16
    ctx, add = rng.integers(0, 50, B), rng.integers(0, 9, B)
    table, lst = random_pool(rng, ctx, P, 5, 6000)
    check_extend(ctx, add, table, lst, 6000, P, int(add.sum()))
    table, lst = random_pool(rng, [17], P, 20000, 20000)       # one sequence, 300 K tokens
    check_extend([17], [300000], table, lst, 20000, P, 300000)


# ------------------------------------------------------------------ packed append
@pytest.mark.parametrize("new,cache", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"),
                                       ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("layout", ["dense", "pairs", "heads first"])
def test_append_tokens_matches_oracle(new, cache, D, layout):
    check_append(new, cache, D, layout, 37, 11)


@pytest.mark.parametrize("new,cache,D", [("bf16", "e4m3", 128), ("f16", "f16", 64)])
def test_append_tokens_many_tokens(new, cache, D):
    check_append(new, cache, D, "dense", 1301, 300)    # an odd number, two to a block


def check_append(new, cache, D, layout, T, pages):
    rng = np.random.default_rng(D + len(new) + len(layout))
    Hq, Hkv, P = 6, 2, 5
    g = torch.Generator().manual_seed(D)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g).to(TYPES[new])
    scale = [torch.rand(Hkv, generator=g) * 0.01 + 0.01 for _ in range(2)] \
        if cache == "e4m3" else [None, None]
    shape = {"dense": (pages, P, Hkv, D), "pairs": (pages, 2, P, Hkv, D),
             "heads first": (pages, Hkv, P, D)}[layout]
    mem = [torch.randn(shape, generator=g).to(TYPES[cache]).to(DEV) for _ in range(2)]
    if layout == "pairs":          # K and V of a page side by side in one tensor
        kc, vc = mem[0][:, 0], mem[0][:, 1]
    else:
        kc, vc = (m if layout == "dense" else m.transpose(1, 2) for m in mem)
    before = [num(kc), num(vc)]
    slots = rng.permutation(pages * P)[:T].astype(np.int64)
    slots[[3, 9]] = -1
    slots[20] = pages * P          # past the cache: skipped
    pos = rng.integers(0, 2 ** 20, T)
    pos[5] = -2                    # no position: skipped
    q, k, v = (x.view(T, -1, D) for x in qkv.to(DEV).split([Hq * D, Hkv * D, Hkv * D], 1))
    q_out = torch.full((T, Hq, D), 7.0, dtype=TYPES[new], device=DEV)
    got = sv.append_tokens(k, v, kc, vc, dev(slots, torch.int64), dev(pos), q=q, q_out=q_out,
                           k_scale=None if scale[0] is None else scale[0].to(DEV),
                           v_scale=None if scale[1] is None else scale[1].to(DEV))
    assert got is q_out
    qn, kn, vn = (num(x) for x in (q, k, v))
    sc = [None if s is None else num(s) for s in scale]
    kref, vref = oapp.append_tokens(*before, kn, vn, slots, pos, P, 10000.0, *sc)
    live = [t for t in range(T) if 0 <= slots[t] < pages * P and pos[t] >= 0]
    at = (slots[live] // P, slots[live] % P)
    rest = np.ones((pages, P), bool)
    rest[at] = False
    for c, ref, b in ((kc, kref, before[0]), (vc, vref, before[1])):
        np.testing.assert_array_equal(num(c)[rest], b[rest])

    def near(got, ref, mag, half, floor=0.0):
        lim = half * np.abs(ref) + 2.0 ** -21 * mag + floor
        assert (np.abs(got - ref) <= lim).all(), np.abs(got - ref).max()

    def pairs(x):                  # |a| + |b| of each rotated pair
        a = np.abs(x[..., :D // 2]) + np.abs(x[..., D // 2:])
        return np.concatenate([a, a], -1)

    lim448 = (lambda x: np.clip(x, -448, 448)) if cache == "e4m3" else (lambda x: x)
    floor = 2.0 ** -10 if cache == "e4m3" else 0.0
    mag = pairs(kn[live]) if sc[0] is None else pairs(kn[live]) / sc[0][:, None]
    near(num(kc)[at], lim448(kref[at]), mag, HALF[cache], floor)
    if sc[1] is None:
        np.testing.assert_array_equal(num(vc)[at], vref[at])
    else:
        near(num(vc)[at], lim448(vref[at]), np.abs(vref[at]), HALF[cache], floor)
    near(num(q_out)[live], oapp.rope(qn[live], pos[live]), pairs(qn[live]), HALF[new])
    skipped = [t for t in range(T) if t not in live]
    assert (num(q_out)[skipped] == 7.0).all()


def test_append_tokens_in_place_far_positions_saturation_and_nan():
    D = 128
    x = torch.randn((4, 1, D), generator=torch.Generator().manual_seed(0)).half().to(DEV)
    pos = dev([2 ** 31 - 1, 131072, 1, 0])
    kc, vc = (torch.zeros((1, 4, 1, D), dtype=torch.float16, device=DEV) for _ in range(2))
    q = x.clone()
    out = sv.append_tokens(x, x, kc, vc, dev([0, 1, 2, 3], torch.int64), pos, q=q, q_out=q,
                           rope_base=500000.0)
    assert out is q and torch.equal(q, kc[0])      # the same rotation; position 0: as it was
    assert torch.equal(q[3], x[3])
    ref = oapp.rope(num(x), num(pos), 500000.0)
    # at 2^31 positions the angle's own 64-bit frequency is 2^-24 turns off: 2^-21 of the pair
    assert np.abs(num(q) - ref).max() <= 2.0 ** -11 * np.abs(ref).max() + 2.0 ** -20 * 8
    # without rotation: no positions, values beyond e4m3 limited, NaN stays NaN
    big = torch.full((1, 1, 64), 1e4, dtype=torch.bfloat16, device=DEV)
    big[0, 0, 1], big[0, 0, 2], big[0, 0, 3] = -1e4, float("nan"), float("inf")
    c8 = [torch.zeros((1, 1, 1, 64), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    sv.append_tokens(big, big, *c8, dev([0], torch.int64), rope_base=0)
    for c in c8:
        row = num(c)[0, 0, 0]
        assert row[0] == 448 and row[1] == -448 and np.isnan(row[2]) and row[3] == 448
    sv.append_tokens(big[:0], big[:0], *c8, dev([], torch.int64), rope_base=0)   # no rows


def test_append_tokens_slots_past_32_bits():
    """More slots than 2^32, on pages that share one page's memory."""
    base = [torch.zeros((1, 4096, 1, 64), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    kc, vc = (b.expand(1 << 20, 4096, 1, 64) for b in base)
    x = torch.randn((3, 1, 64), generator=torch.Generator().manual_seed(1)).half().to(DEV)
    slots = [2 ** 32 - 5, 2 ** 31 + 7, 2 ** 32]          # the last is past the cache
    sv.append_tokens(x, x, kc, vc, dev(slots, torch.int64), rope_base=0)
    want = np.zeros((4096, 64))
    want[4091], want[7] = oapp.e4m3(num(x[0, 0])), oapp.e4m3(num(x[1, 0]))
    for b in base:
        np.testing.assert_array_equal(num(b)[0, :, 0], want)


# ------------------------------------------------------------------ one-token attention
def attention_bound(ref, big, mass, lse, n, D, q_half, cache):
    """What rounding can do.  A score is a sum of D exact products in fp32 (D 2^-23 of the
    largest sum of magnitudes `big`, at most); scaling, the subtraction and ex2 add
    2^-22 of the score's size and 2^-21.  P is two bf16 (2^-16), or one fp16 (2^-11; 2^-32 of
    the row's largest weight where it is subnormal).  Sums of n weights in fp32 over tiles of
    16 and at most 64 parts: (n / 16 + 128) 2^-23.  All of it relative to sum p |v| (`mass`);
    the output is rounded once."""
    score = D * 2.0 ** -23 * big + 2.0 ** -22 * (big + 16) + 2.0 ** -21
    sums = (n / 16 + 128) * 2.0 ** -23
    p = 2.0 ** -16 if cache == "bf16" else 2.0 ** -11 + n * 2.0 ** -32
    rel = 2 * score + 2 * sums
    out = q_half * np.abs(ref) + (p + rel)[..., None] * mass * (1 + q_half) + 2.0 ** -25
    return out, score + sums + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def make_cache(lens, Hkv, D, P, cache, seed, spare=3, extra=0):
    """Shuffled pages with NaN wherever no token is stored; (k, v, table, scales)."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    lens = [max(0, n) for n in lens]
    width = max(1, max(-(-n // P) for n in lens)) + extra
    total = sum(-(-n // P) for n in lens) + spare
    perm, at = rng.permutation(total), 0
    table = np.full((len(lens), width), -1)
    stored = np.zeros((total, P), bool)
    for b, n in enumerate(lens):
        k = -(-n // P)
        table[b, :k] = perm[at:at + k]
        for t in range(n):
            stored[table[b, t // P], t % P] = True
        at += k
    scale = [torch.rand(Hkv, generator=g) * 0.01 + 0.01 for _ in range(2)] \
        if cache == "e4m3" else [None, None]
    out = []
    for s in scale:
        x = torch.randn((total, P, Hkv, D), generator=g)
        if s is not None:
            x = (x / s[:, None]).clamp(-448, 448)
        x[torch.from_numpy(~stored)] = float("nan")
        out.append(x.to(TYPES[cache]))
    return out[0], out[1], table, scale


def stands_for(c, s):
    x = num(c)
    return x if s is None else x * num(s)[:, None]


def check_decode(q, k, v, table, lens, scale, cache, qt, window=0, sm_scale=None, **kw):
    lens = np.asarray(lens)
    D = q.shape[2]
    args = [q.to(DEV), k.to(DEV), v.to(DEV), dev(table), dev(lens)]
    if scale[0] is not None:
        kw.update(k_scale=scale[0].to(DEV), v_scale=scale[1].to(DEV))
    out, lse = sv.decode_attn(*args, window=window, scale=sm_scale or 0.0, **kw)
    ref, lref, big, mass = odec.decode_attention(num(q), stands_for(k, scale[0]),
                                                 stands_for(v, scale[1]), table,
                                                 np.maximum(lens, 0), sm_scale, window)
    n = np.maximum(lens, 1)[:, None] if window == 0 else np.minimum(np.maximum(lens, 1),
                                                                    window)[:, None]
    tol, ltol = attention_bound(ref, big, mass, lref, n, D, HALF[qt], cache)
    o, l = num(out), num(lse)
    np.testing.assert_array_equal(np.isfinite(l), np.isfinite(lref))
    assert (l[~np.isfinite(lref)] == -np.inf).all()
    fin = np.isfinite(lref)
    assert (np.abs(l[fin] - lref[fin]) <= ltol[fin]).all()
    over = np.abs(o - ref) - tol
    assert (over <= 0).all(), (np.unravel_index(over.argmax(), over.shape), np.abs(o - ref).max())
    return out, lse


LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 130, 517, -4, 1025]


@pytest.mark.parametrize("qt,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"),
                                      ("f16", "e4m3")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G,Hkv", [(1, 3), (4, 2), (8, 1), (9, 1), (16, 2), (20, 1)])
def test_decode_attn_matches_oracle(qt, cache, D, G, Hkv):
    P = {64: 16, 128: 5, 256: 24}[D]
    k, v, table, sc = make_cache(LENS, Hkv, D, P, cache, D + G)
    q = torch.randn((len(LENS), G * Hkv, D),
                    generator=torch.Generator().manual_seed(G)).to(TYPES[qt])
    check_decode(q, k, v, table, LENS, sc, cache, qt)


@pytest.mark.parametrize("P", [1, 3, 8, 16, 64, 100])
@pytest.mark.parametrize("window", [0, 1, 7, 64, 100, 5000])
def test_decode_attn_pages_and_windows(P, window):
    lens = [300, 0, 99, 64, 1, 7, 8, 411]
    k, v, table, sc = make_cache(lens, 2, 64, P, "f16", P + window, extra=2)
    q = torch.randn((len(lens), 8, 64), generator=torch.Generator().manual_seed(P)).half()
    check_decode(q, k, v, table, lens, sc, "f16", "f16", window=window)


@pytest.mark.parametrize("qt,cache,B,n", [("bf16", "bf16", 1, 20000), ("f16", "e4m3", 2, 33333),
                                          ("bf16", "e4m3", 300, 200), ("f16", "f16", 130, 0)])
def test_decode_attn_splits(qt, cache, B, n):
    """Long sequences cut over all the GPU, more sequences than a block has threads, and a
    batch in which only one of 130 sequences sees anything."""
    rng = np.random.default_rng(n)
    lens = [n] * B if B < 100 else (rng.integers(0, n, B) if n else [0] * 77 + [5000] + [0] * 52)
    k, v, table, sc = make_cache(lens, 2, 128, 16, cache, n)
    q = torch.randn((B, 8, 128), generator=torch.Generator().manual_seed(B)).to(TYPES[qt])
    check_decode(q, k, v, table, lens, sc, cache, qt, sm_scale=0.2)


@pytest.mark.parametrize("D,G,lens", [(64, 3, [40000, 0, 100, 39000, 5]), (256, 8, [30001]),
                                      (128, 16, [9000, 20000, 64]), (128, 40, [50000])])
def test_decode_attn_one_kv_head_over_the_whole_gpu(D, G, lens):
    """Sequences cut into more parts than one CTA joins, beside short and idle ones."""
    k, v, table, sc = make_cache(lens, 1, D, 32, "bf16", D + G)
    q = torch.randn((len(lens), G, D), generator=torch.Generator().manual_seed(D)).bfloat16()
    check_decode(q, k, v, table, lens, sc, "bf16", "bf16")
    check_decode(q, k, v, table, lens, sc, "bf16", "bf16", window=8000)


def test_decode_attn_large_scores_and_masked_garbage():
    """Scores that grow along the sequence (the reference moves again and again), queries at
    the ends of bf16's range beside an 8-bit cache, Inf and NaN behind the sequences."""
    lens, D = [700, 700], 128
    k, v, table, sc = make_cache(lens, 1, D, 16, "bf16", 9)
    ramp = torch.zeros_like(k)
    for t in range(700):
        for b in range(2):
            ramp[table[b, t // 16], t % 16] = k[table[b, t // 16], t % 16] * 0.1 + t * 0.05
    q = torch.ones((2, 4, D), dtype=torch.bfloat16)
    check_decode(q, torch.where(k.isnan(), k, ramp), v, table, lens, sc, "bf16", "bf16")
    k8, v8, table, sc = make_cache(lens, 1, D, 16, "e4m3", 10)
    for size in (1e-30, 1e30, 0.0):
        q = (torch.randn((2, 4, D), generator=torch.Generator().manual_seed(3)) * size).bfloat16()
        check_decode(q, k8, v8, table, lens, sc, "e4m3", "bf16",
                     sm_scale=1.0 / size if size else 1.0)


def test_decode_attn_nan_and_inf_that_are_seen_and_pages_that_are_not():
    k, v, table, sc = make_cache([100, 100, 100], 1, 64, 16, "f16", 11)
    q = torch.randn((3, 2, 64), generator=torch.Generator().manual_seed(1)).half()
    k[table[0, 2], 3, 0, 5] = float("nan")
    bad = table.copy()
    bad[1, 1], bad[1, 3] = -1, 10 ** 6              # not pages: their positions are not seen
    out, lse = sv.decode_attn(q.to(DEV), k.to(DEV), v.to(DEV), dev(bad), dev([100] * 3))
    assert out[0].isnan().all() and lse[0].isnan().all() and not out[1:].isnan().any()
    ref, lref, _, _ = odec.decode_attention(num(q), num(k), num(v), bad, [0, 100, 100])
    np.testing.assert_allclose(num(out)[1:], ref[1:], atol=2e-3)
    np.testing.assert_allclose(num(lse)[1:], lref[1:], atol=1e-5)
    none = np.full_like(table, -1)                  # no page at all: zeros and -inf
    out, lse = sv.decode_attn(q.to(DEV), k.to(DEV), v.to(DEV), dev(none), dev([100] * 3))
    assert (out == 0).all() and (lse == -float("inf")).all()
    # lengths past the table's row: as long as the row
    two = sv.decode_attn(q[1:].contiguous().to(DEV), k.to(DEV), v.to(DEV),
                         dev(table[1:, :3]), dev([2 ** 31 - 1, 48]))
    ref, _, _, _ = odec.decode_attention(num(q[1:]), num(k), num(v), table[1:, :3], [48, 48])
    np.testing.assert_allclose(num(two[0]), ref, atol=2e-3)


@pytest.mark.parametrize("layout", ["pairs", "heads first"])
def test_decode_attn_strided_caches_and_queries(layout):
    lens, Hkv, D, P = [77, 300, 5], 2, 128, 8
    k, v, table, sc = make_cache(lens, Hkv, D, P, "bf16", 21)
    q = torch.randn((3, 8, D), generator=torch.Generator().manual_seed(2)).bfloat16()
    a, la = sv.decode_attn(q.to(DEV), k.to(DEV), v.to(DEV), dev(table), dev(lens))
    if layout == "pairs":
        both = torch.stack([k, v], 1).to(DEV)
        kd, vd = both[:, 0], both[:, 1]
    else:
        kd, vd = (x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) for x in (k, v))
    wide = torch.randn((3, 3, 8, D), dtype=torch.bfloat16, device=DEV)
    wide[:, 1] = q.to(DEV)                          # a slice of a fused projection
    b, lb = sv.decode_attn(wide[:, 1], kd, vd, dev(table), dev(lens))
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_decode_attn_offsets_past_32_bits():
    """A cache whose last pages lie more than 2^32 bytes behind its first."""
    P, Hkv, D = 64, 8, 128
    pages = (2 ** 32 + 2 ** 28) // (P * Hkv * D * 2)
    k, v = (torch.zeros((pages, P, Hkv, D), dtype=torch.float16, device=DEV) for _ in range(2))
    g = torch.Generator().manual_seed(4)
    rows = torch.randn((2, 2, P, Hkv, D), generator=g).half()
    at = [pages - 1, pages - 2]
    k[at], v[at] = rows[0].to(DEV), rows[1].to(DEV)
    q = torch.randn((1, 16, D), generator=g).half()
    out, lse = sv.decode_attn(q.to(DEV), k, v, dev([at]), dev([2 * P]))
    ref, lref, big, mass = odec.decode_attention(num(q), num(rows[0]), num(rows[1]),
                                                 np.array([[0, 1]]), [2 * P])
    tol, ltol = attention_bound(ref, big, mass, lref, np.array([[2 * P]]), D, 2.0 ** -11, "f16")
    assert (np.abs(num(out) - ref) <= tol).all() and (np.abs(num(lse) - lref) <= ltol).all()
    # and stored there by slot
    new = torch.randn((1, Hkv, D), generator=g).half().to(DEV)
    sv.append_tokens(new, new, k, v, dev([pages * P - 1], torch.int64), rope_base=0)
    assert torch.equal(k[-1, -1], new[0]) and torch.equal(v[-1, -1], new[0])


@pytest.mark.parametrize("B,Hkv,G", [(2, 700, 1), (5000, 1, 2), (3, 5, 7)])
def test_decode_attn_many_heads_and_sequences(B, Hkv, G):
    """More KV heads than blocks fit the GPU, thousands of sequences, odd head counts."""
    lens = np.random.default_rng(B).integers(0, 40, B)
    k, v, table, sc = make_cache(lens, Hkv, 64, 16, "f16", B)
    q = torch.randn((B, Hkv * G, 64), generator=torch.Generator().manual_seed(B)).half()
    check_decode(q, k, v, table, lens, sc, "f16", "f16")


def test_calls_on_a_stream_of_their_own():
    """stream=: work and outputs belong to that stream; the current one is left alone."""
    s = torch.cuda.Stream()
    ctx, add = [5, 0, 30], [3, 20, 1]
    table, lst = random_pool(np.random.default_rng(1), ctx, 8, 6, 9)
    ins = [dev(x) for x in (ctx, add, table, lst, [9])]
    kc, vc = (torch.zeros((15, 8, 2, 64), dtype=torch.float16, device=DEV) for _ in range(2))
    x = torch.randn((24, 2, 64), device=DEV).half()
    keep = dev([0, 0, 0])
    torch.cuda.synchronize()
    e = sv.extend_tables(*ins, 8, 24, stream=s)
    sv.append_tokens(x, x, kc, vc, e["slot_map"], e["positions"], stream=s)
    out, _ = sv.decode_attn(x[:3], kc, vc, ins[2], e["new_len"], stream=s)
    n, st = sv.release_pages(ins[2], e["new_len"], keep, ins[3], e["free_count"], 8,
                             stream=s)
    s.synchronize()
    ref = otab.extend(ctx, add, table, lst, 9, 8, 24)
    np.testing.assert_array_equal(num(e["slot_map"]), ref["slot_map"])
    assert n.tolist() == [ref["free_count"] + 1 + 3 + 4]
    want, _, _, _ = odec.decode_attention(num(x[:3]), num(kc), num(vc), num(ins[2]), [8, 20, 31])
    assert np.abs(num(out) - want).max() < 2e-3


def test_decode_attn_on_two_streams_at_once():
    """Calls that run side by side, each stream with a workspace of its own, give what they
    give alone."""
    cases = []
    for i, (Hkv, lens) in enumerate([(2, [9000, 300, 4000]), (1, [20000, 64])]):
        k, v, table, _ = make_cache(lens, Hkv, 128, 16, "f16", 60 + i)
        q = torch.randn((len(lens), 8, 128), generator=torch.Generator().manual_seed(i)).half()
        cases.append([x.to(DEV) for x in (q, k, v)] + [dev(table), dev(lens)])
    alone = [sv.decode_attn(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ws = [sv.new_workspace(sv.decode_attn_workspace_size(3, 8, h, 128), DEV) for h in (2, 1)]
    torch.cuda.synchronize()
    outs = [[] for _ in cases]
    for _ in range(20):
        for c, st, w, o in zip(cases, streams, ws, outs):
            o.append(sv.decode_attn(*c, workspace=w, stream=st))
    torch.cuda.synchronize()
    for (a, la), got in zip(alone, outs):
        for b, lb in got:
            assert torch.equal(a, b) and torch.equal(la, lb)


def test_decode_attn_one_workspace_for_all_shapes_and_streams():
    """Calls of other shapes on one workspace, one after the other; the same call again gives
    the same bits; a call on a stream of its own."""
    ws = sv.new_workspace(max(sv.decode_attn_workspace_size(1, h, hk, d) for h, hk, d in
                              ((8, 2, 64), (16, 1, 128), (8, 1, 256))), DEV)
    kept = []
    for rep in range(2):
        for i, (Hq, Hkv, D, lens) in enumerate([(8, 2, 64, [3000, 70, 0]), (16, 1, 128, [9000]),
                                                (8, 1, 256, [100] * 40), (8, 2, 64, [64] * 9)]):
            k, v, table, sc = make_cache(lens, Hkv, D, 16, "f16", i)
            q = torch.randn((len(lens), Hq, D), generator=torch.Generator().manual_seed(i)).half()
            o, l = check_decode(q, k, v, table, lens, sc, "f16", "f16", workspace=ws)
            if rep:
                assert torch.equal(o, kept[i][0]) and torch.equal(l, kept[i][1])
            kept.append((o, l))
    s = torch.cuda.Stream()
    args = [q.to(DEV), k.to(DEV), v.to(DEV), dev(table), dev(lens)]
    torch.cuda.synchronize()
    o, l = sv.decode_attn(*args, stream=s)
    s.synchronize()
    assert torch.equal(o, kept[-1][0])


def test_bindings_refuse():
    bf, i32 = torch.bfloat16, torch.int32
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    q, k, t, n = z(2, 4, 64), z(3, 16, 2, 64), z(2, 2, dtype=i32), z(2, dtype=i32)

    def refuses(match, f, *a, **kw):
        with pytest.raises((ValueError, sv.SpecError), match=match):
            f(*a, **kw)
    d = sv.decode_attn
    refuses("bf16 or fp16", d, q.float(), k, k, t, n)
    refuses("caches must be", d, q, k.half(), k.half(), t, n)
    refuses("one dtype", d, q, k, k.half(), t, n)
    refuses("both alike", d, q, k, k[:2], t, n)
    refuses("same strides", d, q, k, k.transpose(1, 2).contiguous().transpose(1, 2), t, n)
    refuses("head_dim", d, z(2, 4, 128), k, k, t, n)
    refuses("seq_len", d, q, k, k, t, n[:1])
    refuses("contiguous", d, q, k, k, z(2, 4, dtype=i32)[:, ::2], n)
    refuses("contiguous over D", d, z(2, 64, 4).transpose(1, 2), k, k, t, n)
    refuses("scales belong", d, q, k, k, t, n, k_scale=z(2, dtype=torch.float32))
    refuses("workspace", d, q, k, k, t, n, workspace=z(4096))
    refuses("SPEC_EINVAL", d, q, k, k, t, n, workspace=sv.new_workspace(1024, DEV))
    refuses("SPEC_EINVAL", d, z(2, 3, 64), k, k, t, n)              # 3 heads over 2
    refuses("out has shape", d, q, k, k, t, n, out=z(2, 4, 128))
    refuses("must be a tensor on", d, q, k, k, t.cpu(), n)
    a, s = sv.append_tokens, z(5, dtype=torch.int64)
    x = z(5, 2, 64)
    refuses("positions are needed", a, x, x, k, k, s)
    refuses("side by side", a, z(5, 64, 2).transpose(1, 2), x, k, k, s, rope_base=0)
    refuses("slot_map", a, x, x, k, k, s.int(), rope_base=0)
    refuses("same rows", a, x, x[:4], k, k, s, rope_base=0)
    refuses("q_out without q", a, x, x, k, k, s, q_out=x, rope_base=0)
    refuses("SPEC_EINVAL", a, x, x, k, k, s, z(5, dtype=i32), rope_base=0.5)
    e = sv.extend_tables
    lst, cnt = z(8, dtype=i32), z(1, dtype=i32)
    refuses("add_len", e, n, n[:1], t, lst, cnt, 16, 4)
    refuses("block_table", e, n, n, t[:1], lst, cnt, 16, 4)
    refuses("free_count", e, n, n, t, lst, z(2, dtype=i32), 16, 4)
    refuses("page_size", e, n, n, t, lst, cnt, 0, 4)
    refuses("page_size", e, n, n, t, lst, cnt, 2 ** 32 + 16, 4)
    refuses("max_tokens", e, n, n, t, lst, cnt, 16, -1)
    refuses("window", d, q, k, k, t, n, window=2 ** 32)
    refuses("window", d, q, k, k, t, n, window=-1)
    left = e(n, n, t, lst, cnt, 16, 4)
    refuses("SPEC_EINVAL", e, n, n, t, lst, left["free_count"], 16, 4, out=left)
    refuses("SPEC_EINVAL", e, left["new_len"], n, t, lst, cnt, 16, 4, out=left)
    refuses("slot_map has shape", e, n, n, t, lst, cnt, 16, 5, out=left)
    refuses("out must be the dict", e, n, n, t, lst, cnt, 16, 4, out=[])
    refuses("out has no slot_map", e, n, n, t, lst, cnt, 16, 4, out={})
    refuses("must be a tensor on", e, n, [1, 2], t, lst, cnt, 16, 4)
    for bad in ("x", None, 1.5):
        with pytest.raises(TypeError):
            e(n, n, t, lst, cnt, bad, 4)
    with pytest.raises(OverflowError):
        e(n, n, t, lst, cnt, 2 ** 70, 4)
    refuses("page_size", sv.release_pages, t, n, n, lst, cnt, 0)
    refuses("SPEC_EINVAL", sv.release_pages, t, n, n, lst, cnt, 16, total=cnt)


# ------------------------------------------------------------------ a run of them together
def test_draft_steps_in_a_captured_graph():
    """Prompts, then single-token steps of a drafter with an 8-bit cache: tables, slots,
    rotation, store and attention of every step replayed from ONE captured graph whose
    lengths live on the GPU; an idle row in the batch."""
    B, Hq, Hkv, D, P, pool, steps = 4, 8, 2, 64, 8, 64, 7
    g = torch.Generator(device=DEV).manual_seed(5)
    scale = torch.full((Hkv,), 0.02, device=DEV)
    kc, vc = (torch.zeros((pool, P, Hkv, D), dtype=torch.float8_e4m3fn, device=DEV)
              for _ in range(2))
    table = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    lst = torch.randperm(pool, generator=g, device=DEV).int()
    ctx, count = dev([0] * B), dev([pool])
    prompts = [13, 8, 0, 21]
    T = sum(prompts) + 6
    rows = torch.randn((3, T, Hq, D), generator=g, device=DEV).half()
    e = sv.extend_tables(ctx, dev(prompts), table, lst, count, P, T)
    sv.append_tokens(rows[1, :, :Hkv].contiguous(), rows[2, :, :Hkv].contiguous(), kc, vc,
                     e["slot_map"], e["positions"], k_scale=scale, v_scale=scale)
    assert e["status"].tolist() == [0] * 4 and e["slot_map"][-6:].tolist() == [-1] * 6
    ctx.copy_(e["new_len"])
    count.copy_(e["free_count"])
    add = dev([1, 1, 0, 1])                       # the third row stays idle
    fed = torch.zeros((3, B, Hq, D), dtype=torch.float16, device=DEV)
    q_rot = torch.zeros((B, Hq, D), dtype=torch.float16, device=DEV)
    ws = sv.new_workspace(sv.decode_attn_workspace_size(B, Hq, Hkv, D), DEV)
    live = torch.tensor([0, 1, 3], device=DEV)    # rows of the packed step

    def step():
        e = sv.extend_tables(ctx, add, table, lst, count, P, B)
        sv.append_tokens(fed[1, :, :Hkv], fed[2, :, :Hkv], kc, vc, e["slot_map"], e["positions"],
                         q=fed[0], q_out=q_rot, k_scale=scale, v_scale=scale)
        q = torch.zeros_like(q_rot)
        q[live] = q_rot[:3]
        seen = torch.where(add > 0, e["new_len"], 0)
        out, lse = sv.decode_attn(q, kc, vc, table, seen, k_scale=scale, v_scale=scale,
                                  workspace=ws)
        ctx.copy_(e["new_len"])
        count.copy_(e["free_count"])
        return q, out, lse, e["status"]

    side = torch.cuda.Stream()
    saved = [x.clone() for x in (ctx, count, table, kc.view(torch.uint8), vc.view(torch.uint8))]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                    # warm-up
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((ctx, count, table, kc.view(torch.uint8), vc.view(torch.uint8)), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, out, lse, status = step()
    lens = list(prompts)
    for i in range(steps):
        fed.copy_(torch.randn((3, B, Hq, D), generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        lens = [n + a for n, a in zip(lens, (1, 1, 0, 1))]
        assert ctx.tolist() == lens and status.tolist() == [0] * 4
        assert count.tolist() == [pool - sum(-(-n // P) for n in lens)]
        want = oapp.rope(num(fed[0]), np.array([lens[0], lens[1], lens[3], 1]) - 1)[:3]
        assert np.abs(num(q)[[0, 1, 3]] - want).max() <= 2.0 ** -11 * 6 + 1e-5
        seen = [lens[0], lens[1], 0, lens[3]]
        ref, lref, big, mass = odec.decode_attention(
            num(q), stands_for(kc, scale), stands_for(vc, scale), num(table), seen)
        tol, ltol = attention_bound(ref, big, mass, lref, np.full((B, 1), 32), D, 2.0 ** -11,
                                    "e4m3")
        assert (np.abs(num(out) - ref) <= tol).all()
        assert (num(lse)[2] == -np.inf).all() and (num(out)[2] == 0).all()
    # every page is held once: the tables and the list share none
    held = [p for b, n in enumerate(lens) for p in table[b, :-(-n // P)].tolist()]
    free = lst[:count.item()].tolist()
    assert sorted(held + free) == list(range(pool))


def test_a_verify_round_on_built_tables():
    """Pages and slots, prompts, the block, the verify attention, acceptance, commit and
    release: what the verify step reads is what the tables built, and the rejected pages
    are back on the list."""
    B, R, Hq, Hkv, D, P, pool, V = 3, 5, 8, 2, 128, 16, 40, 64
    g = torch.Generator(device=DEV).manual_seed(8)
    kc, vc = (torch.zeros((pool, P, Hkv, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.zeros((B, 8), dtype=torch.int32, device=DEV)
    lst = torch.randperm(pool, generator=g, device=DEV).int()
    prompts = [30, 62, 15]
    new = lambda T, H: torch.randn((T, H, D), generator=g, device=DEV).bfloat16()  # noqa: E731
    e = sv.extend_tables(dev([0] * B), dev(prompts), table, lst, dev([pool]), P, 107)
    kp, vp = new(107, Hkv), new(107, Hkv)
    sv.append_tokens(kp, vp, kc, vc, e["slot_map"], e["positions"])
    ctx = e["new_len"]
    f = sv.extend_tables(ctx, dev([R] * B), table, lst, e["free_count"], P, B * R)
    kb, vb, qb = (new(B * R, H).view(B, R, H, D) for H in (Hkv, Hkv, Hq))
    st = sv.append_block(kb, vb, kc, vc, table, ctx, q=qb)
    assert st.tolist() == [0] * B
    # the same rows by slot land in the same places
    k2, v2 = kc.clone(), vc.clone()
    sv.append_tokens(kb.view(B * R, Hkv, D), vb.view(B * R, Hkv, D), k2, v2, f["slot_map"],
                     f["positions"])
    assert torch.equal(vc, v2) and (num(kc) - num(k2)).__abs__().max() <= 2.0 ** -8 * 6
    out, _ = sv.verify_attn(qb, kc, vc, table, ctx, None)
    masks = np.array([[(1 << (i + 1)) - 1 for i in range(R)]] * B, dtype=np.uint64)
    ref, _ = verify_attention(num(qb), num(kc), num(vc), num(table), np.array(prompts), masks)
    assert np.abs(num(out) - ref).max() < 2e-2
    # the block's last row is the one-token attention over everything stored
    one, _ = sv.decode_attn(qb[:, -1], kc, vc, table, f["new_len"])
    assert np.abs(num(one) - ref[:, -1]).max() < 2e-2
    w = wl.make_sampler_inputs(wl.Spec("round", B=B, Hq=Hq, Hkv=Hkv, D=D, V=V, ctx=(1, 1),
                                       gamma=R - 1, seed=3), seed=3)
    res = sv.accept_sample(w.logits.to(DEV), w.draft_probs.to(DEV), w.draft_tokens.to(DEV),
                           w.uniforms.to(DEV), sv.SamplerConfig())
    acc = osm.accept_chain_batch(w.logits.numpy(), w.draft_probs.numpy(),
                                 w.draft_tokens.numpy(), w.uniforms.numpy(), osm.SamplerCfg())
    assert res["accepted_len"].tolist() == acc["accepted_len"].tolist()
    new_len, keep, st = sv.kv_commit(kc, vc, table, ctx, res["accepted_len"], R=R)
    count, st = sv.release_pages(table, f["new_len"], keep, lst, f["free_count"], P)
    assert st.tolist() == [0] * B
    want = [n + 1 + int(a) for n, a in zip(prompts, acc["accepted_len"])]
    assert new_len.tolist() == want
    held = [p for b in range(B) for p in table[b, :-(-want[b] // P)].tolist()]
    free = lst[:count.item()].tolist()
    assert sorted(held + free) == list(range(pool))
