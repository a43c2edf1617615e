"""GPU parity of verify_attn_scaled against the float64 oracle, what masked places may hold, its
refusals, and a verify step over a scaled cache run together.

Tolerances: see bound().
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import rope as orope
from oracle import scaled as osc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def num(t):
    return t.detach().float().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).to(DEV)


def bound(ref, aux, lse, D, half, width):
    """What rounding can do.  A row of q may be held as a sum of 8-bit parts, off by at most
    2^-10 beside a largest element of 224 or more (2^-17 of it): 2^-17 of `edge` on a score.
    The score is a sum of at most 3 D exact products in fp32 (3 D 2^-23 of `big`); scales, the
    logarithm of V's scale, the subtraction and ex2 add 2^-21 (big + 16) and 2^-20.  A weight is
    held in 11 bits (2^-11, on the safe side), and what is below 2^-27 of the row's largest
    may be lost: n 2^-26 of its largest p |v|, times D's spread (the largest |v|).  Sums of n
    weights in fp32 over groups of 16 and at most 512 parts: (n / 16 + 512) 2^-23.  All of it
    relative to sum p |v|; the output is rounded once."""
    n = aux["n"]
    score = 2.0 ** -17 * aux["edge"] + 3 * D * 2.0 ** -23 * aux["big"] + 2.0 ** -21 * (aux["big"] + 16) + 2.0 ** -20
    sums = (n / 16 + 512) * 2.0 ** -23
    rel = 2.0 ** -11 + 2 * score + 2 * sums
    out = half * np.abs(ref) + (rel[..., None] * aux["mass"] + (n * 2.0 ** -26 * aux["peak"])[..., None]) * (1 + half) \
        + 2.0 ** -25
    return out, score + sums + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def tree_masks(R, rng):
    masks = [1]
    for i in range(1, R):
        masks.append(masks[rng.integers(max(0, i - 4), i)] | 1 << i)
    return masks


def chain_masks(R):
    return [(2 << i) - 1 for i in range(R)]


def signed(rows):
    return [[m - (1 << 64) if m >> 63 else m for m in r] for r in rows]


def make_cache(lens, Hkv, D, P, block, seed, spare=3, extra=0, spread=6):
    """Shuffled pages, blocks of different magnitude, NaN wherever no token is stored:
    (codes, scales) of K and V on the GPU, the table, and the values in float64."""
    rng = np.random.default_rng(seed)
    width = max(1, max(-(-max(0, n) // P) for n in lens)) + extra
    total = sum(-(-max(0, n) // P) for n in lens) + spare
    perm, at = rng.permutation(total), 0
    table = np.full((len(lens), width), -1)
    stored = np.zeros((total, P), bool)
    for b, n in enumerate(lens):
        k = -(-max(0, n) // P)
        table[b, :k] = perm[at:at + k]
        for t in range(n):
            stored[table[b, t // P], t % P] = True
        at += k
    nb, out, vals = P // block, [], []
    for i in range(2):
        x = rng.normal(size=(total, nb, block, Hkv, D))
        x *= 2.0 ** rng.integers(-spread, 1 if i else 2, (total, nb, 1, Hkv, 1)) if spread else 1.0
        s = 2.0 ** np.ceil(np.log2(np.abs(x).max((2, 4)) / 448))
        codes = torch.from_numpy(x / s[:, :, None, :, None]).float().reshape(total, P, Hkv, D)
        codes[torch.from_numpy(~stored)] = float("nan")
        codes = codes.to(torch.float8_e4m3fn)
        scales = torch.from_numpy(s).float()
        scales[torch.from_numpy(~stored.reshape(total, nb, block).any(2))] = float("nan")
        out += [codes.to(DEV), scales.to(DEV)]
        vals.append(osc.values(num(codes), num(scales)))
    return (out[0], out[2], out[1], out[3]), vals, table


def check(lens, R, Hq, Hkv, D, P, block, new, seed, tree=False, window=0, masks=None, scale=0.0,
          table_edit=None, extra=0, spread=6, q_scale=1.0):
    rng = np.random.default_rng(seed)
    B = len(lens)
    cache, (k, v), table = make_cache(lens, Hkv, D, P, block, seed, extra=extra, spread=spread)
    if table_edit:
        table_edit(table)
    ctx = [n - R if n >= R else -1 for n in lens]
    if masks is None:
        masks = [tree_masks(R, rng) if tree else chain_masks(R) for _ in range(B)]
    q = torch.from_numpy(rng.normal(size=(B, R, Hq, D)) * q_scale).to(TYPES[new]).to(DEV)
    anc = dev(signed(masks), torch.int64) if tree else None
    out, lse = sv.verify_attn_scaled(q, *cache, dev(table), dev(ctx), anc, scale=scale, window=window)
    ref, rl, aux = osc.attention(num(q), k, v, table, ctx, masks, scale=scale or None, window=window)
    ob, lb = bound(ref, aux, rl, D, HALF[new], table.shape[1] * P)
    err = np.abs(num(out) - ref)
    assert (err <= ob).all(), ("out", (err - ob).max(), np.unravel_index((err - ob).argmax(), err.shape))
    fin = np.isfinite(rl)
    np.testing.assert_array_equal(np.isfinite(num(lse)), fin)
    assert (num(lse)[~fin] == -np.inf).all() and not num(out)[~fin].any()
    le = np.abs(num(lse)[fin] - rl[fin])
    assert (le <= lb[fin]).all(), ("lse", (le - lb[fin]).max())
    return cache, q, table, ctx, anc, out, lse


@pytest.mark.parametrize("D,P,block", [(128, 16, 16), (64, 24, 8), (256, 64, 64), (128, 5, 5), (64, 1, 1),
                                       (256, 128, 32)])
@pytest.mark.parametrize("R,G,Hkv", [(1, 1, 2), (1, 8, 1), (5, 4, 2), (8, 4, 2), (3, 5, 1), (16, 4, 1),
                                     (13, 7, 1)])
@pytest.mark.parametrize("new", ["bf16", "f16"])
def test_chains(D, P, block, R, G, Hkv, new):
    lens = [R, 130 + R, 0, 300, 127 + R, 128 + R, R + 1]
    check(lens, R, G * Hkv, Hkv, D, P, block, new, seed=D + R + G)


@pytest.mark.parametrize("R,G,Hkv,D", [(64, 8, 1, 128), (64, 1, 2, 64), (33, 3, 1, 256), (17, 4, 2, 128),
                                       (2, 16, 1, 128), (64, 5, 1, 64)])
@pytest.mark.parametrize("new", ["bf16", "f16"])
def test_trees(R, G, Hkv, D, new):
    check([R, 200, 0, R + 128], R, G * Hkv, Hkv, D, 16, 8, new, seed=R + G, tree=True)


@pytest.mark.parametrize("R,window", [(1, 1), (1, 100), (5, 5), (5, 131), (8, 400), (16, 17)])
@pytest.mark.parametrize("tree", [False, True])
def test_windows(R, window, tree):
    check([R, 260, 0, 140, 513], R, 4, 2, 64, 24, 12, "bf16", seed=R + window, tree=tree, window=window)


def test_masks_that_leave_rows_empty():
    """Rows without a block position see the committed ones, or nothing where there are none;
    bits behind the block's rows do not count."""
    masks = [[0, 1, 3, 0, 2 ** 64 - 1], [0, 2, 0, 8, 31]]
    check([5, 40], 5, 4, 2, 128, 16, 16, "f16", seed=1, tree=True, masks=masks)


def test_pages_that_are_not_there():
    def edit(table):
        table[0, 1], table[0, 3], table[1, 0], table[2, :] = -1, 10 ** 6, -7, 2 ** 31 - 1
    check([100, 40, 64], 4, 8, 2, 128, 16, 8, "bf16", seed=2, table_edit=edit)
    # a table narrower than the sequence: positions past it are not seen
    cache, q, table, ctx, _, _, _ = check([64, 33], 4, 8, 2, 128, 16, 8, "bf16", seed=3)
    out, lse = sv.verify_attn_scaled(q, *cache, dev(table[:, :2].copy()), dev(ctx))
    k, v = (osc.values(num(cache[i]), num(cache[i + 2])) for i in range(2))
    ref, rl, aux = osc.attention(num(q), k, v, table[:, :2], ctx, [chain_masks(4)] * 2)
    ob, lb = bound(ref, aux, rl, 128, HALF["bf16"], 32)
    assert (np.abs(num(out) - ref) <= ob).all() and (np.abs(num(lse) - rl) <= lb).all()


def test_many_sequences_and_head_groups():
    rng = np.random.default_rng(4)
    check(rng.integers(0, 70, 301).tolist(), 2, 6, 3, 64, 16, 16, "bf16", seed=4)
    check([90, 17], 2, 48, 24, 64, 16, 16, "f16", seed=5)


def test_one_long_sequence():
    check([20000], 4, 4, 1, 128, 64, 64, "bf16", seed=6)
    check([9000, 3], 3, 40, 2, 64, 128, 64, "f16", seed=7, tree=True)


def test_scales_far_apart_and_sharp_scores():
    """Value scales over 2^40, and scores sharp enough that one position has all the weight."""
    check([400, 77], 4, 4, 2, 128, 16, 8, "f16", seed=8, spread=40)
    check([400, 77], 4, 4, 2, 128, 16, 8, "bf16", seed=9, q_scale=30.0)
    check([400, 77], 4, 4, 2, 128, 16, 8, "f16", seed=10, q_scale=1e-3, scale=3.0)


def test_scales_that_are_no_powers_of_two():
    cache, q, table, ctx, _, _, _ = check([200, 50], 4, 8, 2, 128, 16, 8, "f16", seed=11)
    kc, vc, ks, vs = cache
    ks, vs = ks * 1.37, vs * 0.81
    out, lse = sv.verify_attn_scaled(q, kc, vc, ks, vs, dev(table), dev(ctx))
    k, v = osc.values(num(kc), num(ks)), osc.values(num(vc), num(vs))
    ref, rl, aux = osc.attention(num(q), k, v, table, ctx, [chain_masks(4)] * 2)
    ob, lb = bound(ref, aux, rl, 128, HALF["f16"], 0)
    assert (np.abs(num(out) - ref) <= ob).all() and (np.abs(num(lse) - rl) <= lb).all()


def test_a_long_tail_behind_one_position():
    """One position of weight 1 and 30000 whose weights are 2^-20 each: 3 % of the sum, which
    must not be lost."""
    n, D = 30001, 64
    k = torch.zeros((1, n, 1, D)).to(torch.float8_e4m3fn)
    k[0, 0, 0, 0] = 8.0
    v = torch.ones((1, n, 1, D))
    v[0, 0] = 0.0
    q = torch.zeros((1, 1, 1, D), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    one = torch.ones((1, n, 1), device=DEV)
    scale = 20 * np.log(2) / 8
    out, lse = sv.verify_attn_scaled(q.to(DEV), k.to(DEV), v.to(torch.float8_e4m3fn).to(DEV), one, one,
                                     dev([[0]]), dev([n - 1]), scale=scale)
    tail = (n - 1) * 2.0 ** -20
    want = tail / (1 + tail)
    # n 2^-26 of the largest weight may be lost: 2^-6 of the tail
    assert (np.abs(num(out) - want) <= want * (2.0 ** -8 + 2.0 ** -6)).all()
    assert abs(num(lse)[0, 0, 0] - (20 * np.log(2) + np.log1p(tail))) < 1e-4


def test_nan_in_masked_places_stays_there():
    """NaN codes in block rows and window edges that only some rows see."""
    R, ctx, D, P = 6, 150, 128, 16
    cache, (k, v), table = make_cache([ctx + R], 2, D, P, 16, 12, spread=0)
    q = torch.from_numpy(np.random.default_rng(0).normal(size=(1, R, 8, D))).to(torch.bfloat16).to(DEV)
    masks = [[1, 3, 5, 9, 0b10011, 0b100101]]
    for window in (0, 100):
        clean, _ = sv.verify_attn_scaled(q, *cache, dev(table), dev([ctx]), dev(masks, torch.int64),
                                         window=window)
        bad = [x.clone() for x in cache]
        for c in bad[:2]:                       # block row 1 (seen by rows 1 and 4), head 0
            t = ctx + 1
            c.view(torch.uint8)[table[0, t // P], t % P, 0, 5:9] = 0xFF
        if window:                              # the oldest position that rows 0 sees, head 1
            t = ctx + 1 - window
            bad[1].view(torch.uint8)[table[0, t // P], t % P, 1, 64] = 0x7F
        out, lse = sv.verify_attn_scaled(q, *bad, dev(table), dev([ctx]), dev(masks, torch.int64),
                                         window=window)
        hit = np.zeros((R, 8, D), bool)
        hit[[1, 4], :4] = True                  # a NaN score: the whole row
        if window:
            hit[0, 4:, 64] = True               # row 0 alone: a NaN value, that element
        np.testing.assert_array_equal(np.isnan(num(out)[0]), hit)
        assert (num(out)[0][~hit] == num(clean)[0][~hit]).all()
        # values alone: the element of the rows that see it
        bad = [x.clone() for x in cache]
        t = ctx + 2                             # seen by rows 2 and 5
        bad[1].view(torch.uint8)[table[0, t // P], t % P, 0, 77] = 0x7F
        out, lse = sv.verify_attn_scaled(q, *bad, dev(table), dev([ctx]), dev(masks, torch.int64),
                                         window=window)
        hit = np.zeros((R, 8, D), bool)
        hit[[2, 5], :4, 77] = True
        np.testing.assert_array_equal(np.isnan(num(out)[0]), hit)
        assert (num(out)[0][~hit] == num(clean)[0][~hit]).all() and np.isfinite(num(lse)).all()


def test_queries_that_are_not_finite():
    cache, q, table, ctx, _, clean, _ = check([200, 50], 4, 8, 2, 128, 16, 8, "bf16", seed=13)
    q = q.clone()
    q[0, 1, 2, 3], q[1, 3, 7, 0] = float("nan"), float("inf")
    out, _ = sv.verify_attn_scaled(q, *cache, dev(table), dev(ctx))
    hit = np.zeros((2, 4, 8, 128), bool)
    hit[0, 1, 2], hit[1, 3, 7] = True, True
    assert np.isnan(num(out)[hit]).all() and (num(out)[~hit] == num(clean)[~hit]).all()


def test_strided_queries_and_caches():
    cache, q, table, ctx, _, clean, lse = check([150, 40], 3, 4, 2, 64, 16, 8, "f16", seed=14)
    # queries as a slice of a fused projection, the cache heads first inside a wider pool
    wide = torch.zeros((2, 3, 8, 64), dtype=q.dtype, device=DEV)
    wide[:, :, 4:] = q
    pools = []
    for c in cache[:2]:
        pool = torch.zeros((c.shape[0], 3, 2, 16, 64), dtype=torch.uint8, device=DEV)
        pool[:, 1] = c.view(torch.uint8).transpose(1, 2)
        pools.append(pool.view(torch.float8_e4m3fn)[:, 1].transpose(1, 2))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, l2 = sv.verify_attn_scaled(wide[:, :, 4:], *pools, *cache[2:], dev(table), dev(ctx), stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, clean) and torch.equal(l2, lse)
    with pytest.raises(ValueError, match="share memory"):
        sv.verify_attn_scaled(q, *cache, dev(table), dev(ctx), out=q)
    with pytest.raises(ValueError, match="shape"):
        sv.verify_attn_scaled(q, *cache[:3], cache[3][:, :1], dev(table), dev(ctx))
    with pytest.raises(ValueError, match="anc_mask"):
        sv.verify_attn_scaled(q, *cache, dev(table), dev(ctx), dev([[1, 3, 7]] * 2))


def test_captured_graphs_share_a_workspace_and_lengths_change():
    """Two graphs on one workspace, replayed in turn with lengths that change on the GPU."""
    R, Hq, Hkv, D, P = 4, 8, 2, 128, 16
    lens = [300, 64, 7]
    cache, (k, v), table = make_cache([400] * 3, Hkv, D, P, 16, 15, spread=0)
    ws = sv.new_workspace(sv.verify_attn_scaled_workspace_size(3, R, Hq, Hkv, D), DEV)
    ctx, q = dev([0, 0, 0]), torch.randn((3, R, Hq, D), device=DEV).bfloat16()
    q2 = torch.randn((3, 1, Hq, D), device=DEV).bfloat16()
    graphs = []
    for x in (q, q2):
        g = torch.cuda.CUDAGraph()
        sv.verify_attn_scaled(x, *cache, dev(table), ctx, workspace=ws)
        t = dev(table)
        with torch.cuda.graph(g):
            o = sv.verify_attn_scaled(x, *cache, t, ctx, workspace=ws)
        graphs.append((g, x, o, t))
    for lens in ([300, 64, 7], [4, 396, -1], [100, 0, 396]):
        ctx.copy_(dev(lens))
        for g, *_ in graphs:
            g.replay()
        for _, x, (out, lse), _ in graphs:
            a, b = sv.verify_attn_scaled(x, *cache, dev(table), ctx)
            assert torch.equal(out, a) and torch.equal(lse, b)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("tree", [False, True])
def test_a_verify_step_on_a_scaled_cache(tree):
    """Prompts, then two rounds of: tables, append, attention, served logits, acceptance,
    commit, release -- all from lengths on the GPU, against the oracle's view of the cache."""
    torch.manual_seed(3)
    B, R, Hq, Hkv, D, P, block, V = 3, 6, 8, 2, 64, 16, 8, 50
    pages, width = 40, 12
    z = dict(dtype=torch.int32, device=DEV)
    table = torch.full((B, width), -1, **z)
    pool = torch.randperm(pages).int().to(DEV)
    kc = torch.zeros((pages, P, Hkv, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    vc, ks = kc.clone(), torch.zeros((pages, P // block, Hkv), device=DEV)
    vs = ks.clone()
    rope = sv.Rope(32, 1e4, interleaved=True, scaling="parts", factor=4.0, original_len=64.0)
    freqs = orope.frequencies(32, 1e4, "parts", 4.0, 64.0)
    parent = dev([[-1, 0, 0, 1, 1, 3]] * B) if tree else None
    said = [[] for _ in range(B)]               # every stored (position, key, value), by sequence
    ctx, count = torch.zeros(B, **z), dev([pages])

    def store(add, pos=None):
        nonlocal ctx, count
        T = int(sum(add)) + 2
        e = sv.extend_tables(ctx, dev(add), table, pool, count, P, T)
        k = torch.randn((T, Hkv, D), device=DEV).bfloat16()
        v, q = torch.randn_like(k), torch.randn((T, Hq, D), device=DEV).bfloat16()
        at = e["positions"] if pos is None else pos
        qr = sv.append_scaled(k, v, kc, vc, ks, vs, e["slot_map"], at, q=q, rope=rope)
        return e, k, v, qr

    def truth(ctx):
        return osc.values(num(kc), num(ks)), osc.values(num(vc), num(vs))

    prompts = [20, 3, 9]
    e, *_ = store(prompts)
    ctx, count = e["new_len"], e["free_count"]
    for step in range(2):
        depth = [0, 1, 1, 2, 2, 3] if tree else list(range(R))
        pos = torch.cat([(ctx[:, None] + dev(depth)).flatten(), dev([-1, -1])]).int()
        e, k, v, q = store([R] * B, pos)
        mask = sv.tree_prepare(parent, ctx)[0] if tree else None
        out, lse = sv.verify_attn_scaled(q[:B * R].view(B, R, Hq, D), kc, vc, ks, vs, table, ctx, mask)
        masks = [[int(m) for m in r] for r in mask.tolist()] if tree else [chain_masks(R)] * B
        kk, vv = truth(ctx)
        ref, rl, aux = osc.attention(num(q[:B * R]).reshape(B, R, Hq, D), kk, vv, num(table), num(ctx), masks)
        ob, lb = bound(ref, aux, rl, D, HALF["bf16"], 0)
        assert (np.abs(num(out) - ref) <= ob).all() and (np.abs(num(lse) - rl) <= lb).all()
        # keys in the cache are the turned ones, within e4m3's half step of the block's scale
        slots = num(e["slot_map"])[:B * R]
        want = orope.turn(num(k)[:B * R], num(pos)[:B * R], freqs, True)
        got = kk.reshape(-1, Hkv, D)[slots]
        scale = num(ks).reshape(-1, Hkv)[slots // block][..., None]
        assert (np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 2.0 ** -18) + scale * 2.0 ** -9).all()
        # the served logits feed the sampler
        x = torch.randn((B, R, V), device=DEV).bfloat16()
        toks = torch.randint(0, V, (B, R if tree else R - 1), device=DEV).int()
        allowed = torch.full((1, 2), -1, **z)
        served = sv.logits_process(x, history=torch.randint(0, V, (B, 5), device=DEV).int(), block_tokens=toks,
                                   parent=parent, presence=torch.full((B,), 0.5, device=DEV), mask=allowed,
                                   mask_row=torch.zeros((B, R), **z))
        cfg, u = sv.SamplerConfig(greedy=True), torch.rand((B, R), device=DEV)
        if tree:
            res = sv.accept_sample_tree(served, None, toks, parent, u, cfg)
            path = res["path"]
        else:
            res, path = sv.accept_sample(served, None, toks, u, cfg), None
        if step == 0 and tree:                 # a path that moves rows, whatever was accepted
            res["accepted_len"], path = dev([3, 1, 0]), dev([[1, 3, 5, -1, -1, -1], [2] + [-1] * 5, [-1] * 6])
        before = osc.values(num(kc), num(ks)), osc.values(num(vc), num(vs))
        tab, c0 = num(table), num(ctx)
        ctx, keep, status = sv.kv_commit(kc, vc, table, ctx, res["accepted_len"], path, parent if tree else None,
                                         R=R, k_scale=ks, v_scale=vs)
        assert not status.any()
        if tree:
            for b, a in enumerate(res["accepted_len"].tolist()):
                for j in range(a):
                    src, dst = int(c0[b]) + int(path[b, j]), int(c0[b]) + j + 1
                    for old, c, s in zip(before, (kc, vc), (ks, vs)):
                        now = osc.values(num(c), num(s))[tab[b, dst // P], dst % P]
                        at = num(s)[tab[b, dst // P], dst % P // block][:, None]
                        assert (np.abs(now - old[tab[b, src // P], src % P]) <= at * 2.0 ** -10).all()
        count, _ = sv.release_pages(table, e["new_len"], keep, pool, e["free_count"], P)
