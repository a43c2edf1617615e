"""A verify step over an 8-bit cache that scales itself: cases, plain forms and exact values.

Four operators that such a step runs one after the other:

  rotate   rotate: queries and keys turned for their positions -- halves or
           neighbours paired, part of the head, frequencies scaled for long contexts;
  cache    append_scaled and read_scaled: packed keys (turned) and values stored in an
           e4m3 cache whose scales, one per block of tokens and head, come from what is
           stored; the rows read back as the values they stand for;
  attn     verify_attn_scaled: the block of a chain or a draft tree, or single tokens,
           against that cache;
  logits   logits_process: repetition, frequency and presence penalties over each row's
           own prefix, biases and grammar masks, in front of the acceptance sampler.

`run` computes them in plain torch operations (32-bit arithmetic), or with the
package's calls where `own` is set.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3_MAX = 448.0
LEAST = -64  # exponent of the scale of a block that holds only zeros


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the rows of a batched verify step: neighbours paired over half of the head,
        # frequencies below a wavelength stretched eight times
        dict(name="rotate verify block, half of the head", op="rotate", T=320, Hq=32, Hkv=8, D=128,
             new="bf16", rot=64, interleaved=True, scaling="parts", factor=8.0),
        # prompts of a long-context model
        dict(name="rotate prompts", op="rotate", T=16384, Hq=32, Hkv=8, D=128, new="bf16",
             rot=128, interleaved=False, scaling="ntk", factor=4.0),
        # one token per sequence of a serving batch, each into a block that holds others
        dict(name="cache draft step", op="cache", B=64, lo=64, hi=2048, add=1, Hq=32, Hkv=8,
             D=128, new="bf16", page=16, block=16, rot=128, interleaved=False, pad=0),
        # an odd model's verify block: small heads, short blocks in long pages, padded rows
        dict(name="cache verify block, odd", op="cache", B=77, lo=0, hi=2000, add=13, Hq=12, Hkv=4,
             D=64, new="f16", page=24, block=8, rot=32, interleaved=True, pad=23),
        # ragged prompts behind contexts that are already stored
        dict(name="cache prompts", op="cache", B=16, lo=0, hi=400, add=1024, Hq=32, Hkv=8, D=128,
             new="bf16", page=64, block=64, rot=128, interleaved=False, pad=0),
        # single tokens of a drafter of small heads with a sliding window, some rows idle
        dict(name="attn single tokens, window", op="attn", B=37, lo=0, hi=4099, R=1, tree=False,
             Hq=16, Hkv=4, D=64, q="f16", page=24, block=8, window=1000),
        # one request: an anchor and seven drafts at 8192 tokens
        dict(name="attn one chain", op="attn", B=1, lo=8192, hi=8192, R=8, tree=False, Hq=32,
             Hkv=8, D=128, q="bf16", page=16, block=16, window=0),
        # a serving batch of ragged contexts, an anchor and four drafts each
        dict(name="attn chain batch", op="attn", B=64, lo=512, hi=16384, R=5, tree=False, Hq=32,
             Hkv=8, D=128, q="bf16", page=16, block=16, window=0),
        # draft trees of 64 nodes on long contexts, eight query heads to a key-value head
        dict(name="attn draft trees", op="attn", B=4, lo=32768, hi=32768, R=64, tree=True, Hq=64,
             Hkv=8, D=128, q="bf16", page=64, block=32, window=0),
        # one long context and a long chain
        dict(name="attn long chain", op="attn", B=1, lo=131072, hi=131072, R=16, tree=False,
             Hq=64, Hkv=8, D=128, q="f16", page=128, block=64, window=0),
        # one request's chain: bf16 logits of the last layer, biases and a grammar
        dict(name="logits one chain", op="logits", B=1, R=8, tree=False, V=128256, H=500,
             logits="bf16", n_bias=300, mask=1.0, allow=0.02, penalties=True),
        # a serving batch: penalties over long histories, a grammar on a quarter of the requests
        dict(name="logits batch", op="logits", B=64, R=5, tree=False, V=152064, H=4099,
             logits="f32", n_bias=17, mask=0.25, allow=0.3, penalties=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "cache", "attn", "attn", "logits"])
    new = rng.choice(["bf16", "f16"])
    if op == "logits":
        B, R, V = _log(rng, 1, 64), _log(rng, 1, 64), _log(rng, 1000, 172032)
        R = max(1, min(R, 320 * 152064 // (B * V)))
        return dict(op=op, B=B, R=R, tree=R > 1 and rng.random() < 0.5, V=V, H=_log(rng, 1, 8192),
                    logits=rng.choice(["bf16", "f16", "f32"]), n_bias=rng.choice([0, 3, 100, 300]),
                    mask=rng.choice([0.0, 0.5, 1.0]), allow=rng.choice([0.001, 0.3, 0.9]),
                    penalties=rng.random() < 0.8)
    Hkv, G = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    D = rng.choice([64, 128, 128, 256])
    rot, inter = rng.choice([D, D, D // 2, D // 4]), rng.random() < 0.4
    if op == "rotate":
        T = min(_log(rng, 1, 16384), 16384 * 40 * 128 // ((G + 1) * Hkv * D))
        return dict(op=op, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, new=rng.choice([new, "f32"][:1 + (T < 8000)]),
                    rot=rot, interleaved=inter, scaling=rng.choice(["none", "linear", "ntk", "parts"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 32.0]))
    page, block = rng.choice([(1, 1), (5, 5), (16, 16), (16, 8), (24, 12), (32, 32), (64, 16),
                              (64, 64), (128, 64)])
    if op == "cache":
        B = _log(rng, 1, 300)
        add = max(1, min(_log(rng, 1, 2000), 16384 * 48 * 128 // (B * (G + 2) * Hkv * D)))
        hi = min(_log(rng, 1, 2000), 200000 // B)
        return dict(op=op, B=B, lo=rng.choice([0, hi, hi // 3]), hi=hi, add=add, Hq=G * Hkv,
                    Hkv=Hkv, D=D, new=new, page=page, block=block, rot=rot, interleaved=inter,
                    pad=rng.choice([0, 0, 9]))
    B, hi = _log(rng, 1, 96), _log(rng, 1, 32768)
    R = rng.choice([1, 1, 2, 4, 5, 8, 13, 16, 33, 64])
    G = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if R * g <= 512])
    # no more rows of the cache than the listed batch, no more products than the listed trees
    most = min(500000 * 8 * 128, 4 * 32768 * 512 * 8 * 128 // (R * G))
    hi = max(R, min(hi, most // (B * Hkv * D)))
    lo = rng.choice([hi, R, hi // 2])
    return dict(op=op, B=B, lo=rng.choice([lo, lo, 0]), hi=hi, R=R, tree=R > 1 and rng.random() < 0.5,
                Hq=G * Hkv, Hkv=Hkv, D=D, q=new, page=page, block=block,
                window=rng.choice([0, 0, 0, max(R, hi // 3)]))


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n):
    """n whole numbers over lo .. hi, the same for every seed (their order is not)."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _order(values, r):
    values = list(values)
    r.shuffle(values)
    return values


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _ceil(a, b):
    return -(-a // b)


def _tables(counts, spare, gen):
    """A block table of `counts` pages per sequence out of a shuffled pool, -1 behind them."""
    total = sum(counts)
    perm = torch.randperm(total + spare, generator=gen, device=DEV).int()
    width = max(1, max(counts))
    c = _ints(counts, torch.int64)
    first = torch.cumsum(c, 0) - c
    j = torch.arange(width, device=DEV)
    at = (first[:, None] + j).clamp(max=max(0, total + spare - 1))
    return torch.where(j < c[:, None], perm[at], -1).int()


def _power(x):
    """The smallest 2^k with x / 2^k <= 448."""
    m, e = torch.frexp(x.float())
    k = torch.where(x > 0, torch.where(m <= 0.875, e - 9, e - 8), LEAST).clamp(LEAST, 127)
    return (k.int() + 127 << 23).view(torch.float32)


def _codes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _stored(shape, nb, block, gen):
    """A cache of `shape` [pages, P, Hkv, D] with rows of several magnitudes: codes, scales."""
    n, P, H, D = shape
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty((n, nb, H), device=DEV)
    gain = torch.exp2(torch.randint(-1, 3, (H, D), generator=gen, device=DEV).float() * 0.5)
    step = max(1, (1 << 25) // (P * H * D))
    for i in range(0, n, step):
        x = torch.randn((min(step, n - i), nb, block, H, D), generator=gen, device=DEV) * gain
        s = _power(x.abs().amax((2, 4)))
        codes[i:i + step] = _codes(x / s[:, :, None, :, None]).view(-1, P, H, D)
        scales[i:i + step] = s
    return codes, scales


def _parents(R, tree, r):
    """A parent row: a chain, or up to four children of each node down to depth 6."""
    if not tree:
        return list(range(-1, R - 1))
    parent, depth, at, left = [-1], [0], 0, r.randint(1, 4)
    while len(parent) < R:
        while left == 0 or depth[at] >= 6:
            at += 1
            if at == len(parent):      # everything is at its depth: the root has more
                at, depth[0] = 0, -1 << 30
            left = r.randint(1, 4)
        parent.append(at)
        depth.append(max(0, depth[at]) + 1)
        left -= 1
    # storage order puts a child behind its parent; breadth first it is already
    return parent


def _masks(parent):
    rows = []
    for i, p in enumerate(parent):
        rows.append((rows[p] if p >= 0 else 0) | 1 << i)
    return [m - (1 << 64) if m >> 63 else m for m in rows]


def prepare(case, seed):
    r = random.Random(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case=dict(case))

    def randn(shape, dtype):
        x = torch.empty(shape, dtype=dtype, device=DEV)
        n = max(1, (1 << 26) // max(1, math.prod(shape[1:])))
        for i in range(0, shape[0], n):
            x[i:i + n] = torch.randn((min(n, shape[0] - i),) + tuple(shape[1:]), generator=gen,
                                     device=DEV)
        return x

    if case["op"] == "rotate":
        T, width = case["T"], (case["Hq"] + case["Hkv"]) * case["D"]
        # queries and keys side by side, as a fused projection leaves them
        s["qk"] = randn((T, width), TYPES[case["new"]])
        s["positions"] = torch.randint(0, 131072, (T,), generator=gen, device=DEV).int()
        return s
    if case["op"] == "logits":
        B, R, V, H = case["B"], case["R"], case["V"], case["H"]
        s["logits"] = randn((B * R, V), torch.float32).mul_(3).to(TYPES[case["logits"]]).view(B, R, V)
        # words of a text return: ids are drawn from the cube of a uniform number
        def words(shape):
            u = torch.rand(shape, generator=gen, device=DEV)
            return (u ** 3 * V).int().clamp(max=V - 1)
        s["history"] = words((B, H))
        lens = _ints(_order(_spread(H // 2, H, B), r))
        s["history"][torch.arange(H, device=DEV)[None] >= lens[:, None]] = -1
        s["prompt_len"] = _ints(_order(_spread(0, H // 2, B), r))
        s["parent"] = _ints([_parents(R, True, r) for _ in range(B)]) if case["tree"] else None
        s["block_tokens"] = words((B, R if case["tree"] else R - 1))
        u = torch.rand((3, B), generator=gen, device=DEV)
        on = case["penalties"]
        s["repetition"] = 1 + 0.5 * u[0] if on else None
        s["frequency"], s["presence"] = (0.4 * u[1], u[2] - 0.2) if on else (None, None)
        n = case["n_bias"]
        s["bias_ids"] = s["bias"] = None
        if n:  # distinct ids of a sequence; the rows end ragged
            first = torch.randint(0, V, (B, 1), generator=gen, device=DEV)
            step = max(1, V // n)
            ids = (first + step * torch.arange(n, device=DEV)) % V
            ids[torch.rand((B, n), generator=gen, device=DEV) < 0.1] = -1
            s["bias_ids"] = ids.int()
            s["bias"] = torch.randn((B, n), generator=gen, device=DEV) * 5
        s["mask"] = s["mask_row"] = None
        if case["mask"]:
            rows = [i < max(1, int(case["mask"] * B)) for i in range(B)]
            r.shuffle(rows)
            M = sum(rows) * R
            bits = torch.zeros((M, _ceil(V, 32) * 32), dtype=torch.bool, device=DEV)
            bits[:, :V] = torch.rand((M, V), generator=gen, device=DEV) < case["allow"]
            word = torch.zeros((M, _ceil(V, 32)), dtype=torch.int64, device=DEV)
            for k in range(32):
                word |= bits[:, k::32].long() << k
            s["mask"] = torch.where(word >= 1 << 31, word - (1 << 32), word).int()
            at = iter(range(M))
            s["mask_row"] = _ints([[next(at) if on else -1 for _ in range(R)] for on in rows])
        s["out"] = torch.empty((B, R, V), device=DEV)
        return s
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    P, block, B = case["page"], case["block"], case["B"]
    nb = P // block
    if case["op"] == "cache":
        # every sequence adds `add` tokens on the average to what it holds
        more = _spread(_ceil(case["add"], 2), case["add"] + case["add"] // 2, B)
        pairs = zip(_spread(case["lo"], case["hi"], B), _order(more, random.Random(1)))
        ctx, add = zip(*_order(pairs, r))
        T = sum(add) + case["pad"]
        s["block_table"] = _tables([_ceil(c + a, P) for c, a in zip(ctx, add)], 3, gen)
        c, a = _ints(ctx, torch.int64), _ints(add, torch.int64)
        b = torch.repeat_interleave(torch.arange(B, device=DEV), a)
        pos = c[b] + torch.arange(len(b), device=DEV) - (a.cumsum(0) - a)[b]
        slot = s["block_table"][b, pos // P].long() * P + pos % P
        s["slot_map"] = torch.full((T,), -1, dtype=torch.int64, device=DEV)
        s["positions"] = torch.full((T,), -1, dtype=torch.int32, device=DEV)
        s["slot_map"][:len(b)], s["positions"][:len(b)] = slot, pos.int()
        pages = sum(_ceil(x + y, P) for x, y in zip(ctx, add)) + 3
        for n in "kv":
            s[n + "_cache"], s[n + "_scale"] = _stored((pages, P, Hkv, D), nb, block, gen)
        # rows of several magnitudes, so that some blocks' scales grow
        s["qkv"] = randn((T, (Hq + 2 * Hkv) * D), TYPES[case["new"]])
        loud = torch.exp2(torch.randint(-2, 4, (T, 1), generator=gen, device=DEV).float())
        s["qkv"] *= loud.to(s["qkv"].dtype)
        s["q_out"] = torch.zeros((T, Hq, D), dtype=TYPES[case["new"]], device=DEV)
        for n in "kv":
            s[n + "_read"] = torch.zeros((T, Hkv, D), dtype=torch.bfloat16, device=DEV)
        return s
    # attn: lens tokens are stored, the last R of them the block; shorter ones are idle
    R = case["R"]
    lens = _order(_spread(case["lo"], case["hi"], B), r)
    lens = [n if n >= R else 0 for n in lens]
    s["block_table"] = _tables([_ceil(n, P) for n in lens], 3, gen)
    s["ctx_len"] = _ints([n - R if n else -1 for n in lens])
    s["anc_mask"] = _ints([_masks(_parents(R, True, r)) for _ in range(B)], torch.int64) \
        if case["tree"] else None
    s["q"] = randn((B, R, Hq, D), TYPES[case["q"]])
    pages = sum(_ceil(n, P) for n in lens) + 3
    stored = torch.zeros(pages, P, dtype=torch.bool, device=DEV)
    j = torch.arange(s["block_table"].shape[1], device=DEV)[:, None] * P + torch.arange(P, device=DEV)
    for b, n in enumerate(lens):
        k = _ceil(n, P)
        stored[s["block_table"][b, :k].long()] = j[:k] < n
    for n in "kv":
        codes, scales = _stored((pages, P, Hkv, D), nb, block, gen)
        # what no token was stored to holds anything: here NaN
        codes.view(torch.uint8)[~stored] = 0x7F
        scales[~stored.view(pages, nb, block).any(2)] = math.nan
        s[n + "_cache"], s[n + "_scale"] = codes, scales
    return s


# ------------------------------------------------------------------ plain forms
ORIGINAL, LOW, HIGH, BASE, LOUD = 8192, 1.0, 4.0, 500000.0, 1.1


def _frequencies(c):
    """The pairs' angles per position, in 64 bits."""
    n, base = c["rot"], BASE
    how, factor = c.get("scaling", "none"), c.get("factor", 1.0)
    if how == "ntk":
        base *= factor ** (n / (n - 2))
    f = base ** (-torch.arange(0, n, 2, device=DEV, dtype=torch.float64) / n)
    if how == "linear":
        f = f / factor
    if how == "parts":  # turns within the original context: many stay, few are stretched
        keep = ((ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f


def _turn(c, positions, *rows):
    """rows [T, H, D] in fp32, turned for their positions."""
    n, loud = c["rot"], LOUD if c.get("scaling") == "parts" else 1.0
    angle = positions.double()[:, None] * _frequencies(c)
    cos, sin = (angle.cos() * loud).float()[:, None], (angle.sin() * loud).float()[:, None]
    out = []
    for x in rows:
        if c["interleaved"]:
            a, b = x[..., 0:n:2], x[..., 1:n:2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = x[..., :n // 2], x[..., n // 2:n]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        out.append(torch.cat([y, x[..., n:]], -1))
    return out


def _split(s):
    c = s["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    x = s["qk"] if c["op"] == "rotate" else s["qkv"]
    parts = x.split([Hq * D] + [Hkv * D] * (x.shape[1] // D - Hq) if Hkv == 1 else
                    [Hq * D] + [Hkv * D] * ((x.shape[1] // D - Hq) // Hkv), dim=1)
    return [p.unflatten(1, (-1, D)) for p in parts]


def _plain_store(x, slot, cache, scale):
    """x [T, H, D] in fp32 into the blocks of a cache: codes, scales."""
    n, P, H, D = cache.shape
    nb = scale.shape[1]
    block, live = P // nb, slot >= 0
    at = torch.where(live, slot // block, n * nb)           # blocks lie one after another
    off = torch.where(live, slot % block, 0)
    rows = torch.where(live, slot, n * P)
    big = x.abs().amax(-1)
    need = torch.zeros((n * nb + 1, H), device=x.device)
    need = need.scatter_reduce(0, at[:, None].expand_as(big), big, "amax")[:-1]
    hit = torch.zeros(n * nb + 1, dtype=torch.bool, device=x.device)
    hit[at] = True
    fresh = torch.zeros(n * nb + 1, dtype=torch.bool, device=x.device)
    fresh[torch.where(off == 0, at, n * nb)] = True
    old, hit, fresh = scale.view(n * nb, H), hit[:-1, None], fresh[:-1, None]
    want = _power(need)
    new = torch.where(hit, torch.where(fresh, want, torch.maximum(old, want)), old)
    # what stays in a block is held by its new scale; a block begun anew keeps its bytes
    codes = cache.view(n * nb, block, H, D)
    held = _codes(codes.float() * (old / new)[:, None, :, None])
    grown = (hit & ~fresh & (new > old))[:, None, :, None]
    bits = torch.where(grown, held.view(torch.uint8), codes.view(torch.uint8))
    bits = torch.cat([bits.view(n * P, H, D), bits.view(n * P, H, D)[:1]])
    by = new[torch.where(live, at, 0)]
    bits[rows] = _codes(x / by[:, :, None]).view(torch.uint8)
    return bits[:-1].view(torch.float8_e4m3fn).view(cache.shape), new.view(scale.shape)


def _plain_cache(s):
    c, slot = s["case"], s["slot_map"]
    q, k, v = (x.float() for x in _split(s))
    q, k = _turn(c, s["positions"], q, k)
    live = (slot >= 0)[:, None, None]
    out = dict(q=torch.where(live, q.to(s["q_out"].dtype), s["q_out"]))
    for n, x in (("k", k), ("v", v)):
        codes, scales = _plain_store(x, slot, s[n + "_cache"], s[n + "_scale"])
        out[n + "_cache"], out[n + "_scale"] = codes, scales
        at = slot.clamp(min=0)
        block = c["block"]
        y = codes.view(-1, c["Hkv"], c["D"])[at].float() * \
            scales.view(-1, c["Hkv"])[at // block][:, :, None]
        out[n + "_read"] = torch.where(live, y.to(torch.bfloat16), 0)
    return out


def _plain_attn(s):
    c = s["case"]
    q, table, P = s["q"].float(), s["block_table"].long(), c["page"]
    B, R, Hq, D = q.shape
    Hkv, L, block = c["Hkv"], table.shape[1] * P, c["block"]
    pos = torch.arange(L, device=q.device)
    ctx = s["ctx_len"].long()
    if s["anc_mask"] is None:
        see = torch.ones(R, R, dtype=torch.bool, device=q.device).tril().expand(B, R, R)
    else:
        see = (s["anc_mask"][:, :, None] >> torch.arange(R, device=q.device) & 1).bool()
    see = see & (ctx >= 0)[:, None, None]
    least = ctx[:, None] + see.sum(-1) - c["window"] if c["window"] else ctx[:, None] * 0 + see.sum(-1) * 0
    inside = (pos < ctx[:, None])[:, None] & (pos >= least[:, :, None])          # [B, R, L]
    j = pos[None] - ctx[:, None]
    own_rows = torch.gather(see, 2, j.clamp(0, R - 1)[:, None].expand(B, R, L))
    seen = inside | (own_rows & ((j >= 0) & (j < R))[:, None])
    at = (table.clamp(min=0)[:, :, None] * P + torch.arange(P, device=q.device)).reshape(B, L)

    def rows(name):
        x = s[name + "_cache"].view(-1, Hkv, D)[at].float()
        return x * s[name + "_scale"].view(-1, Hkv)[at // block][..., None]      # [B, L, Hkv, D]
    k = rows("k")
    x = torch.einsum("brhgd,blhd->bhrgl", q.view(B, R, Hkv, -1, D), k) / math.sqrt(D)
    del k
    x = torch.where(seen[:, None, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)                     # a row that sees nothing
    p = torch.exp(x - top)
    del x
    total = p.sum(-1)
    v = torch.where(seen.any(1)[:, :, None, None], rows("v"), 0.0)
    out = torch.einsum("bhrgl,blhd->bhrgd", p, v)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    lse = top[..., 0] + torch.log(total)
    return dict(out=out.permute(0, 2, 1, 3, 4).reshape(B, R, Hq, D).to(s["q"].dtype),
                lse=lse.permute(0, 2, 1, 3).reshape(B, R, Hq))


def _prefix(s):
    """How often each id stands in each row's own block, [B, R, V]; and in front of it, [B, V]."""
    c, h = s["case"], s["history"].long()
    B, R, V = c["B"], c["R"], c["V"]
    tokens = torch.full((B, R), -1, dtype=torch.long, device=h.device)
    if R > 1:
        tokens[:, 1:] = s["block_tokens"].long()[:, (1 if c["tree"] else 0):]
    see = torch.ones(R, R, dtype=torch.bool, device=h.device).tril().repeat(B, 1, 1)
    if c["tree"]:
        see = torch.eye(R, dtype=torch.bool, device=h.device).repeat(B, 1, 1)
        up = torch.zeros(B, R, R, device=h.device).scatter_(
            2, s["parent"].long().clamp(min=0)[..., None], 1.0)
        up[:, 0] = 0
        step = see.float()
        for _ in range(R.bit_length() if R < 8 else 8):   # depth is at most 7
            step = step @ up
            see = see | (step > 0)
    see[:, :, 0] = False
    block = torch.zeros(B, R, V, device=h.device).scatter_add_(
        2, tokens.clamp(min=0)[:, None].expand(B, R, R), (see & (tokens >= 0)[:, None]).float())
    new = torch.arange(h.shape[1], device=h.device) >= s["prompt_len"][:, None]
    said = torch.zeros(B, V, device=h.device).scatter_add_(1, h.clamp(min=0), ((h >= 0) & new).float())
    prompt = torch.zeros(B, V, device=h.device).scatter_add_(1, h.clamp(min=0), ((h >= 0) & ~new).float())
    return block, said, prompt


def _allowed(s):
    V = s["case"]["V"]
    bit = s["mask"][:, :, None].long() >> torch.arange(32, device=DEV) & 1
    bit = bit.flatten(1)[:, :V].bool()
    at = s["mask_row"].long()
    return torch.where((at >= 0)[..., None], bit[at.clamp(min=0)], True)


def _plain_logits(s):
    x = s["logits"].float()
    if s["repetition"] is not None:
        count, said, prompt = _prefix(s)
        count += said[:, None]
        rep = s["repetition"][:, None, None]
        x = torch.where((count + prompt[:, None]) > 0, torch.where(x > 0, x / rep, x * rep), x)
        x = x - s["frequency"][:, None, None] * count
        x = x - s["presence"][:, None, None] * (count > 0).float()
    if s["bias"] is not None:
        ids = s["bias_ids"].long()
        add = torch.zeros((ids.shape[0], x.shape[2]), device=x.device)
        x = x + add.scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, s["bias"], 0.0))[:, None]
    if s["mask"] is not None:
        x = torch.where(_allowed(s), x, -math.inf)
    return x


# ------------------------------------------------------------------ one pass
def _rope(sv, c):
    how = c.get("scaling", "none")
    return sv.Rope(dim=c["rot"], base=BASE, interleaved=c["interleaved"], scaling=how,
                   factor=c.get("factor", 1.0) if how != "none" else 1.0, original_len=ORIGINAL,
                   low=LOW, high=HIGH, magnitude=LOUD if how == "parts" else 1.0)


def run(state):
    op, c = state["case"]["op"], state["case"]
    if own:
        import speculative_decoding_verification_76_gb300 as sv
        if op in ("rotate", "cache") and "rope" not in state:
            state["rope"] = _rope(sv, c)
        if op == "rotate":
            if "q_out" not in state:  # what a serving loop keeps
                state["q_out"] = state["k_out"] = None
            q, k = _split(state)
            state["q_out"], state["k_out"] = sv.rotate(
                q, state["positions"], state["rope"], k=k, q_out=state["q_out"],
                k_out=state["k_out"])
            return dict(q=state["q_out"], k=state["k_out"])
        if op == "cache":
            q, k, v = _split(state)
            caches = (state["k_cache"], state["v_cache"], state["k_scale"], state["v_scale"])
            sv.append_scaled(k, v, *caches, state["slot_map"], state["positions"], q=q,
                             q_out=state["q_out"], rope=state["rope"])
            sv.read_scaled(*caches, state["slot_map"], k_out=state["k_read"],
                           v_out=state["v_read"])
            return dict(q=state["q_out"], k_cache=caches[0], k_scale=caches[2],
                        k_read=state["k_read"], v_cache=caches[1], v_scale=caches[3],
                        v_read=state["v_read"])
        if op == "logits":
            return sv.logits_process(
                state["logits"], out=state["out"], history=state["history"],
                prompt_len=state["prompt_len"], block_tokens=state["block_tokens"],
                parent=state["parent"], repetition=state["repetition"],
                frequency=state["frequency"], presence=state["presence"],
                bias_ids=state["bias_ids"], bias=state["bias"], mask=state["mask"],
                mask_row=state["mask_row"])
        if "workspace" not in state:
            state["workspace"] = sv.new_workspace(
                sv.verify_attn_scaled_workspace_size(c["B"], c["R"], c["Hq"], c["Hkv"], c["D"]),
                state["q"].device)
        out, lse = sv.verify_attn_scaled(
            state["q"], state["k_cache"], state["v_cache"], state["k_scale"], state["v_scale"],
            state["block_table"], state["ctx_len"], state["anc_mask"], window=c["window"],
            workspace=state["workspace"])
        return dict(out=out, lse=lse)
    if op == "rotate":
        q, k = (x.float() for x in _split(state))
        q, k = _turn(c, state["positions"], q, k)
        return dict(q=q.to(state["qk"].dtype), k=k.to(state["qk"].dtype))
    if op == "cache":
        return _plain_cache(state)
    return _plain_logits(state) if op == "logits" else _plain_attn(state)


# ------------------------------------------------------------------ least work
def work(case):
    if case["op"] == "logits":
        B, R, V = case["B"], case["R"], case["V"]
        size = 4 if case["logits"] == "f32" else 2
        masks = max(1, int(case["mask"] * B)) * R * _ceil(V, 32) * 4 if case["mask"] else 0
        return dict(bytes=B * R * V * (size + 4) + masks + 4 * B * (case["H"] + R)
                    + 8 * B * case["n_bias"], flops=0)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "rotate":
        size = 4 if case["new"] == "f32" else 2
        return dict(bytes=case["T"] * ((Hq + Hkv) * D * 2 * size + 4),
                    flops=case["T"] * 3 * (Hq + Hkv) * case["rot"])
    if case["op"] == "cache":
        add = _spread(_ceil(case["add"], 2), case["add"] + case["add"] // 2, case["B"])
        live = sum(add)
        # rows in, queries and codes out; codes in, rows out; the touched blocks' scales
        rows = (Hq + 2 * Hkv) * D * 2 + Hq * D * 2 + 2 * Hkv * D * (1 + 1 + 2)
        blocks = sum(_ceil(a, case["block"]) for a in add)
        return dict(bytes=live * (rows + 20) + blocks * Hkv * 2 * 8,
                    flops=live * 3 * (Hq + Hkv) * case["rot"])
    R, W = case["R"], case["window"]
    lens = [n for n in _spread(case["lo"], case["hi"], case["B"]) if n >= R]
    kept = sum(min(n, W + R - 1) if W else n for n in lens)
    seen = sum(R * (min(n - R, W) if W else n - R) + R * (R + 1) // 2 for n in lens)
    return dict(bytes=kept * 2 * Hkv * (D + 4 / case["block"]) + case["B"] * R * Hq * (4 * D + 4)
                + 4 * sum(_ceil(n, case["page"]) for n in lens), flops=4 * seen * Hq * D)


# ------------------------------------------------------------------ 64 bits
def _exact_turn(c, positions, x):
    """x [T, H, D]: pairs as complex numbers times a number on a circle, in 64 bits."""
    n = c["rot"]
    i = torch.arange(n // 2, device=DEV, dtype=torch.float64)
    how, factor = c.get("scaling", "none"), c.get("factor", 1.0)
    log = math.log(BASE) + (n / (n - 2) * math.log(factor) if how == "ntk" else 0.0)
    f = torch.exp(-2 * i / n * log)
    if how == "linear":
        f = f / factor
    if how == "parts":
        wave = 2 * math.pi / f
        t = torch.clip((ORIGINAL / wave - LOW) / (HIGH - LOW), 0.0, 1.0)
        f = f / factor + t * (f - f / factor)
    size = torch.full((), LOUD if how == "parts" else 1.0, dtype=torch.float64, device=DEV)
    turn = torch.polar(size, positions.double()[:, None, None] * f)
    x = x.double()
    pair = x[..., :n].unflatten(-1, (n // 2, 2)) if c["interleaved"] else \
        x[..., :n].unflatten(-1, (2, n // 2)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    y = y if c["interleaved"] else y.transpose(-1, -2)
    return torch.cat([y.flatten(-2), x[..., n:]], -1)


def _grid(x):
    """x to the nearest e4m3 value (ties to even), limited to +-448, in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(max=8) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return dict(zip("qk", (_exact_turn(case, s["positions"], x) for x in _split(s))))
    if case["op"] == "logits":
        B, R, V = case["B"], case["R"], case["V"]
        x = s["logits"].double()
        if s["repetition"] is not None:
            h, lens, parent = s["history"].tolist(), s["prompt_len"].tolist(), \
                s["parent"].tolist() if case["tree"] else [list(range(-1, R - 1))] * B
            tok = s["block_tokens"].tolist()
            for b in range(B):
                rep, fr, pr = (float(s[n][b]) for n in ("repetition", "frequency", "presence"))
                base, seen = {}, set()
                for at, t in enumerate(h[b]):
                    if t >= 0:
                        seen.add(t)
                        if at >= lens[b]:
                            base[t] = base.get(t, 0) + 1
                for i in range(R):
                    count, v = dict(base), i
                    while v > 0:
                        t = tok[b][v if case["tree"] else v - 1]
                        count[t] = count.get(t, 0) + 1
                        v = parent[b][v]
                    ids = sorted(seen | set(count))
                    if not ids:
                        continue
                    at = _ints(ids, torch.int64)
                    n = torch.tensor([count.get(t, 0) for t in ids], dtype=torch.float64, device=DEV)
                    y = x[b, i, at]
                    y = torch.where(y > 0, y / rep, y * rep) - fr * n - pr * (n > 0)
                    x[b, i, at] = y
        if s["bias"] is not None:
            for b in range(B):
                on = s["bias_ids"][b] >= 0
                x[b, :, s["bias_ids"][b][on].long()] += s["bias"][b][on].double()
        if s["mask"] is not None:
            x.masked_fill_(~_allowed(s), -math.inf)
        return x
    Hkv, D, block = case["Hkv"], case["D"], case["block"]
    if case["op"] == "cache":
        q, k, v = _split(s)
        slot, P = s["slot_map"], case["page"]
        rows = (slot >= 0).nonzero()[:, 0]
        out = dict(q=s["q_out"].double())
        out["q"][rows] = _exact_turn(case, s["positions"], q)[rows]
        at = slot[rows]
        for n, x in (("k", _exact_turn(case, s["positions"], k)), ("v", v.double())):
            scale = s[n + "_scale"].double().view(-1, Hkv).clone()
            codes = s[n + "_cache"].double().view(-1, block, Hkv, D).clone()
            hit, where = torch.unique(at // block, return_inverse=True)
            big = torch.zeros(len(hit), Hkv, dtype=torch.float64, device=DEV)
            big.scatter_reduce_(0, where[:, None].expand(-1, Hkv), x[rows].abs().amax(-1), "amax")
            fresh = torch.zeros(len(hit), dtype=torch.bool, device=DEV)
            fresh[where[at % block == 0]] = True
            m, e = torch.frexp(big / E4M3_MAX)
            want = torch.exp2(torch.where(m == 0.5, e - 1, e).clamp(min=LEAST).double())
            old = scale[hit]
            new = torch.where(fresh[:, None], want, torch.maximum(old, want))
            keep = codes[hit]
            moved = _grid(keep * (old / new)[:, None, :, None])
            codes[hit] = torch.where((fresh[:, None] | (new <= old))[:, None, :, None], keep, moved)
            scale[hit] = new
            codes.view(-1, Hkv, D)[at] = _grid(x[rows] / new[where][..., None])
            out[n + "_cache"] = codes.view(s[n + "_cache"].shape)
            out[n + "_scale"] = scale.view(s[n + "_scale"].shape)
            out[n + "_read"] = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
            out[n + "_read"][rows] = codes.view(-1, Hkv, D)[at] * scale[at // block][..., None]
        return out
    B, R, Hq, P, W = case["B"], case["R"], case["Hq"], case["page"], case["window"]
    G = Hq // Hkv
    out = torch.zeros(B, R, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, R, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, ctx in enumerate(s["ctx_len"].tolist()):
        if ctx < 0:
            continue
        masks = [m % (1 << 64) for m in s["anc_mask"][b].tolist()] if case["tree"] else \
            [(2 << i) - 1 for i in range(R)]
        n = ctx + R
        pages = s["block_table"][b, :_ceil(n, P)].long()
        k, v = ((s[x + "_cache"][pages].double().view(-1, block, Hkv, D)
                 * s[x + "_scale"][pages].double().view(-1, 1, Hkv, 1)).view(-1, Hkv, D)[:n].transpose(0, 1)
                for x in "kv")
        q = s["q"][b].double().view(R, Hkv, G, D).transpose(0, 1).reshape(Hkv, R * G, D)
        x = (q @ k.transpose(1, 2) * D ** -0.5).view(Hkv, R, G, n)
        for i, m in enumerate(masks):
            if W:
                x[:, i, :, :max(0, ctx + bin(m).count("1") - W)] = -math.inf
            gone = [ctx + j for j in range(R) if not m >> j & 1]
            x[:, i, :, gone] = -math.inf
        y = torch.logsumexp(x, -1)
        p = torch.exp(x - y[..., None]).view(Hkv, R * G, n)
        lse[b] = y.permute(1, 0, 2).reshape(R, Hq)
        out[b] = (p @ v).view(Hkv, R, G, D).permute(1, 0, 2, 3).reshape(R, Hq, D)
    return dict(out=out, lse=lse)
