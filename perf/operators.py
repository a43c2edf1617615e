"""The cache side of a decoding step: cases, plain forms and exact values.

Three operators that run one after the other around the verify step, on the
same paged key-value cache:

  tables   extend_tables and release_pages: pages for a step's new tokens taken
           from a free list, the block tables, slot map and positions built from
           the requests' lengths, and the pages behind the kept tokens given back;
  append   append_tokens: a packed batch's keys and values rotated for their
           positions and stored at their slots (16-bit or e4m3 cache), the
           queries rotated;
  decode   decode_attn: attention of one new token per sequence over the cache.

`run` computes them in plain torch operations (32-bit arithmetic), or with the
package's calls where `own` is set.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0
BAD_LEN, NO_PAGES = 16, 32  # bits of a sequence's status


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token per sequence: a drafter's step of a serving batch
        dict(name="tables draft step", op="tables", B=64, lo=512, hi=16384, add_lo=1, add_hi=1,
             keep=1, page=16, pool=1.0, finish=0.0),
        # a verify step's block of five rows over many requests, one in thirty finishing,
        # with a pool that runs out before the last requests
        dict(name="tables verify step, short pool", op="tables", B=1000, lo=1, hi=4099, add_lo=5,
             add_hi=5, keep=2, page=16, pool=0.9, finish=0.03),
        # prompts of ragged length, some of them not there, added to their contexts
        dict(name="tables ragged prompts", op="tables", B=200, lo=0, hi=2000, add_lo=0,
             add_hi=1309, keep=2000, page=32, pool=1.0, finish=0.1),
        # the block of a batched verify step: 64 sequences x 5 rows
        dict(name="append verify block", op="append", T=320, Hq=32, Hkv=8, D=128, new="bf16",
             cache="bf16", rope=10000.0, pad=0.0),
        # an odd number of tokens of a small drafter, padded as for a captured graph
        dict(name="append odd, D 64", op="append", T=1001, Hq=12, Hkv=4, D=64, new="f16",
             cache="f16", rope=500000.0, pad=0.1),
        # prompts into an 8-bit cache
        dict(name="append prompts, e4m3", op="append", T=16384, Hq=32, Hkv=8, D=128, new="bf16",
             cache="e4m3", rope=500000.0, pad=0.0),
        # a drafter of small heads with a sliding window, idle rows among the batch
        dict(name="decode window, D 64", op="decode", B=37, lo=0, hi=4099, Hq=16, Hkv=4, D=64,
             q="f16", cache="f16", page=5, window=1000),
        # one request at 8192 tokens
        dict(name="decode one request", op="decode", B=1, lo=8192, hi=8192, Hq=32, Hkv=8, D=128,
             q="bf16", cache="bf16", page=16, window=0),
        # a serving batch of ragged contexts in 16 and in 8 bits
        dict(name="decode batch", op="decode", B=64, lo=512, hi=16384, Hq=32, Hkv=8, D=128,
             q="bf16", cache="bf16", page=16, window=0),
        dict(name="decode batch, e4m3", op="decode", B=64, lo=512, hi=16384, Hq=32, Hkv=8, D=128,
             q="bf16", cache="e4m3", page=16, window=0),
        # one long context, eight query heads to a key-value head
        dict(name="decode long, e4m3", op="decode", B=1, lo=131072, hi=131072, Hq=64, Hkv=8,
             D=128, q="f16", cache="e4m3", page=64, window=0),
        # wide heads, all of them on one key-value head
        dict(name="decode one KV head, D 256", op="decode", B=24, lo=1000, hi=32768, Hq=8, Hkv=1,
             D=256, q="bf16", cache="bf16", page=24, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "decode"])
    if op == "tables":
        B, page = _log(rng, 1, 2000), rng.choice([1, 5, 8, 16, 24, 32, 64, 128])
        add_hi = min(_log(rng, 1, 4096), max(1, 200000 // B))
        hi = min(_log(rng, 1, 32768), 4000000 // B)
        return dict(op=op, B=B, lo=rng.randint(0, hi), hi=hi, add_lo=rng.randint(0, add_hi),
                    add_hi=add_hi, keep=rng.randint(0, add_hi), page=page,
                    pool=rng.choice([1.0, 1.0, 0.5, 0.9]), finish=rng.choice([0.0, 0.05, 0.5]))
    Hkv, G, D = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 12, 16]), \
        rng.choice([64, 128, 128, 256])
    new = rng.choice(["bf16", "f16"])
    cache = rng.choice([new, "e4m3"])
    if op == "append":
        T = min(_log(rng, 1, 16384), (16384 * 48 * 128) // ((G + 2) * Hkv * D))
        return dict(op=op, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, new=new, cache=cache,
                    rope=rng.choice([0.0, 10000.0, 500000.0]), pad=rng.choice([0.0, 0.0, 0.2]))
    B, hi = _log(rng, 1, 96), _log(rng, 1, 32768)
    hi = max(1, min(hi, 500000 * 8 * 128 // (B * Hkv * D)))
    lo = rng.choice([hi, 0, hi // 20, hi // 2])
    return dict(op=op, B=B, lo=lo, hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, q=new, cache=cache,
                page=rng.choice([1, 5, 8, 16, 16, 24, 32, 64, 128]),
                window=rng.choice([0, 0, 0, 1 + hi // 3]))


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


def _randn(shape, dtype, gen, scale=None):
    """N(0, 1) in `dtype`; for e4m3 what is stored for it under the heads' scales."""
    x = torch.empty(shape, dtype=TYPES[dtype], device=DEV)
    n = max(1, (1 << 26) // max(1, x[0].numel())) if shape[0] else 1
    for i in range(0, shape[0], n):
        y = torch.randn((min(n, shape[0] - i),) + tuple(shape[1:]), generator=gen, device=DEV)
        if scale is not None:
            y = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        x[i:i + n] = y.to(x.dtype)
    return x


def _scales(Hkv, cache, gen):
    if cache != "e4m3":
        return None
    return torch.empty(Hkv, device=DEV).uniform_(0.011, 0.014, generator=gen)


def _tables(counts, spare, r, gen):
    """A block table of `counts` pages per sequence out of a shuffled pool, -1 behind
    them, and the `spare` pages that are left."""
    total = sum(counts)
    perm = torch.randperm(total + spare, generator=gen, device=DEV).int()
    width = max(1, max(counts))
    c = _ints(counts, torch.int64)
    first = torch.cumsum(c, 0) - c
    j = torch.arange(width, device=DEV)
    at = (first[:, None] + j).clamp(max=max(0, total + spare - 1))
    table = torch.where(j < c[:, None], perm[at], -1).int()
    return table, perm[total:].contiguous()


def prepare(case, seed):
    r = random.Random(seed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case=dict(case))
    if case["op"] == "tables":
        P, B = case["page"], case["B"]
        # requests of every length get every number of new tokens; the seed sets their order
        pairs = zip(_spread(case["lo"], case["hi"], B),
                    _order(_spread(case["add_lo"], case["add_hi"], B), random.Random(1)))
        ctx, add = zip(*_order(pairs, r))
        had = [_ceil(c, P) for c in ctx]
        need = sum(_ceil(c + a, P) - h for c, a, h in zip(ctx, add, had))
        free = max(1, int(need * case["pool"]))
        table, rest = _tables(had, free, r, gen)
        width = max(1, max(_ceil(c + a, P) for c, a in zip(ctx, add)))
        s["block_table"] = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        w = min(width, table.shape[1])
        s["block_table"][:, :w] = table[:, :w]
        s["free_list"] = torch.full((sum(had) + free,), -1, dtype=torch.int32, device=DEV)
        s["free_list"][:free] = rest
        s["free_count"] = _ints([free])
        done = [i < int(case["finish"] * B) for i in range(B)]
        r.shuffle(done)
        s["ctx_len"], s["add_len"] = _ints(ctx), _ints(add)
        s["keep_pages"] = _ints([0 if d else _ceil(c + min(a, case["keep"]), P)
                                 for c, a, d in zip(ctx, add, done)])
        s["max_tokens"] = _ceil(sum(add) + 1, 64) * 64
        return s
    Hq, Hkv, D, cache = case["Hq"], case["Hkv"], case["D"], case["cache"]
    s["k_scale"], s["v_scale"] = _scales(Hkv, cache, gen), _scales(Hkv, cache, gen)
    if case["op"] == "append":
        T, P = case["T"], 16
        pages = _ceil(T, P) + 3
        # queries, keys and values side by side, as a fused projection leaves them
        s["qkv"] = _randn((T, (Hq + 2 * Hkv) * D), case["new"], gen)
        s["k_cache"] = _randn((pages, P, Hkv, D), cache, gen, s["k_scale"])
        s["v_cache"] = _randn((pages, P, Hkv, D), cache, gen, s["v_scale"])
        slots = torch.randperm(pages * P, generator=gen, device=DEV)[:T]
        live = T - int(case["pad"] * T)  # a captured step's rows behind the last request
        s["slot_map"] = torch.where(torch.arange(T, device=DEV) < live, slots, -1)
        s["positions"] = torch.randint(0, 131072, (T,), generator=gen, device=DEV).int()
        s["q_out"] = torch.zeros((T, Hq, D), dtype=TYPES[case["new"]], device=DEV)
        return s
    P, B = case["page"], case["B"]
    lens = _order(_spread(case["lo"], case["hi"], B), r)
    s["block_table"], _ = _tables([_ceil(n, P) for n in lens], 3, r, gen)
    s["seq_len"] = _ints(lens)
    pages = sum(_ceil(n, P) for n in lens) + 3
    s["q"] = _randn((B, Hq, D), case["q"], gen)
    stored = torch.zeros(pages, P, dtype=torch.bool, device=DEV)
    j = torch.arange(s["block_table"].shape[1], device=DEV)[:, None] * P + torch.arange(P, device=DEV)
    for b, n in enumerate(lens):
        k = _ceil(n, P)
        stored[s["block_table"][b, :k].long()] = j[:k] < n
    for name in ("k_cache", "v_cache"):
        c = _randn((pages, P, Hkv, D), cache, gen, s[name[0] + "_scale"])
        # what no token was stored to holds anything: here NaN
        bits, nan = (torch.uint8, 0x7F) if cache == "e4m3" else (torch.int16, 0x7FFF)
        c.view(bits)[~stored] = nan
        s[name] = c
    return s


# ------------------------------------------------------------------ plain forms
def _plain_tables(s):
    c = s["case"]
    P, (B, width), cap = c["page"], s["block_table"].shape, s["max_tokens"]
    pool = s["free_list"].shape[0]
    ctx, add = s["ctx_len"].long(), s["add_len"].long()
    cu = torch.cat([add.new_zeros(1), add.clamp(min=0).cumsum(0)])
    have, want = (ctx + P - 1) // P, (ctx + add + P - 1) // P
    bad = (ctx < 0) | (add < 0) | (want > width) | (cu[1:] > cap)
    need = torch.where(bad, 0, want - have)
    upto = need.cumsum(0)
    count = s["free_count"].long()
    short = ~bad & (need > 0) & (upto > count)
    served = ~bad & ~short
    taken = (need * served).sum()
    # block table: new page k of the step is the k-th from the free list's end
    j = torch.arange(width, device=ctx.device)
    new = served[:, None] & (j >= have[:, None]) & (j < want[:, None])
    k = (upto - need)[:, None] + j - have[:, None]
    page = s["free_list"][(count - 1 - k).clamp(0, pool - 1)]
    table = torch.where(new, page, s["block_table"])
    # one row per token: its sequence, its place in it, its slot
    t = torch.arange(cap, device=ctx.device)
    starts = torch.zeros(cap + 1, dtype=torch.long, device=ctx.device)
    starts.index_add_(0, cu[1:].clamp(max=cap), torch.ones_like(ctx))
    b = starts.cumsum(0)[:cap].clamp(max=B - 1)
    pos = ctx[b] + t - cu[b]
    on = served[b] & (t < cu[-1])
    page = table[b, torch.where(on, pos // P, 0)].long()
    on = on & (page >= 0) & (page < pool)
    slot = torch.where(on, page * P + pos % P, -1)
    status = BAD_LEN * bad.int() + NO_PAGES * short.int()
    new_len = torch.where(served, ctx + add, ctx).int()
    out = dict(block_table=table, slot_map=slot, positions=torch.where(on, pos, -1).int(),
               cu_len=cu.int(), new_len=new_len, left=(count - taken).int(),
               status=status.int())
    # the pages behind the kept ones go back on the list
    keep, held = s["keep_pages"].long(), (new_len.long() + P - 1) // P
    bad = (keep < 0) | (keep > held)
    n = torch.where(bad, 0, held - keep)
    upto = n.cumsum(0)
    count = count - taken
    full = ~bad & (n > 0) & (upto + count > pool)
    go = ~bad & ~full
    give = go[:, None] & (j >= keep[:, None]) & (j < held[:, None])
    at = torch.where(give, count + (upto - n)[:, None] + j - keep[:, None], pool)
    listed_ = torch.cat([s["free_list"], s["free_list"].new_zeros(1)])
    listed_[at.reshape(-1)] = table.reshape(-1)
    out.update(free_list=listed_[:pool], free_count=(count + (n * go).sum()).int(),
               released=(BAD_LEN * bad.int() + NO_PAGES * full.int()).int())
    return out


def _split(s):
    c = s["case"]
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    q, k, v = s["qkv"].split([Hq * D, Hkv * D, Hkv * D], dim=1)
    return q.view(T, Hq, D), k.view(T, Hkv, D), v.view(T, Hkv, D)


def _plain_append(s):
    c = s["case"]
    q, k, v = (x.float() for x in _split(s))
    D, half = c["D"], c["D"] // 2
    if c["rope"]:
        i = torch.arange(half, device=q.device, dtype=torch.float64)
        angle = s["positions"].double()[:, None] * c["rope"] ** (-2.0 * i / D)
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        q, k = (torch.cat([x[..., :half] * cos - x[..., half:] * sin,
                           x[..., :half] * sin + x[..., half:] * cos], -1) for x in (q, k))
    slot = s["slot_map"]
    live = (slot >= 0)[:, None, None]
    out = dict(q=torch.where(live, q.to(s["q_out"].dtype), s["q_out"]))
    for name, x in (("k_cache", k), ("v_cache", v)):
        cache = s[name]
        if c["cache"] == "e4m3":
            x = (x / s[name[0] + "_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        # rows without a slot go to a row behind the cache
        bits = torch.uint8 if c["cache"] == "e4m3" else torch.int16
        flat = cache.view(bits).reshape((-1,) + tuple(cache.shape[2:]))
        flat = torch.cat([flat, flat[:1]])
        flat[torch.where(slot >= 0, slot, flat.shape[0] - 1)] = x.to(cache.dtype).view(bits)
        out[name] = flat[:-1].view(cache.dtype).view(cache.shape)
    return out


def _plain_decode(s):
    c = s["case"]
    q, table, P = s["q"].float(), s["block_table"].long(), c["page"]
    B, Hq, D = q.shape
    Hkv, L = c["Hkv"], table.shape[1] * P
    pos = torch.arange(L, device=q.device)
    n = s["seq_len"].long()[:, None]
    seen = (pos < n) & (pos >= (n - c["window"] if c["window"] else 0))
    at = (table.clamp(min=0)[:, :, None] * P + torch.arange(P, device=q.device)).reshape(B, L)
    k = s["k_cache"].view(-1, Hkv, D)[at].float()                    # [B, L, Hkv, D]
    if s["k_scale"] is not None:
        k *= s["k_scale"][:, None]
    x = torch.einsum("bhgd,blhd->bhgl", q.view(B, Hkv, -1, D), k) / math.sqrt(D)
    del k
    x = torch.where(seen[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)                     # a row that sees nothing
    p = torch.exp(x - top)
    total = p.sum(-1)
    v = s["v_cache"].view(-1, Hkv, D)[at].float()
    if s["v_scale"] is not None:
        v *= s["v_scale"][:, None]
    v = torch.where(seen[:, :, None, None], v, 0.0)
    out = torch.einsum("bhgl,blhd->bhgd", p, v)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    lse = top[..., 0] + torch.log(total)
    return dict(out=out.reshape(B, Hq, D).to(s["q"].dtype), lse=lse.reshape(B, Hq))


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        import speculative_decoding_verification_76_gb300 as sv
        c = state["case"]
        if op == "tables":
            if "out" not in state:  # what a serving loop keeps: outputs, the list to release into
                state["out"], state["pool"] = None, state["free_list"].clone()
                state["total"] = torch.empty_like(state["free_count"])
                state["released"] = torch.empty_like(state["ctx_len"])
            e = state["out"] = sv.extend_tables(
                state["ctx_len"], state["add_len"], state["block_table"], state["free_list"],
                state["free_count"], c["page"], state["max_tokens"], out=state["out"])
            count, released = sv.release_pages(
                state["block_table"], e["new_len"], state["keep_pages"], state["pool"],
                e["free_count"], c["page"], total=state["total"], status=state["released"])
            out = dict(e, block_table=state["block_table"], left=e["free_count"],
                       free_list=state["pool"], released=released)
            out["free_count"] = count
            return out
        if op == "append":
            q, k, v = _split(state)
            sv.append_tokens(k, v, state["k_cache"], state["v_cache"], state["slot_map"],
                             state["positions"], q=q, q_out=state["q_out"],
                             rope_base=c["rope"], k_scale=state["k_scale"],
                             v_scale=state["v_scale"])
            return dict(q=state["q_out"], k_cache=state["k_cache"], v_cache=state["v_cache"])
        if "workspace" not in state:
            state["workspace"] = sv.new_workspace(
                sv.decode_attn_workspace_size(c["B"], c["Hq"], c["Hkv"], c["D"]),
                state["q"].device)
        out, lse = sv.decode_attn(state["q"], state["k_cache"], state["v_cache"],
                                  state["block_table"], state["seq_len"], window=c["window"],
                                  k_scale=state["k_scale"], v_scale=state["v_scale"],
                                  workspace=state["workspace"])
        return dict(out=out, lse=lse)
    return {"tables": _plain_tables, "append": _plain_append, "decode": _plain_decode}[op](state)


# ------------------------------------------------------------------ least work
def work(case):
    if case["op"] == "tables":
        P, B = case["page"], case["B"]
        ctx, add = _spread(case["lo"], case["hi"], B), _spread(case["add_lo"], case["add_hi"], B)
        tokens = sum(add)
        # lengths in, lengths and statuses out; a slot and a position per token; a page id read
        # and written per page taken (about a page per `page` tokens), and again per page given
        return dict(bytes=4 * 8 * B + 12 * tokens + 8 * (tokens // P + B), flops=0)
    size = {"bf16": 2, "f16": 2, "e4m3": 1}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        live = case["T"] - int(case["pad"] * case["T"])
        rows = (Hq + 2 * Hkv) * D * 2 + Hq * D * 2 + 2 * Hkv * D * size[case["cache"]]
        return dict(bytes=live * (rows + 12), flops=live * 6 * (Hq + Hkv) * D // 2)
    lens = _spread(case["lo"], case["hi"], case["B"])
    seen = sum(min(n, case["window"]) if case["window"] else n for n in lens)
    rows = case["B"] * Hq * (4 * D + 4)
    return dict(bytes=seen * 2 * Hkv * D * size[case["cache"]] + rows
                + 4 * sum(_ceil(n, case["page"]) for n in lens), flops=4 * seen * Hq * D)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None  # whole numbers
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "append":
        q, k, v = (x.double() for x in _split(s))
        if case["rope"]:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                               s["positions"].double()[:, None, None] * torch.exp(
                                   torch.arange(0, D, 2, device=DEV, dtype=torch.float64)
                                   * (-math.log(case["rope"]) / D)))
            rotated = []
            for x in (q, k):
                z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * turn
                rotated.append(torch.cat([z.real, z.imag], -1))
            q, k = rotated
        rows = (s["slot_map"] >= 0).nonzero()[:, 0]
        out = dict(q=s["q_out"].double())
        out["q"][rows] = q[rows]
        for name, x in (("k_cache", k), ("v_cache", v)):
            c = s[name].double()
            if case["cache"] == "e4m3":
                x = (x / s[name[0] + "_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
            c.view(-1, Hkv, D)[s["slot_map"][rows]] = x[rows]
            out[name] = c
        return out
    B, Hq, P = case["B"], case["Hq"], case["page"]
    out = torch.zeros(B, Hkv, Hq // Hkv, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hkv, Hq // Hkv), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["seq_len"].tolist()):
        first = max(0, n - case["window"]) if case["window"] else 0
        if first >= n:
            continue
        pages = s["block_table"][b, first // P:_ceil(n, P)].long()
        skip = first % P

        def rows(name):
            x = s[name][pages].reshape(-1, Hkv, D)[skip:skip + n - first].double()
            sc = s[name[0] + "_scale"]
            return (x if sc is None else x * sc.double()[:, None]).transpose(0, 1)
        q = s["q"][b].double().view(Hkv, -1, D) * D ** -0.5
        x = q @ rows("k_cache").transpose(1, 2)
        lse[b] = torch.logsumexp(x, -1)
        out[b] = torch.exp(x - lse[b][..., None]) @ rows("v_cache")
    return dict(out=out.view(B, Hq, D), lse=lse.view(B, Hq))
