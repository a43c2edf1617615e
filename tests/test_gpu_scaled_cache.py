"""GPU parity of rotate, append_scaled, read_scaled and kv_commit on scaled caches against the
float64 oracle.

Tolerances.  A turned element is rounded once to its type (half a step: bf16 2^-8, fp16 2^-11,
fp32 2^-24 of the value) after fp32 arithmetic on an angle of 2^-32 of a turn, a sine and
cosine of 2 ulp, the magnitude and two products: 2^-20 (|a| + |b|).  Below 2^-14 fp16's steps are
2^-24, whatever the value: half of one, 2^-25, more.  Codes: a key may fall on the other side of a
midpoint, one e4m3 step (2^-3 of the value, 2^-9 of the scale where the type is subnormal); values
are equal.  Scales of keys are equal unless the largest key lies within 2^-20 of 448 times a power
of two; of values they are equal.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import rope as orope
from oracle import scaled as osc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def num(t):
    return t.detach().float().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).to(DEV)


def make_rope(dim, interleaved, scaling="none"):
    kw = dict(none={}, linear=dict(factor=4.0), ntk=dict(factor=4.0),
              parts=dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0))[scaling]
    mag = 1.25 if scaling == "parts" else 1.0
    f = orope.frequencies(dim, 5e5, scaling, **kw)
    return sv.Rope(dim, 5e5, interleaved, scaling, magnitude=mag, **kw), f, mag


def turn_bound(x, ref, interleaved, n, half):
    """Rounding of the turned pairs (see above); what stays is equal."""
    b = np.zeros_like(ref)
    i = np.arange(n // 2)
    p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + n // 2)
    size = (np.abs(x[..., p]) + np.abs(x[..., q])) * 1.25 * 2.0 ** -20
    b[..., p], b[..., q] = size, size
    b[..., :n] += half * (np.abs(ref[..., :n]) + b[..., :n])
    if half == HALF["f16"]:  # subnormal: a step is 2^-24, a nearest value at most half of it away
        b[..., :n] += 2.0 ** -25
    return b


# ------------------------------------------------------------------ rotate
@pytest.mark.parametrize("new", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,dim,interleaved,scaling", [
    (128, 128, False, "none"), (128, 64, True, "parts"), (64, 16, False, "ntk"), (256, 256, True, "linear"),
    (80, 32, False, "parts"), (16, 6, True, "none"), (512, 512, False, "ntk"), (96, 2, True, "linear"),
    (128, 0, False, "none")])
def test_rotate(new, D, dim, interleaved, scaling):
    g = torch.Generator().manual_seed(D + dim)
    T, Hq, Hkv = 37, 5, 2
    pos = np.array([0, 1, 131071, 2 ** 31 - 1, -1, 4097] * 7)[:T]
    qk = torch.randn((T, (Hq + Hkv) * D + 16), generator=g).to(TYPES[new]).to(DEV)  # strided rows
    q, k = qk[:, :Hq * D].unflatten(1, (Hq, D)), qk[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    if dim == 0:
        rope, f, mag = sv.Rope(0), np.zeros(0), 1.0
    else:
        rope, f, mag = make_rope(dim, interleaved, scaling)
    q_out = torch.full((T, Hq, D), 7.0, dtype=TYPES[new], device=DEV)
    qo, ko = sv.rotate(q, dev(pos), rope, k=k, q_out=q_out)
    assert qo is q_out
    live = pos >= 0
    for x, y, skipped in ((q, qo, 7.0), (k, ko, 0.0)):
        ref = orope.turn(num(x)[live], pos[live], f, interleaved, mag)
        err = np.abs(num(y)[live] - ref)
        # (an angle of pos f radians in float64 is off by pos f 2^-53 in the oracle: 2^-22 at most)
        bound = turn_bound(num(x)[live], ref, interleaved, dim, HALF[new])
        bound[..., :dim] += 2.0 ** -21 * np.abs(num(x)[live]).max()
        assert (err <= bound).all(), (err - bound).max()
        assert (num(y)[~live] == skipped).all()
    # in place, and queries alone
    both = q.clone()
    assert sv.rotate(both, dev(pos), rope, q_out=both)[0] is both
    assert torch.equal(both[dev(live, torch.bool)], qo[dev(live, torch.bool)])
    assert torch.equal(both[~dev(live, torch.bool)], q[~dev(live, torch.bool)])


def test_rotate_own_frequencies_and_far_positions():
    f = np.array([0.0, -1.0, 7.5, 1e-9] + [0.1] * 4)
    g = torch.Generator().manual_seed(0)
    x = torch.randn((3, 2, 32), generator=g)
    pos = np.array([0, 1000, 123456])
    y = sv.rotate(x.to(DEV), dev(pos), sv.Rope(16, freqs=tuple(f)))[0]
    ref = orope.turn(num(x), pos, f)
    assert (np.abs(num(y) - ref) <= turn_bound(num(x), ref, False, 16, HALF["f32"]) + 2.0 ** -20).all()
    # two positions whose difference is a whole number of turns: frequency 1/4 turn
    z = sv.rotate(x[:1].repeat(2, 1, 1).to(DEV), dev([3, 2 ** 31 - 1]),
                  sv.Rope(16, freqs=(np.pi / 2,) * 8))[0]
    assert (np.abs(num(z[0]) - num(z[1])) < 1e-6).all()


def test_rotate_refuses_overlaps():
    x = torch.zeros((4, 6, 64), device=DEV)
    q, k = x[:, :4], x[:, 4:]
    rope, pos = sv.Rope(64), dev([0, 1, 2, 3])
    sv.rotate(q, pos, rope, k=k, q_out=q, k_out=k)          # slices of one projection, in place
    for kw in (dict(q_out=x[:, 1:5]), dict(k=k, k_out=x[:, 3:5]), dict(k=k, q_out=q, k_out=x[:, :2])):
        with pytest.raises(ValueError, match="share memory"):
            sv.rotate(q, pos, rope, **kw)
    with pytest.raises(ValueError, match="k_out without k"):
        sv.rotate(q, pos, rope, k_out=k)
    with pytest.raises(ValueError, match="rope"):
        sv.rotate(q, pos, 7)


# ------------------------------------------------------------------ append, read
def new_cache(pages, P, nb, H, D, seed, bad=False):
    """A cache with something in it; bad: unwritten blocks hold NaN codes and odd scales."""
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(2):
        x = rng.normal(size=(pages * P, H, D)) * 2.0 ** rng.integers(-3, 3, (pages * P, 1, 1))
        x = torch.from_numpy(x).bfloat16().float().double().numpy()
        c, s = osc.append(np.zeros((pages, P, H, D)), np.zeros((pages, nb, H)), x, np.arange(pages * P))
        out.append([c, s])
    return out


def to_gpu(c, s):
    # (torch's own conversion keeps what is on the grid)
    return torch.from_numpy(c).float().to(torch.float8_e4m3fn).to(DEV), torch.from_numpy(s).float().to(DEV)


def packed(ctx, add, P, seed, spare=2):
    """Shuffled pages, slots and positions of a step's rows."""
    rng = np.random.default_rng(seed)
    had = [-(-(c + a) // P) for c, a in zip(ctx, add)]
    perm, at, slots, pos, table = rng.permutation(sum(had) + spare), 0, [], [], []
    for c, a, n in zip(ctx, add, had):
        pages = perm[at:at + n]
        at += n
        table.append(pages)
        slots += [pages[t // P] * P + t % P for t in range(c, c + a)]
        pos += list(range(c, c + a))
    return np.array(slots, np.int64), np.array(pos), sum(had) + spare, table


def check_append(D, Hq, Hkv, new, P, block, ctx, add, rope_args, seed, pad=0, loud=None):
    g = torch.Generator().manual_seed(seed)
    slots, pos, pages, _ = packed(ctx, add, P, seed)
    slots, pos = np.append(slots, [-1] * pad).astype(np.int64), np.append(pos, [-1] * pad)
    T = len(slots)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g)
    qkv = (qkv * torch.exp2(torch.randint(-4, 5, (T, 1), generator=g).float())).to(TYPES[new])
    if loud is not None:
        loud(qkv.view(T, -1, D))
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.to(DEV).split([Hq * D, Hkv * D, Hkv * D], 1))
    (kc, ks), (vc, vs) = new_cache(pages, P, P // block, Hkv, D, seed)
    gk, gks = to_gpu(kc, ks)
    gv, gvs = to_gpu(vc, vs)
    rope, f, mag = make_rope(*rope_args) if rope_args else (None, np.zeros(0), 1.0)
    q_out = torch.full((T, Hq, D), 7.0, dtype=TYPES[new], device=DEV)
    sv.append_scaled(k, v, gk, gv, gks, gvs, dev(slots, torch.int64), dev(pos), q=q, q_out=q_out,
                     rope=rope)
    dim, inter = len(f) * 2, bool(rope_args and rope_args[1])
    live = slots >= 0
    kk = num(k).copy()
    kk[live] = orope.turn(num(k)[live], pos[live], f, inter, mag)
    # queries
    ref = orope.turn(num(q)[live], pos[live], f, inter, mag)
    got, fin = num(q_out)[live], np.isfinite(ref)
    np.testing.assert_array_equal(got[~fin], ref[~fin])
    assert (np.abs(got - ref)[fin] <= turn_bound(num(q)[live], ref, inter, dim, HALF[new])[fin]).all()
    assert (num(q_out)[~live] == 7.0).all()
    # values: equal
    rc, rs = osc.append(vc, vs, num(v), slots)
    np.testing.assert_array_equal(num(gvs), rs)
    np.testing.assert_array_equal(num(gv), rc)
    # keys: scales equal, codes within a step
    rc, rs = osc.append(kc, ks, kk, slots)
    np.testing.assert_array_equal(num(gks), rs)
    with np.errstate(invalid="ignore"):
        off = np.abs(num(gk) - rc)
    nan = np.isnan(rc)
    np.testing.assert_array_equal(np.isnan(num(gk)), nan)
    assert (off[~nan] <= np.maximum(np.abs(rc) * 2.0 ** -3, 2.0 ** -9)[~nan]).all()
    assert (off[~nan] > 0).mean() < 1e-3
    # what the cache stands for, read back (bf16 holds it exactly), once with repeated slots
    twice = np.append(slots, slots[::-1])
    rk, rv = sv.read_scaled(gk, gv, gks, gvs, dev(twice, torch.int64))
    lv = twice >= 0
    for y, c, s in ((rk, num(gk), rs), (rv, num(gv), num(gvs))):
        ref = osc.values(c, s).reshape(pages * P, Hkv, D)[twice[lv]]
        np.testing.assert_array_equal(num(y)[lv], ref)
        assert not num(y)[~lv].any()
    return gk, gks


@pytest.mark.parametrize("D,Hq,Hkv,new,P,block,rope_args", [
    (128, 8, 2, "bf16", 16, 16, (128, False, "none")), (64, 3, 1, "f16", 24, 8, (32, True, "parts")),
    (256, 2, 2, "bf16", 64, 64, (256, False, "ntk")), (128, 4, 4, "f16", 5, 5, (64, False, "linear")),
    (64, 4, 2, "bf16", 1, 1, (64, True, "none")), (128, 2, 1, "bf16", 128, 32, None),
    (256, 4, 1, "f16", 12, 12, (64, True, "ntk"))])
@pytest.mark.parametrize("shape", ["one", "steps", "block", "prompts"])
def test_append_and_read(D, Hq, Hkv, new, P, block, rope_args, shape):
    ctx, add = dict(one=([0], [1]), steps=([0, 7, 16, 63, 130], [1] * 5),
                    block=([3, 0, 29, 64], [5, 5, 5, 5]), prompts=([0, 1, 77], [200, 131, 64]))[shape]
    check_append(D, Hq, Hkv, new, P, block, ctx, add, rope_args, seed=D + P + len(ctx), pad=3)


@pytest.mark.parametrize("block", [1, 16, 64])
def test_append_many_rows(block):
    """More rows than one CTA each: tiles of sixteen, runs that cross them."""
    rng = np.random.default_rng(block)
    ctx, add = rng.integers(0, 100, 40), rng.integers(1, 140, 40)
    add[3:9] = 1
    check_append(64, 2, 2, "bf16", 64, block, ctx, add, (64, False, "none"), seed=block, pad=37)


def test_append_values_that_are_not_finite():
    def loud(x):
        x[0, :, 3], x[1, :, 5], x[2], x[3, :, 7] = np.inf, np.nan, 0.0, -np.inf
        x[4] = 3e38
        x[5] = 1e-38
    check_append(64, 1, 2, "bf16", 8, 8, [0, 16, 2], [4, 1, 2], None, seed=5, loud=loud)


def test_append_beside_unusable_scales():
    """Blocks whose scale is no positive finite number, or no power of two."""
    D, P = 64, 8
    kc = torch.full((4, P, 1, D), 448.0).to(torch.float8_e4m3fn).to(DEV)
    vc = kc.clone()
    ks = torch.tensor([float("nan"), 0.0, 3.0, 2.0 ** -20], device=DEV).view(4, 1, 1)
    vs = ks.clone()
    x = torch.ones((4, 1, D), dtype=torch.bfloat16, device=DEV)
    sv.append_scaled(x, x, kc, vc, ks, vs, dev([3, P + 3, 2 * P + 3, 3 * P + 3], torch.int64))
    one = 2.0 ** -8  # 1 = 256 * 2^-8
    assert ks.flatten().tolist() == [one, one, 4.0, one] and torch.equal(ks, vs)
    got = num(kc)[:, :, 0, 0]
    assert got[0].tolist() == [448] * 3 + [256] + [448] * 4       # unusable: the codes stay
    assert got[2].tolist() == [320] * 3 + [0.25] + [320] * 4      # 448 * 3 / 4 = 336: a tie, to even
    assert got[3].tolist() == [448 * 2.0 ** -12] * 3 + [256] + [448 * 2.0 ** -12] * 4


def test_strided_caches_far_offsets_and_streams():
    """Heads first, as a slice of a wider pool, beyond 2^32 bytes, on another stream."""
    pages, P, Hkv, D = 530000, 16, 2, 128
    pool = torch.zeros((pages, 2, Hkv, P, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    kc, vc = pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2)
    ks, vs = (torch.zeros((pages, 2, Hkv), device=DEV) for _ in range(2))
    assert (pages - 1) * kc.stride(0) > 2 ** 32
    rows = torch.randn((6, 2, D), device=DEV).bfloat16()
    slots = dev([5, (pages - 1) * P + 7, (pages - 1) * P + 8, 3 * P, pages * P, -5], torch.int64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    sv.append_scaled(rows, rows * 2, kc, vc, ks, vs, slots, stream=st)
    k, v = sv.read_scaled(kc, vc, ks, vs, slots, k_out=torch.full((6, 2, D), 9.0, device=DEV), stream=st)
    torch.cuda.current_stream().wait_stream(st)
    ref = num(rows)[:4]
    assert (np.abs(num(k)[:4] - ref) <= np.abs(ref) * 2.0 ** -4 + 2.0 ** -15).all()
    assert (num(k)[4:] == 9.0).all() and k.dtype == v.dtype == torch.float32
    assert torch.equal(v[:4], k[:4] * 2)
    # half precision too
    h = sv.read_scaled(kc, vc, ks, vs, slots[:4], k_out=torch.empty((4, 2, D), dtype=torch.float16, device=DEV))
    assert torch.equal(h[0].float(), k[:4]) and h[1].dtype == torch.float16


def test_append_in_a_captured_graph_repeats_itself():
    ctx, add, P = [3, 15, 40], [2, 2, 2], 16
    slots, pos, pages, _ = packed(ctx, add, P, 0)
    (kc, ks), (vc, vs) = new_cache(pages, P, 1, 2, 64, 0)
    k = torch.randn((6, 2, 64), device=DEV).bfloat16() * 50
    state = [to_gpu(kc, ks), to_gpu(vc, vs)]
    other = [to_gpu(kc, ks), to_gpu(vc, vs)]
    rope = sv.Rope(64)
    args = (dev(slots, torch.int64), dev(pos))
    sv.append_scaled(k, k, other[0][0], other[1][0], other[0][1], other[1][1], *args, rope=rope)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.append_scaled(k, k, state[0][0], state[1][0], state[0][1], state[1][1], *args, rope=rope)
    for _ in range(3):
        g.replay()
    for a, b in zip(state, other):
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


def test_append_scaled_refuses():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=DEV)
    c = torch.zeros((3, 16, 2, 64), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    s, slots = torch.zeros((3, 2, 2), device=DEV), dev([0, 1, 2, 3], torch.int64)
    for kw, what in ((dict(ks=s[:, :, :1]), "shape"), (dict(ks=torch.zeros((3, 3, 2), device=DEV)), "k_scale"),
                     (dict(vs=torch.zeros((3, 1, 2), device=DEV)), "shape"), (dict(k=x.float()), "bf16"),
                     (dict(kc=c.view(torch.uint8)), "Float8"), (dict(slots=slots[:3]), "shape"),
                     (dict(slots=slots.int()), "Long|long"), (dict(rope=sv.Rope(64)), "positions"),
                     (dict(rope=3, pos=dev([0] * 4)), "rope")):
        a = dict(dict(k=x, v=x, kc=c, vc=c.clone(), ks=s, vs=s.clone(), slots=slots, pos=None, rope=None), **kw)
        with pytest.raises(ValueError, match=what):
            sv.append_scaled(a["k"], a["v"], a["kc"], a["vc"], a["ks"], a["vs"], a["slots"], a["pos"],
                             rope=a["rope"])
    with pytest.raises(sv.SpecError):   # more tokens to a block than the kernels take
        sv.append_scaled(x, x, torch.zeros((3, 128, 2, 64), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                         torch.zeros((3, 128, 2, 64), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                         torch.zeros((3, 1, 2), device=DEV), torch.zeros((3, 1, 2), device=DEV), slots)


# ------------------------------------------------------------------ commit
@pytest.mark.parametrize("D,P,block", [(64, 16, 8), (128, 5, 5), (256, 64, 64), (128, 4, 1)])
def test_commit_scaled(D, P, block):
    rng = np.random.default_rng(D + P)
    B, R, Hkv = 5, 17, 2
    ctx = np.array([0, 3, 12, 61, 7])
    slots, pos, pages, table = packed(ctx, [R] * B, P, 1)
    width = max(len(t) for t in table)
    bt = np.full((B, width), -1)
    for b, t in enumerate(table):
        bt[b, :len(t)] = t
    (kc, ks), (vc, vs) = new_cache(pages, P, P // block, Hkv, D, 3)
    accepted = np.array([4, 0, 16, 7, 2])
    path = np.full((B, R), -1)
    for b, a in enumerate(accepted):
        path[b, :a] = np.sort(rng.choice(np.arange(1, R), a, replace=False))
    path[4, :2] = [5, 3]                                       # not in storage order: refused
    gk, gks = to_gpu(kc, ks)
    gv, gvs = to_gpu(vc, vs)
    new_len, keep, status = sv.kv_commit(gk, gv, dev(bt), dev(ctx), dev(accepted), dev(path),
                                         k_scale=gks, v_scale=gvs)
    assert status.tolist() == [0, 0, 0, 0, sv.api.SEQ_BAD_TREE]
    assert new_len.tolist() == [5, 4, 29, 69, 7]
    assert keep.tolist() == [-(-n // P) for n in (5, 4, 29, 69, 7)]
    accepted[4] = 0
    for (c, s), y, z in (((kc, ks), gk, gks), ((vc, vs), gv, gvs)):
        rc, rs = osc.commit(c, s, bt, ctx, accepted, path)
        np.testing.assert_array_equal(num(z), rs)
        np.testing.assert_array_equal(num(y), rc)
    # a chain moves nothing
    before = gk.view(torch.uint8).clone()
    n, _, _ = sv.kv_commit(gk, gv, dev(bt), dev(ctx), dev(accepted), R=R, k_scale=gks, v_scale=gvs)
    assert n.tolist() == (ctx + 1 + accepted).tolist() and torch.equal(before, gk.view(torch.uint8))
    with pytest.raises(ValueError, match="together"):
        sv.kv_commit(gk, gv, dev(bt), dev(ctx), dev(accepted), dev(path), k_scale=gks)
