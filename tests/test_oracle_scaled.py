"""Pins of the oracle's rotary forms, scaled caches, their attention and the served logits, and
the host-side refusals of the calls they belong to (CPU only)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import append, attention, logits, rope, scaled
from speculative_decoding_verification_76_gb300 import api


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_76_gb300 import build
    build.build()
    return sv.load()


# ------------------------------------------------------------------ rotary forms
def test_rope_forms_by_hand():
    np.testing.assert_allclose(rope.frequencies(4, 100.0), [1.0, 0.1])
    np.testing.assert_allclose(rope.frequencies(4, 100.0, "linear", 8.0), [0.125, 0.0125])
    # ntk: the fastest pair stays, the slowest is divided by the factor
    f, g = rope.frequencies(64, 1e4), rope.frequencies(64, 1e4, "ntk", 16.0)
    assert g[0] == f[0] and g[-1] == pytest.approx(f[-1] / 16)
    # parts: 8192 / 2 pi = 1303.8 turns of the first pair stay; the slow ones are stretched
    f, g = rope.frequencies(64, 5e5), rope.frequencies(64, 5e5, "parts", 8.0, 8192, 1.0, 4.0)
    turns = 8192 * f / (2 * math.pi)
    assert (g[turns >= 4] == f[turns >= 4]).all() and (turns < 1).any()
    np.testing.assert_allclose(g[turns <= 1], f[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and (g[mid] < f[mid]).all() and (g[mid] > f[mid] / 8).all()
    # a quarter turn of (1, 2) is (-2, 1), in both layouts; what lies behind stays
    x = np.arange(1.0, 7.0)[None, None]
    assert rope.turn(x, [1], [math.pi / 2], True)[0, 0] == pytest.approx([-2, 1, 3, 4, 5, 6])
    y = rope.turn(x, [1], [math.pi / 2, 0.0], False, 2.0)[0, 0]
    assert y == pytest.approx([-6, 4, 2, 8, 5, 6])


def test_rope_agrees_with_the_append_oracle():
    rng = np.random.default_rng(0)
    x, pos = rng.normal(size=(5, 3, 64)), np.array([0, 1, 77, 4096, 131071])
    np.testing.assert_allclose(rope.turn(x, pos, rope.frequencies(64, 1e4)),
                               append.rope(x, pos, 1e4), atol=1e-9)


# ------------------------------------------------------------------ scaled caches
def test_scales_by_hand():
    assert scaled.needed([448.0]) == 1.0 and scaled.needed([448.5]) == 2.0
    assert scaled.needed([0.0]) == 2.0 ** -64 and scaled.needed([np.inf, np.nan, 3.0]) == 2.0 ** -7
    assert scaled.held(0.75) == 1.0 and scaled.held(2.0) == 2.0
    assert scaled.held(-1.0) == scaled.held(np.nan) == scaled.held(np.inf) == 0.0


def test_append_by_hand():
    codes, scales = np.zeros((2, 4, 1, 2)), np.zeros((2, 2, 1))
    # slots 2, 3 are page 0's second block; slot 5 lies inside page 1's first block
    c, s = scaled.append(codes, scales, np.array([[[448.0, 1]], [[2.0, 0]], [[3.5, -1]]]), [2, 3, 5])
    assert s.ravel().tolist() == [0, 1.0, 2.0 ** -7, 0]
    assert c[0, 2:, 0].tolist() == [[448, 1], [2, 0]]
    assert c[1, 1, 0].tolist() == [448, -128]
    # louder rows join the block: its codes move to the larger scale, exactly here
    c, s = scaled.append(c, s, np.array([[[900.0, 5]]]), [3])
    assert s[0, 1, 0] == 4.0 and c[0, 2:, 0].tolist() == [[112, 0.25], [224, 1.25]]
    # the block begins anew with its first token
    c, s = scaled.append(c, s, np.array([[[1.75, 0]]]), [2])
    assert s[0, 1, 0] == 2.0 ** -8 and c[0, 2, 0, 0] == 448
    # outside the cache: skipped
    d, t = scaled.append(c, s, np.ones((2, 1, 2)), [-1, 8])
    assert (d == c).all() and (t == s).all()


def test_commit_moves_values():
    rng = np.random.default_rng(1)
    codes, scales = scaled.append(np.zeros((3, 4, 2, 8)), np.zeros((3, 2, 2)),
                                  rng.normal(size=(10, 2, 8)) * 2.0 ** np.arange(10)[:, None, None],
                                  np.arange(10))
    before = scaled.values(codes, scales)
    c, s = scaled.commit(codes, scales, [[0, 1, 2]], [3], [3], [[2, 4, 6]])
    after = scaled.values(c, s)
    flat = lambda x: x.reshape(12, 2, 8)
    # positions 5, 7, 9 are now 4, 5, 6; what lies in front stays
    for dst, src in ((4, 5), (5, 7), (6, 9), (3, 3), (0, 0)):
        scale = np.repeat(s, 2, 1).reshape(12, 2)[dst][:, None]
        assert (np.abs(flat(after)[dst] - flat(before)[src]) <= scale * 2.0 ** -10).all()


def test_scaled_attention_is_the_verify_attention():
    rng = np.random.default_rng(2)
    q = rng.normal(size=(2, 5, 4, 16))
    k, v = rng.normal(size=(2, 6, 4, 2, 16))
    table, ctx = np.array([[0, 2, 4], [5, 3, 1]]), np.array([7, 0])
    parent = [-1, 0, 0, 1, 3]
    mask = []
    for i, p in enumerate(parent):
        mask.append((mask[p] if p >= 0 else 0) | 1 << i)
    anc = np.array([mask, mask], dtype=np.uint64)
    ref, rl = attention.verify_attention(q, k, v, table, ctx, anc)
    out, lse, aux = scaled.attention(q, k, v, table, ctx, anc)
    np.testing.assert_allclose(out, ref, atol=1e-12)
    np.testing.assert_allclose(lse, rl, atol=1e-12)
    assert aux["n"][0, :, 0].tolist() == [8, 9, 9, 10, 11]
    # a window of 6: row 4 (four block rows seen) keeps 2 of the 7 committed
    _, _, aux = scaled.attention(q, k, v, table, ctx, anc, window=6)
    assert aux["n"][0, :, 0].tolist() == [6, 6, 6, 6, 6] and aux["n"][1, :, 0].tolist() == [1, 2, 2, 3, 4]
    # an idle row, a missing page, an empty mask
    out, lse, aux = scaled.attention(q, k, v, np.array([[0, -1, 9], [5, 3, 1]]), [7, -1],
                                     [[0] * 5, mask])
    assert aux["n"][0, 0, 0] == 4 and not out[1].any() and (lse[1] == -np.inf).all()


# ------------------------------------------------------------------ served logits
def test_logits_by_hand():
    x = np.array([[[1.0, -1.0, 2.0, 3.0, 0.5]] * 3])
    kw = dict(history=[[1, 0, 0, -1, 9]], prompt_len=[1], block_tokens=[[2, 0]], repetition=[2.0],
              frequency=[0.5], presence=[0.25], bias_ids=[[4, -1, 4]], bias=[[1.0, 7.0, -3.0]])
    y = logits.process(x, **kw)[0]
    # id 1 is prompt: repetition alone; id 0 stands twice, and again in front of row 2
    assert y[0].tolist() == [0.5 - 1.25, -2.0, 2.0, 3.0, -1.5]
    assert y[1].tolist() == [0.5 - 1.25, -2.0, 1.0 - 0.75, 3.0, -1.5]
    assert y[2].tolist() == [0.5 - 1.75, -2.0, 1.0 - 0.75, 3.0, -1.5]
    # a tree: node 2 is a child of the anchor, node 1's token is not in front of it
    y = logits.process(x, block_tokens=[[0, 2, 3]], parent=[[-1, 0, 0]], presence=[1.0])[0]
    assert y[1].tolist() == [1, -1, 1, 3, 0.5] and y[2].tolist() == [1, -1, 2, 2, 0.5]
    y = logits.process(x, mask=[[0b10101], [0]], mask_row=[[0, -1, 1]])[0]
    assert y[0].tolist() == [1, -np.inf, 2, -np.inf, 0.5] and (y[1] == x[0, 1]).all()
    assert (y[2] == -np.inf).all()


# ------------------------------------------------------------------ refusals on the host
def _p(x=4096):
    return ctypes.c_void_p(x)


def _rope(**kw):
    r = dict(dim=64, interleaved=0, scaling=0, reserved=0, base=1e4, factor=1.0, original_len=0.0,
             low=1.0, high=4.0, magnitude=1.0, freqs=None)
    r.update(kw)
    return ctypes.byref(api._Rope(**r))


ROTATE = dict(q=_p(), qs=512, qo=_p(8192), qos=512, k=_p(1 << 20), ks=128, ko=_p(1 << 21), kos=128,
              dt=api.SPEC_BF16, pos=_p(), T=4, Hq=8, Hkv=2, D=64, rope=_rope(), st=None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(pos=None), 1), (dict(rope=None), 1), (dict(k=None), 1),
    (dict(ko=None), 1), (dict(Hkv=0), 1), (dict(qs=511), 1), (dict(q=_p(4098)), 1), (dict(T=-1), 1),
    (dict(dt=api.SPEC_E4M3), 1), (dict(qo=_p(), qos=1024), 1), (dict(D=72), 2), (dict(D=528), 2),
    (dict(Hq=5000), 2), (dict(T=2 ** 31 - 1), 2), (dict(rope=_rope(dim=63)), 1),
    (dict(rope=_rope(dim=128)), 1), (dict(rope=_rope(dim=24)), 2), (dict(rope=_rope(base=1.0)), 1),
    (dict(rope=_rope(base=math.nan)), 1), (dict(rope=_rope(scaling=4)), 1),
    (dict(rope=_rope(scaling=1, factor=0.5)), 1), (dict(rope=_rope(reserved=1)), 1),
    (dict(rope=_rope(scaling=2, factor=2.0, dim=2, interleaved=1)), 1),
    (dict(rope=_rope(scaling=3, factor=2.0)), 1), (dict(rope=_rope(magnitude=math.inf)), 1),
    (dict(rope=_rope(scaling=3, factor=2.0, original_len=8192.0, low=4.0, high=4.0)), 1),
    (dict(T=0), 0)])
def test_rotate_refuses_on_the_host(lib, change, code):
    assert lib.spec_rotate(*dict(ROTATE, **change).values()) == code


APPEND = dict(k=_p(), ks=128, v=_p(), vs=128, q=None, qs=0, qo=None, qos=0, nt=api.SPEC_BF16,
              kc=_p(), vc=_p(), sk=_p(), svv=_p(), pages=10, P=16, block=8, sp=2048, stt=128, sh=64,
              slots=_p(), pos=_p(), T=4, Hq=0, Hkv=2, D=64, rope=None, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), 1), (dict(vc=None), 1), (dict(sk=None), 1), (dict(slots=None), 1),
    (dict(pos=None, rope=_rope()), 1), (dict(q=_p()), 1), (dict(block=0), 1), (dict(block=5), 1),
    (dict(P=0), 1), (dict(Hkv=0), 1), (dict(T=-1), 1), (dict(ks=127), 1), (dict(sh=72), 1),
    (dict(kc=_p(4104)), 1), (dict(nt=api.SPEC_E4M3), 1), (dict(nt=api.SPEC_F32), 2),
    (dict(D=96), 2), (dict(P=128, block=128), 2), (dict(Hkv=5000), 2),
    (dict(pages=1 << 27, P=16), 2), (dict(T=2 ** 31 - 1), 2), (dict(rope=_rope(dim=128)), 1),
    (dict(T=0), 0), (dict(T=0, rope=_rope()), 0)])
def test_append_scaled_refuses_on_the_host(lib, change, code):
    assert lib.spec_append_scaled(*dict(APPEND, **change).values()) == code


READ = dict(kc=_p(), vc=_p(), sk=_p(), svv=_p(), pages=10, P=16, block=8, sp=2048, stt=128, sh=64,
            slots=_p(), T=4, Hkv=2, D=64, ko=_p(), kos=128, vo=_p(), vos=128, ot=api.SPEC_BF16,
            st=None)


@pytest.mark.parametrize("change,code", [
    (dict(kc=None), 1), (dict(vc=None), 1), (dict(svv=None), 1), (dict(ko=None), 1),
    (dict(slots=None), 1), (dict(kos=100), 1), (dict(ko=_p(4100)), 1), (dict(ot=api.SPEC_E4M3), 1),
    (dict(block=3), 1), (dict(D=80), 2), (dict(T=2 ** 31 - 1), 2), (dict(T=0), 0)])
def test_read_scaled_refuses_on_the_host(lib, change, code):
    assert lib.spec_read_scaled(*dict(READ, **change).values()) == code


COMMIT = dict(kc=_p(), vc=_p(), sk=_p(), svv=_p(), pages=10, P=16, block=8, Hkv=2, D=64, bt=_p(),
              maxp=4, ctx=_p(), acc=_p(), path=_p(), par=None, B=0, R=8, nl=_p(), kp=None,
              status=None, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(B=1, path=None), 1), (dict(B=1, sk=None), 1), (dict(R=65), 1), (dict(R=0), 1),
    (dict(block=6), 1), (dict(D=96), 2), (dict(maxp=1 << 27), 2), (dict(), 0)])
def test_commit_scaled_refuses_on_the_host(lib, change, code):
    assert lib.spec_commit_scaled(*dict(COMMIT, **change).values()) == code


ATTN = dict(q=_p(), qb=4096, qr=1024, qh=128, qt=api.SPEC_BF16, kc=_p(), vc=_p(), sk=_p(), svv=_p(),
            pages=10, P=16, block=16, sp=4096, stt=256, sh=128, bt=_p(), maxp=4, ctx=_p(),
            mask=None, B=1, R=4, Hq=8, Hkv=2, D=128, window=0, scale=0.0, ws=_p(), wsb=1 << 30,
            out=_p(), lse=None, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(sk=None), 1), (dict(ctx=None), 1), (dict(ws=None), 1),
    (dict(out=None), 1), (dict(Hq=9), 1), (dict(R=0), 1), (dict(B=-1), 1), (dict(block=5), 1),
    (dict(window=-1), 1), (dict(qh=100), 1), (dict(sh=8), 1), (dict(kc=_p(4104)), 1),
    (dict(ws=_p(4096 + 64)), 1), (dict(wsb=16), 1), (dict(qt=api.SPEC_E4M3), 1),
    (dict(qt=api.SPEC_F32), 2), (dict(D=96), 2), (dict(R=65), 2), (dict(window=3), 2),
    (dict(P=128, block=128), 2), (dict(maxp=1 << 27), 2), (dict(B=0), 0)])
def test_verify_attn_scaled_refuses_on_the_host(lib, change, code):
    assert lib.spec_verify_attn_scaled(*dict(ATTN, **change).values()) == code


LOGITS = dict(x=_p(1 << 20), xs=100, dt=api.SPEC_F32, out=_p(1 << 21), B=2, R=3, V=100, hist=_p(),
              H=5, pl=None, tok=_p(), par=None, rep=_p(), fr=_p(), pr=_p(), ids=_p(), bias=_p(),
              nb=3, mask=_p(), nm=6, mr=None, st=None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(hist=None), 1), (dict(tok=None, par=_p()), 1),
    (dict(bias=None), 1), (dict(mask=None), 1), (dict(xs=99), 1), (dict(R=65), 1), (dict(V=0), 1),
    (dict(dt=api.SPEC_E4M3), 1), (dict(out=_p(1 << 20), dt=api.SPEC_BF16), 1),
    (dict(out=_p(1 << 20), xs=104), 1), (dict(x=_p(4097)), 1), (dict(V=2 ** 31 - 1, xs=2 ** 31), 2),
    (dict(B=0), 0)])
def test_logits_process_refuses_on_the_host(lib, change, code):
    assert lib.spec_logits_process(*dict(LOGITS, **change).values()) == code


def test_bindings_refuse_host_tensors(lib):
    z, i = torch.zeros, torch.int32
    e4 = torch.zeros(1, 16, 1, 64).to(torch.float8_e4m3fn)
    h = torch.bfloat16
    s = z(1, 2, 1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.rotate(z(2, 1, 64), z(2, dtype=i), sv.Rope(64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.append_scaled(z(2, 1, 64, dtype=h), z(2, 1, 64, dtype=h), e4, e4, s, s,
                         z(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.read_scaled(e4, e4, s, s, z(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.verify_attn_scaled(z(1, 1, 1, 64, dtype=h), e4, e4, s, s, z(1, 1, dtype=i), z(1, dtype=i))
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.logits_process(z(1, 1, 8))
    with pytest.raises(ValueError, match="scaling"):
        sv.Rope(64, scaling="yes")
