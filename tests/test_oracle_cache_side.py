"""Pins of the oracle's block tables, e4m3 grid, packed append and one-token attention,
and the host-side refusals of the calls they belong to (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import append, attention, decode, tables
from speculative_decoding_verification_76_gb300 import api


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_76_gb300 import build
    build.build()
    return sv.load()


# ------------------------------------------------------------------ tables
def test_extend_by_hand():
    # pages of 4; sequence 0 has 3 tokens on page 7 and gets 3 more: the rest of page 7 and
    # the list's last page; sequence 1 is new: two pages; sequence 2 adds nothing
    table = np.array([[7, -1, -1], [-1, -1, -1], [5, -1, -1]])
    e = tables.extend([3, 0, 4], [3, 5, 0], table, [0, 1, 2, 3, 4, 9, 9, 9], 5, 4, 10)
    assert e["block_table"].tolist() == [[7, 4, -1], [3, 2, -1], [5, -1, -1]]
    assert e["slot_map"].tolist() == [31, 16, 17, 12, 13, 14, 15, 8, -1, -1]
    assert e["positions"].tolist() == [3, 4, 5, 0, 1, 2, 3, 4, -1, -1]
    assert e["cu_len"].tolist() == [0, 3, 8, 8] and e["new_len"].tolist() == [6, 5, 4]
    assert e["free_count"] == 2 and e["status"].tolist() == [0, 0, 0]
    # giving back what lies behind the first page of 0 and all of 1 restores the list
    lst, n, st = tables.release(e["block_table"], e["new_len"], [1, 0, 1],
                                [0, 1, 9, 9, 9, 9, 9, 9], 2, 4)
    assert n == 5 and sorted(lst[:n].tolist()) == [0, 1, 2, 3, 4] and not st.any()


def test_extend_refusals_by_hand():
    table = np.full((6, 2), -1)
    e = tables.extend([0, -1, 0, 0, 3, 0], [4, 1, 9, 8, 1, 4], table, [0, 1, 2], 2, 4, 100)
    # 1: negative; 2: three pages of two; 3: 1 + 2 pages of 2 free; 4: needs none (but its
    # old page is missing); 5: behind a refused one
    assert e["status"].tolist() == [0, tables.BAD_LEN, tables.BAD_LEN, tables.NO_PAGES,
                                    tables.BAD_PAGE, tables.NO_PAGES]
    assert e["free_count"] == 1 and e["new_len"].tolist() == [4, -1, 0, 0, 3, 0]
    assert e["slot_map"][:4].tolist() == [4, 5, 6, 7] and (e["slot_map"][4:] == -1).all()
    e = tables.extend([0, 0], [3, 3], np.full((2, 2), -1), [0, 1], 2, 4, 5)   # 5 rows only
    assert e["status"].tolist() == [0, tables.BAD_LEN] and e["free_count"] == 1


# ------------------------------------------------------------------ e4m3, append
def test_e4m3_grid_is_torchs():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    every = every[np.isfinite(every)]
    np.testing.assert_array_equal(append.e4m3(every), every)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, s, 4000) for s in (1e-3, 0.02, 1.0, 100.0)])
    mids = (np.sort(every)[1:] + np.sort(every)[:-1]) / 2          # ties go to even
    x = np.clip(np.concatenate([x, mids]).astype(np.float32), -448, 448)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(append.e4m3(x), ref)
    assert append.e4m3(1e6) == 448.0 and append.e4m3(-1e6) == -448.0


def test_append_tokens_is_append_block_at_its_slots():
    rng = np.random.default_rng(1)
    kc, vc = rng.normal(size=(2, 6, 4, 2, 8))
    k, v = rng.normal(size=(2, 1, 5, 2, 8))
    table, ctx = np.array([[4, 2, 0]]), np.array([3])
    pos = ctx[:, None] + np.arange(5)
    ref = append.append_block(kc, vc, table, ctx, k, v, pos, 4)
    slots = [int(table[0, t // 4]) * 4 + t % 4 for t in range(3, 8)]
    got = append.append_tokens(kc, vc, k[0], v[0], slots, pos[0], 4)
    for a, b in zip(ref, got):
        np.testing.assert_array_equal(a, b)
    same = append.append_tokens(kc, vc, k[0], v[0], [-1, 24, -5, 99, -1], pos[0], 4)
    np.testing.assert_array_equal(same[0], kc)


# ------------------------------------------------------------------ one-token attention
def test_decode_is_the_verify_attention_of_one_row():
    rng = np.random.default_rng(2)
    q, (kc, vc) = rng.normal(size=(3, 1, 4, 8)), rng.normal(size=(2, 9, 4, 2, 8))
    table = rng.permutation(9).reshape(3, 3)
    ctx = np.array([11, 0, 5])                     # stored tokens before the row's own
    ref, lse_ref = attention.verify_attention(q, kc, vc, table, ctx, np.ones((3, 1), np.uint64))
    out, lse, _, _ = decode.decode_attention(q[:, 0], kc, vc, table, ctx + 1)
    np.testing.assert_allclose(out, ref[:, 0], rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse, lse_ref[:, 0], rtol=1e-12)


def test_decode_window_nothing_seen_and_missing_pages():
    rng = np.random.default_rng(3)
    q, (kc, vc) = rng.normal(size=(1, 2, 8)), rng.normal(size=(2, 4, 4, 1, 8))
    table = np.array([[2, 0, 3]])
    a = decode.decode_attention(q, kc, vc, table, [10], window=1)
    np.testing.assert_allclose(a[0], np.repeat(vc[3, 1][None], 2, 1), rtol=1e-15)  # position 9
    b = decode.decode_attention(q, kc, vc, table, [10], window=50)
    np.testing.assert_array_equal(b[0], decode.decode_attention(q, kc, vc, table, [10])[0])
    z = decode.decode_attention(q, kc, vc, table, [0])
    assert (z[0] == 0).all() and (z[1] == -np.inf).all()
    m = decode.decode_attention(q, kc, vc, np.array([[2, -1, 3]]), [10])
    n = decode.decode_attention(q, kc, vc, np.array([[2, 3]]), [6])   # the same rows
    np.testing.assert_allclose(m[0], n[0], rtol=1e-12)
    # parts join by their log-sum-exp
    whole = decode.decode_attention(q, kc, vc, table, [12])
    parts = [decode.decode_attention(q, kc, vc, t, [n]) for t, n in
             ((np.array([[2]]), 4), (np.array([[0, 3]]), 8))]
    w = [np.exp(x[1] - whole[1])[..., None] for x in parts]
    np.testing.assert_allclose(sum(x[0] * y for x, y in zip(parts, w)), whole[0], rtol=1e-12)


# ------------------------------------------------------------------ refusals on the host
def _p(n=4096):
    return ctypes.c_void_p(n)


def test_extend_and_release_refuse_on_the_host(lib):
    def extend(B=2, P=16, maxp=4, pool=8, cap=64, **ptr):
        a = {k: _p(4096 * (i + 1)) for i, k in enumerate(
            "ctx add table lst cnt slots pos cu new left status".split())}
        a.update(ptr)
        return lib.spec_extend_tables(a["ctx"], a["add"], B, P, a["table"], maxp, a["lst"], pool,
                                      a["cnt"], cap, a["slots"], a["pos"], a["cu"], a["new"],
                                      a["left"], a["status"], None)
    for name in "ctx add table lst cnt slots pos cu new left status".split():
        assert extend(**{name: None}) == api.SPEC_EINVAL, name
    for kw in (dict(B=-1), dict(P=0), dict(maxp=0), dict(pool=0), dict(cap=-1),
               dict(left=_p(7 * 4096), cnt=_p(7 * 4096)), dict(new=_p(9000), ctx=_p(9000)),
               dict(new=_p(9000), add=_p(9000)), dict(cu=_p(9000), ctx=_p(9000)),
               dict(status=_p(9000), add=_p(9000)), dict(table=_p(9000), lst=_p(9000))):
        assert extend(**kw) == api.SPEC_EINVAL, kw
    for kw in (dict(B=8193), dict(maxp=1 << 28), dict(cap=2 ** 31 - 1), dict(pool=2 ** 31 - 1)):
        assert extend(**kw) == api.SPEC_EUNSUPPORTED, kw

    def release(B=2, P=16, maxp=4, pool=8, **ptr):
        a = {k: _p(4096 * (i + 1)) for i, k in enumerate(
            "table len keep lst cnt total status".split())}
        a.update(ptr)
        return lib.spec_release_pages(a["table"], maxp, a["len"], a["keep"], B, P, a["lst"], pool,
                                      a["cnt"], a["total"], a["status"], None)
    for name in "table len keep lst cnt total".split():
        assert release(**{name: None}) == api.SPEC_EINVAL, name
    assert release(total=_p(5), cnt=_p(5)) == api.SPEC_EINVAL
    assert release(status=_p(5), keep=_p(5)) == api.SPEC_EINVAL
    assert release(lst=_p(5), table=_p(5)) == api.SPEC_EINVAL
    assert release(P=0) == api.SPEC_EINVAL
    assert release(B=8193) == api.SPEC_EUNSUPPORTED


APPEND = dict(k=_p(), ks=1024, v=_p(), vs=1024, q=_p(), qs=4096, qo=_p(8192), qos=4096,
              dt=api.SPEC_BF16, kc=_p(), vc=_p(), ct=api.SPEC_BF16, sk=None, sv=None, pages=4,
              P=16, sp=16384, st=1024, sh=128, slots=_p(), pos=_p(), T=3, Hq=32, Hkv=8, D=128,
              base=10000.0, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(slots=None), 1), (dict(pos=None), 1), (dict(q=None), 1), (dict(qo=None), 1),
    (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(P=0), 1), (dict(pages=0), 1), (dict(base=1.0), 1),
    (dict(base=-2.0), 1), (dict(base=float("nan")), 1), (dict(base=float("inf")), 1),
    (dict(dt=api.SPEC_E4M3), 1), (dict(ct=api.SPEC_F16), 1), (dict(sk=_p()), 1),
    (dict(k=_p(4104)), 1), (dict(ks=1023), 1), (dict(sh=100), 1), (dict(ks=-1024), 1),
    (dict(qo=_p(), qos=8192), 1), (dict(D=96), 2), (dict(D=512), 2),
    (dict(dt=api.SPEC_F32, ct=api.SPEC_E4M3), 2), (dict(T=0), 0)])
def test_append_tokens_refuses_on_the_host(lib, change, code):
    assert lib.spec_append_tokens(*dict(APPEND, **change).values()) == code


DECODE = dict(q=_p(), qb=4096, qh=128, qt=api.SPEC_BF16, kc=_p(), vc=_p(), ct=api.SPEC_BF16,
              sk=None, sv=None, pages=64, P=16, sp=16384, st=1024, sh=128, table=_p(), maxp=8,
              lens=_p(), B=2, Hq=32, Hkv=8, D=128, window=0, scale=0.0, ws=_p(), wsb=1 << 40,
              out=_p(), lse=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(table=None), 1),
    (dict(lens=None), 1), (dict(ws=None), 1), (dict(out=None), 1), (dict(B=-1), 1),
    (dict(Hq=33), 1), (dict(Hkv=0), 1), (dict(window=-1), 1), (dict(P=0), 1), (dict(maxp=0), 1),
    (dict(ct=api.SPEC_F16), 1), (dict(sk=_p()), 1), (dict(qt=api.SPEC_E4M3), 1),
    (dict(ws=_p(4096 + 128)), 1), (dict(wsb=1000), 1), (dict(qb=4097), 1), (dict(st=0), 1),
    (dict(kc=_p(4112)), 1), (dict(vc=_p(4112)), 1), (dict(sh=136), 1), (dict(out=_p(4104)), 1),
    (dict(q=_p(4104)), 1), (dict(qt=api.SPEC_F32, ct=api.SPEC_F32), 2), (dict(D=96), 2),
    (dict(sp=1000 * 1024 + 512), 2), (dict(pages=1 << 28), 2), (dict(maxp=1 << 28), 2),
    (dict(Hq=4097, Hkv=4097), 2), (dict(maxp=1 << 26, B=8192), 2), (dict(B=0), 0)])
def test_decode_attn_refuses_on_the_host(lib, change, code):
    assert lib.spec_decode_attn(*dict(DECODE, **change).values()) == code


def test_decode_workspace(lib):
    one = sv.decode_attn_workspace_size(1, 32, 8, 128)
    # header, 8192 counters, partial rows of fp32: no dependence on the batch
    assert one == sv.decode_attn_workspace_size(4096, 32, 8, 128) > 256 + 8192 * 4
    assert sv.decode_attn_workspace_size(1, 33, 8, 128) == 0
    assert sv.decode_attn_workspace_size(1, 32, 8, 96) == 0
    ws = sv.decode_attn_workspace_size(2, 32, 8, 128)
    assert lib.spec_decode_attn(*dict(DECODE, wsb=ws // 2).values()) == api.SPEC_EINVAL


def test_bindings_refuse_host_tensors(lib):
    z = torch.zeros
    i = torch.int32
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.extend_tables(z(2, dtype=i), z(2, dtype=i), z(2, 4, dtype=i), z(8, dtype=i),
                         z(1, dtype=i), 16, 8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.release_pages(z(2, 4, dtype=i), z(2, dtype=i), z(2, dtype=i), z(8, dtype=i),
                         z(1, dtype=i), 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.append_tokens(z(2, 1, 64), z(2, 1, 64), z(1, 16, 1, 64), z(1, 16, 1, 64),
                         z(2, dtype=torch.int64), rope_base=0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.decode_attn(z(1, 1, 64, dtype=torch.bfloat16), z(1, 16, 1, 64, dtype=torch.bfloat16),
                       z(1, 16, 1, 64, dtype=torch.bfloat16), z(1, 1, dtype=i), z(1, dtype=i))


def test_kv_commit_takes_the_new_cache_types(lib):
    buf = (ctypes.c_int32 * 128)()
    p = ctypes.c_void_p((ctypes.addressof(buf) + 15) & ~15)

    def commit(elem, D):   # an empty batch: checked, nothing launched
        return lib.spec_kv_commit(p, p, elem, 1, 16, 1, D, p, 1, p, p, None, None, 0, 8, p, None,
                                  None, None)
    for elem, D in ((1, 64), (1, 128), (1, 256), (2, 256)):
        assert commit(elem, D) == api.SPEC_OK
    assert commit(4, 256) == api.SPEC_EUNSUPPORTED
