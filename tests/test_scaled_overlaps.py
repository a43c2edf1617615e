"""Arguments of the scaled cache's calls that share memory: refused before anything is launched."""
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from tests.test_oracle_scaled import APPEND, COMMIT, _p

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return sv.load()


# places that do not meet: 10 pages of 16 tokens, 2 heads of 64, blocks of 8; 3 sequences, 8 rows, 4 pages
WRITE = dict(kc=_p(1 * MB), vc=_p(2 * MB), sk=_p(3 * MB), svv=_p(4 * MB))


@pytest.mark.parametrize("change", [
    dict(vc=_p(1 * MB)), dict(svv=_p(3 * MB)), dict(svv=_p(3 * MB + 10 * 2 * 2 * 4 - 4))])
def test_append_scaled(lib, change):
    args = dict(APPEND, **WRITE)
    args.update(k=_p(5 * MB), v=_p(6 * MB), slots=_p(7 * MB), pos=_p(8 * MB))
    args.update(change)
    assert lib.spec_append_scaled(*args.values()) == 1


COMMITTED = dict(COMMIT, **WRITE, bt=_p(5 * MB), ctx=_p(6 * MB), acc=_p(7 * MB), path=_p(8 * MB),
                 par=_p(9 * MB), B=3, nl=_p(10 * MB), kp=_p(11 * MB), status=_p(12 * MB))


@pytest.mark.parametrize("change", [
    dict(nl=_p(6 * MB)), dict(nl=_p(6 * MB + 8)), dict(nl=_p(7 * MB)), dict(kp=_p(6 * MB)),
    dict(status=_p(7 * MB + 4)), dict(nl=_p(5 * MB + 44)), dict(kp=_p(8 * MB + 92)), dict(status=_p(9 * MB)),
    dict(kp=_p(10 * MB)), dict(status=_p(11 * MB + 8)), dict(vc=_p(1 * MB)), dict(vc=_p(1 * MB + 16)),
    dict(svv=_p(3 * MB)), dict(sk=_p(2 * MB + 64)), dict(nl=_p(4 * MB))])
def test_commit_scaled(lib, change):
    assert lib.spec_commit_scaled(*dict(COMMITTED, **change).values()) == 1


DEV = "cuda:0"


def append_args():
    """Everything of a call inside one buffer, so that places can be moved over one another."""
    pool = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)

    def at(mb, shape, dtype, shift=0):
        n = torch.Size(shape).numel() * dtype.itemsize
        return pool[mb * MB + shift:mb * MB + shift + n].view(dtype).view(shape)
    e4 = torch.float8_e4m3fn
    a = dict(k=at(0, (4, 2, 64), torch.bfloat16), v=at(1, (4, 2, 64), torch.bfloat16),
             kc=at(2, (10, 16, 2, 64), e4), vc=at(3, (10, 16, 2, 64), e4), ks=at(4, (10, 2, 2), torch.float32),
             vs=at(5, (10, 2, 2), torch.float32), slots=at(6, (4,), torch.int64), pos=at(6, (4,), torch.int32, 4096),
             q=at(7, (4, 8, 64), torch.bfloat16), q_out=at(7, (4, 8, 64), torch.bfloat16, MB // 2))
    a["slots"].copy_(torch.arange(4))
    a["pos"].copy_(torch.arange(4))
    return at, a


def append(a):
    return sv.append_scaled(a["k"], a["v"], a["kc"], a["vc"], a["ks"], a["vs"], a["slots"], a["pos"], q=a["q"],
                            q_out=a["q_out"], rope=sv.Rope(64))


@pytest.mark.gpu
@pytest.mark.parametrize("name,place", [
    ("kc", (3, 0)), ("kc", (0, 64)), ("kc", (7, 0)), ("vc", (1, 0)), ("vc", (7, 2048)), ("ks", (5, 16)),
    ("ks", (2, 256)), ("vs", (3, 1024)), ("vs", (6, 0)), ("ks", (6, 4096)), ("q_out", (6, 0)), ("q_out", (6, 4096)),
    ("q_out", (4, 0)), ("q_out", (5, 0)), ("q_out", (2, 16)), ("q_out", (3, 0)), ("q_out", (0, 0)), ("q_out", (1, 32)),
    ("q_out", (7, 128))])
def test_append_scaled_binding(name, place):
    at, a = append_args()
    assert append(a) is a["q_out"]
    old = a[name]
    a[name] = at(place[0], old.shape, old.dtype, place[1])
    with pytest.raises(ValueError, match="share memory"):
        append(a)


@pytest.mark.gpu
def test_append_scaled_binding_takes_what_does_not_meet():
    """Queries in place, slices of one projection, K and V between one another in a pool."""
    qkv = torch.randn((4, 12, 64), device=DEV).bfloat16()
    pool = torch.zeros((10, 2, 16, 2, 64), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    ks, vs = torch.zeros((10, 2, 2), device=DEV), torch.zeros((10, 2, 2), device=DEV)
    slots = torch.arange(4, device=DEV)
    pos = torch.arange(4, device=DEV, dtype=torch.int32)
    q = qkv[:, :8]
    want = sv.append_scaled(qkv[:, 8:10], qkv[:, 10:], pool[:, 0], pool[:, 1], ks, vs, slots, pos, q=q,
                            rope=sv.Rope(64))
    codes = pool.view(torch.uint8).clone()
    got = sv.append_scaled(qkv[:, 8:10], qkv[:, 10:], pool[:, 0], pool[:, 1], ks, vs, slots, pos, q=q, q_out=q,
                           rope=sv.Rope(64))
    assert got is q and torch.equal(q, want) and torch.equal(pool.view(torch.uint8), codes)


@pytest.mark.gpu
def test_commit_scaled_binding():
    i = dict(dtype=torch.int32, device=DEV)
    c = torch.zeros((4, 16, 2, 64), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    s = torch.ones((4, 2, 2), device=DEV)
    table, ctx = torch.arange(4, **i).view(1, 4), torch.tensor([3], **i)
    acc, path = torch.tensor([1], **i), torch.tensor([[2, -1, -1]], **i)
    call = lambda **kw: sv.kv_commit(c, c.clone(), table, ctx, acc, path, k_scale=s, v_scale=s.clone(), **kw)
    assert call()[0].item() == 5
    for kw in (dict(new_len=ctx), dict(new_len=acc), dict(keep_pages=ctx), dict(status=acc)):
        with pytest.raises(sv.SpecError):
            call(**kw)
    assert ctx.item() == 3
