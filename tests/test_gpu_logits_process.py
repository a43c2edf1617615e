"""GPU parity of logits_process: equal, element for element, to the same steps in fp32 (each step
is one rounded operation; counts are whole numbers), and its refusals."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import logits as olog

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def make(B, R, V, H, new, seed, tree=False, n_bias=7, masks="some", ids=None):
    r = np.random.default_rng(seed)
    some = lambda shape: r.integers(0, min(V, ids or V), shape)
    x = torch.from_numpy(r.normal(size=(B, R, V)) * 3).to(TYPES[new])
    kw = dict(history=some((B, H)), prompt_len=r.integers(0, H + 1, B),
              block_tokens=some((B, R if tree else R - 1)), parent=None,
              repetition=r.uniform(0.5, 2, B).astype(np.float32),
              frequency=r.normal(size=B).astype(np.float32), presence=r.normal(size=B).astype(np.float32))
    kw["history"][r.random((B, H)) < 0.1] = -1
    kw["history"][r.random((B, H)) < 0.05] = V + 3
    if tree:
        kw["parent"] = np.array([[-1] + [r.integers(0, i) for i in range(1, R)] for _ in range(B)])
    if n_bias:
        kw["bias_ids"] = some((B, n_bias))
        kw["bias_ids"][r.random((B, n_bias)) < 0.1] = -1
        kw["bias"] = r.normal(size=(B, n_bias)).astype(np.float32) * 3
    if masks:
        W = -(-V // 32)
        n = B * R if masks == "all" else 3
        kw["mask"] = r.integers(-2 ** 31, 2 ** 31, (n, W))
        kw["mask"][0] = -1
        kw["mask"][1 % n, :W // 2] = 0
        if masks == "some":
            kw["mask_row"] = r.integers(-1, n + 1, (B, R))
    return x, {k: v for k, v in kw.items() if v is not None}


def on_gpu(kw):
    return {k: torch.from_numpy(np.ascontiguousarray(v)).to(torch.float32 if v.dtype.kind == "f" else torch.int32)
            .to(DEV) for k, v in kw.items()}


def same(y, ref):
    np.testing.assert_array_equal(y.cpu().numpy(), ref)


@pytest.mark.parametrize("new", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,R,V,tree", [(1, 1, 1, False), (2, 5, 1013, False), (1, 1, 4096, False), (3, 17, 130, True),
                                        (2, 3, 4099, True), (1, 2, 12290, False), (1, 64, 33, True)])
def test_process(new, B, R, V, tree):
    x, kw = make(B, R, V, 60, new, B + R + V, tree)
    ref = olog.process(x.float().numpy(), fp=np.float32, **kw)
    g = on_gpu(kw)
    same(sv.logits_process(x.to(DEV), **g), ref)
    out = torch.empty((B, R, V), device=DEV)
    assert sv.logits_process(x.to(DEV), out=out, **g) is out
    same(out, ref)
    if new == "f32":
        y = x.to(DEV)
        assert sv.logits_process(y, out=y, **g) is y
        same(y, ref)


@pytest.mark.parametrize("drop", [("repetition",), ("frequency",), ("presence",), ("repetition", "frequency", "presence"),
                                  ("history", "prompt_len"), ("block_tokens",), ("bias_ids", "bias"),
                                  ("mask", "mask_row"), ("prompt_len",)])
@pytest.mark.parametrize("in_place", [False, True])
def test_parts(drop, in_place):
    x, kw = make(2, 4, 517, 30, "f32", 5)
    kw = {k: v for k, v in kw.items() if k not in drop}
    y = x.to(DEV)
    same(sv.logits_process(y, out=y if in_place else None, **on_gpu(kw)),
         olog.process(x.float().numpy(), fp=np.float32, **kw))


def test_nothing_asked():
    x = torch.randn((2, 3, 77), device=DEV).half()
    assert torch.equal(sv.logits_process(x), x.float())
    y = x.float()
    assert torch.equal(sv.logits_process(y, out=y), x.float())
    assert sv.logits_process(x[:0]).shape == (0, 3, 77)


def test_ids_that_repeat():
    """Three ids carry everything: counts in the thousands, biases listed many times, tokens of a
    tree's path that repeat."""
    x, kw = make(2, 9, 700, 5000, "f32", 6, tree=True, n_bias=900, ids=3)
    same(sv.logits_process(x.to(DEV), **on_gpu(kw)), olog.process(x.numpy(), fp=np.float32, **kw))


def test_a_mask_for_every_row():
    x, kw = make(3, 4, 1000, 10, "bf16", 7, masks="all")
    same(sv.logits_process(x.to(DEV), **on_gpu(kw)), olog.process(x.float().numpy(), fp=np.float32, **kw))


def test_masked_places_and_rows_that_are_not_finite():
    x, kw = make(1, 2, 300, 40, "f32", 8)
    kw["mask"], kw["mask_row"] = np.zeros((2, 10), np.int64), np.array([[0, 1]])
    kw["mask"][1, :] = 0x0f0f0f0f
    x[0, 0, :] = float("nan")
    x[0, 1, ::3], x[0, 1, 1::3] = float("inf"), -float("inf")
    x[0, 1, 8] = float("nan")
    y = sv.logits_process(x.to(DEV), **on_gpu(kw)).cpu().numpy()
    assert (y[0, 0] == -np.inf).all()
    with np.errstate(invalid="ignore"):
        same(torch.from_numpy(y), olog.process(x.numpy(), fp=np.float32, **kw))
    assert np.isnan(y[0, 1, 8]) and (y[0, 1, 4:8] == -np.inf).all()


def test_strided_rows_odd_addresses_and_streams():
    """Rows wider than the vocabulary (a padded last layer), an output that starts off 16 bytes."""
    B, R, V = 2, 3, 1021
    x, kw = make(B, R, V, 50, "bf16", 9)
    wide = torch.full((B, R, V + 11), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[..., 5:V + 5] = x.to(DEV)
    ref = olog.process(x.float().numpy(), fp=np.float32, **kw)
    flat = torch.empty(B * R * V + 3, device=DEV)
    st = torch.cuda.Stream()
    g = on_gpu(kw)
    for shift in range(4):
        out = flat[shift:shift + B * R * V].view(B, R, V)
        st.wait_stream(torch.cuda.current_stream())
        sv.logits_process(wide[..., 5:V + 5], out=out, stream=st, **g)
        torch.cuda.current_stream().wait_stream(st)
        same(out, ref)


def test_large_vocabulary_in_a_captured_graph():
    B, R, V = 3, 5, 152064
    x, kw = make(B, R, V, 3000, "f32", 10, masks="some")
    g, dx = on_gpu(kw), x.to(DEV)
    out = torch.empty_like(dx)
    graph = torch.cuda.CUDAGraph()
    sv.logits_process(dx, out=out, **g)
    with torch.cuda.graph(graph):
        sv.logits_process(dx, out=out, **g)
    out.zero_()
    graph.replay()
    # the oracle on the ids that anything touches, and the masks on all of them
    m = {k: v for k, v in kw.items() if k not in ("mask", "mask_row")}
    ref = olog.process(x.numpy(), fp=np.float32, **m)
    bits = (kw["mask"][:, :, None] >> np.arange(32) & 1).reshape(3, -1)[:, :V].astype(bool)
    for b in range(B):
        for i in range(R):
            r = kw["mask_row"][b][i]
            if 0 <= r < 3:
                ref[b, i][~bits[r]] = -np.inf
    same(out, ref)


def test_refusals():
    x = torch.zeros((2, 3, 64), device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    f32 = lambda *s: torch.zeros(s, device=DEV)
    for kw, what in ((dict(history=i32(3, 4)), "shape"), (dict(prompt_len=i32(2)), "without history"),
                     (dict(parent=i32(2, 3)), "without block_tokens"), (dict(block_tokens=i32(2, 3)), "shape"),
                     (dict(repetition=f32(3)), "shape"), (dict(frequency=i32(2)), "Float"),
                     (dict(bias=f32(2, 4)), "together"), (dict(bias_ids=i32(2, 4), bias=f32(2, 3)), "shape"),
                     (dict(mask=i32(6, 3)), "shape"), (dict(mask=i32(5, 2)), "rows"),
                     (dict(mask_row=i32(2, 3)), "without mask"), (dict(out=x[:, :, ::2]), "shape"),
                     (dict(out=x, mask=x.view(torch.int32).view(-1)[:12].view(6, 2)), "share memory")):
        with pytest.raises(ValueError, match=what):
            sv.logits_process(x, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        sv.logits_process(x.transpose(0, 1))
    with pytest.raises(ValueError, match="bf16"):
        sv.logits_process(x.double())
    with pytest.raises(sv.SpecError):
        sv.logits_process(torch.zeros((1, 65, 8), device=DEV))
