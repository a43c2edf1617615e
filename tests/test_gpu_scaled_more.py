"""The scaled cache's calls at the sizes where their work is dealt out differently: full row tiles, many
short segments, lists longer than a CTA, and calls back to back with lengths that change between them."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import logits as olog
from tests.test_gpu_logits_process import make, on_gpu, same
from tests.test_gpu_scaled_attn import check, dev, make_cache
from tests.test_gpu_scaled_cache import check_append

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("D,Hkv,block,new,inter", [(256, 3, 64, "bf16", False), (128, 2, 16, "f16", True),
                                                   (64, 1, 8, "bf16", True), (128, 5, 64, "f16", False)])
def test_append_full_row_tiles(D, Hkv, block, new, inter):
    """Sixteen rows of a CTA, teams of one to eight warps, long runs that cross several tiles."""
    rng = np.random.default_rng(D + Hkv)
    add = np.append(rng.integers(1, 400, 24), [1300, 64, 65, 1])
    ctx = rng.integers(0, 200, len(add))
    check_append(D, Hkv, Hkv, new, 64, block, ctx, add, (D // 2, inter, "none"), seed=D, pad=5)


@pytest.mark.parametrize("new,B,R,V,H,n_bias,tree", [
    ("f16", 5, 7, 70001, 9001, 1300, False), ("f32", 64, 5, 20011, 4100, 17, False), ("bf16", 3, 30, 16384, 700, 513, True)])
def test_logits_long_lists_and_row_groups(new, B, R, V, H, n_bias, tree):
    """Lists of several turns of a CTA; all rows of a sequence in a CTA, some of them, one."""
    x, kw = make(B, R, V, H, new, V, tree=tree, n_bias=n_bias)
    ref = olog.process(x.float().numpy(), fp=np.float32, **kw)
    g = on_gpu(kw)
    y = x.to(DEV)
    same(sv.logits_process(y, **g), ref)
    if new == "f32":
        same(sv.logits_process(y, out=y, **g), ref)


@pytest.mark.parametrize("R,G,Hkv,D,lens", [
    (1, 4, 2, 64, [1, 2, 3] * 100), (16, 4, 1, 128, [16, 300, 17, 144, 0] * 8),
    (5, 4, 2, 128, [133, 5, 640, 0, 128, 129] * 20), (3, 2, 1, 256, [1000, 3] * 9)])
def test_many_short_segments(R, G, Hkv, D, lens):
    """Ranges that lie in what a sequence's ends are counted as, that begin there, that hold many ends."""
    check(lens, R, G * Hkv, Hkv, D, 16, 8, "bf16", seed=R + D)


@pytest.mark.parametrize("R,G,D", [(1, 4, 64), (5, 4, 128), (64, 1, 128)])
def test_lengths_that_change_between_calls(R, G, D):
    """The joining kernel reads the lengths before the attention is complete: never the next call's."""
    Hkv, lens = 2, [5000, 300, 2500]
    cache, _, table = make_cache(lens, Hkv, D, 16, 16, seed=R)
    q = torch.randn((3, R, G * Hkv, D), device=DEV, dtype=torch.bfloat16)
    ctx = torch.zeros(3, dtype=torch.int32, device=DEV)
    ws = sv.new_workspace(sv.verify_attn_scaled_workspace_size(3, R, G * Hkv, Hkv, D), DEV)
    tab = dev(table)
    steps = [dev([a - R, b - R, c - R]) for a, b, c in
             ((5000, 300, 2500), (64, 299, 2000), (4000, 65, 64), (129, 130, 131), (4999, 64, 64))]
    alone = []
    for s in steps:
        ctx.copy_(s)
        torch.cuda.synchronize()
        alone.append(sv.verify_attn_scaled(q, *cache, tab, ctx, workspace=ws))
        torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in steps:
            ctx.copy_(s)
            got.append(sv.verify_attn_scaled(q, *cache, tab, ctx, workspace=ws))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, alone[i % len(steps)][0]) and torch.equal(lse, alone[i % len(steps)][1])
    assert sv.workspace_error(ws) == 0
