"""Bounded device waits of verify_attn_scaled: one that runs out ends the kernel with an error word.

spec_debug_attn_fault makes the load warps withhold one tile and bounds every wait by 20 us.  Each role
has bounded waits only, the groups of warps leave their loops together (by votes), a warp whose wait ran
out gives nothing back (a barrier's phase must not get more arrivals than it counts), and tensor memory is
freed behind the last tensor-core operation; so the call returns, the error word reads
SPEC_ERR_MBAR_TIMEOUT, and the next call on a fresh workspace is right.
"""
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from speculative_decoding_verification_76_gb300 import api
from tests.test_gpu_scaled_attn import DEV, chain_masks, check, dev, make_cache

pytestmark = pytest.mark.gpu
SPEC_ERR_MBAR_TIMEOUT = 0x100


# rows of 16, 32 and 64 a tile, each head size, several segments of a CTA, a first and a later tile
@pytest.mark.parametrize("stage", [0, 2])
@pytest.mark.parametrize("D,R,G,Hkv,lens", [
    (64, 1, 4, 2, [300, 700, 40]), (128, 5, 4, 2, [9000, 70000, 300]), (128, 16, 4, 1, [130000, 600]),
    (256, 8, 2, 1, [90000, 500]), (64, 64, 1, 1, [100000])])
def test_withheld_tile_times_out_then_recovers(D, R, G, Hkv, lens, stage):
    cache, _, table = make_cache([60] * 3, Hkv, D, 16, 16, seed=1)
    # a long context of the same few pages: only the number of tiles matters
    pages = table[table >= 0]
    long = [[int(pages[i % len(pages)]) for i in range(-(-max(lens) // 16))] for _ in lens]
    q = torch.randn(len(lens), R, G * Hkv, D, device=DEV, dtype=torch.bfloat16)
    size = sv.verify_attn_scaled_workspace_size(len(lens), R, G * Hkv, Hkv, D)
    args = (q, *cache, dev(long), dev([n - R for n in lens]))
    ws = sv.new_workspace(size, DEV)
    try:
        assert api.load().spec_debug_attn_fault(stage, 20_000) == api.SPEC_OK
        sv.verify_attn_scaled(*args, workspace=ws)
        torch.cuda.synchronize()
        # (a CTA with fewer tiles meets nothing)
        tiles = Hkv * sum(-(-n // 128) for n in lens)
        if stage == 0 or tiles > 152 * 3 * 2:
            assert sv.workspace_error(ws) == SPEC_ERR_MBAR_TIMEOUT
    finally:
        assert api.load().spec_debug_attn_fault(-1, 0) == api.SPEC_OK
    # the context is usable and a normal call is right
    ws = sv.new_workspace(size, DEV)
    sv.verify_attn_scaled(*args, workspace=ws)
    torch.cuda.synchronize()
    assert sv.workspace_error(ws) == 0
    check([R + 130, 300], R, G * Hkv, Hkv, D, 16, 16, "bf16", seed=3, masks=[chain_masks(R)] * 2)
