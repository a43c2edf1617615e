"""KV commit on the caches of the packed append: e4m3, fp16 and heads of 256 move bit for
bit along the accepted path."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import commit
from tests.test_gpu_commit import _case, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,P", [
    (torch.float8_e4m3fn, 64, 5), (torch.float8_e4m3fn, 128, 16), (torch.float8_e4m3fn, 256, 1),
    (torch.float16, 64, 24), (torch.float16, 128, 16), (torch.float16, 256, 7),
    (torch.bfloat16, 256, 16)])
@pytest.mark.parametrize("R,Hkv", [(2, 1), (16, 3), (64, 2)])
def test_tree_paths_move_in_every_cache_type(dtype, D, P, R, Hkv):
    ctx, table, k, v, acc, paths, path, parent = _case(5, R, Hkv, D, P, dtype, D + R, True)
    ko, vo, new_len, keep, status = _run(ctx, table, k, v, acc, path, R, parent)
    bits = torch.uint8 if dtype == torch.float8_e4m3fn else torch.int16
    for src, out in ((k, ko), (v, vo)):
        ref = commit.compact_path(src.view(bits).double().numpy(), table, ctx, paths, P)
        np.testing.assert_array_equal(out.view(bits).double().numpy(), ref)
    n = commit.committed_length(ctx, acc)
    np.testing.assert_array_equal(new_len, n)
    np.testing.assert_array_equal(keep, (n + P - 1) // P)
    assert (status == 0).all()


@pytest.mark.parametrize("dtype,D", [(torch.float8_e4m3fn, 256), (torch.float16, 64)])
def test_chains_and_bad_paths_leave_them_alone(dtype, D):
    B, R = 4, 6
    ctx, table, k, v, acc, _, _, _ = _case(B, R, 2, D, 16, dtype, 3, False)
    bits = torch.uint8 if dtype == torch.float8_e4m3fn else torch.int16
    ko, vo, new_len, _, status = _run(ctx, table, k, v, acc, None, R)
    assert torch.equal(ko.view(bits), k.view(bits)) and torch.equal(vo.view(bits), v.view(bits))
    np.testing.assert_array_equal(new_len, commit.committed_length(ctx, acc))
    path = np.tile(np.array([2, 1, 3, 4, 5, -1], np.int32), (B, 1))     # does not ascend
    ko, vo, new_len, _, status = _run(ctx, table, k, v, np.full(B, 3, np.int32), path, R)
    assert torch.equal(ko.view(bits), k.view(bits)) and torch.equal(vo.view(bits), v.view(bits))
    assert (status == sv.api.SEQ_BAD_TREE).all() and (new_len == ctx).all()
