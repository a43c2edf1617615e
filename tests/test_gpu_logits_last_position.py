"""logits_process on one row per sequence, where the distance from row to row is the batch's."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import logits as olog
from tests.test_gpu_logits_process import make, on_gpu, same

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("new", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B", [1, 3])
def test_the_last_position_of_a_longer_tensor(new, B):
    V = 1021
    x, kw = make(B, 1, V, 50, new, 3)
    ref, g = olog.process(x.float().numpy(), fp=np.float32, **kw), on_gpu(kw)
    whole = torch.full((B, 7, V), float("nan"), dtype=x.dtype, device=DEV)
    whole[:, -1:] = x.to(DEV)
    same(sv.logits_process(whole[:, -1:], **g), ref)
    # a padded last layer's rows, one per sequence
    wide = torch.full((B, V + 3), float("nan"), dtype=x.dtype, device=DEV)
    wide[:, :V] = x.to(DEV)[:, 0]
    same(sv.logits_process(wide[:, :V].unsqueeze(1), **g), ref)
    if new == "f32":                            # in place only where the rows stand together
        y = x.to(DEV)
        assert sv.logits_process(y, out=y, **g) is y
        same(y, ref)
        if B > 1:
            with pytest.raises(ValueError, match="contiguous"):
                sv.logits_process(whole[:, -1:], out=whole[:, -1:], **g)


def test_rows_that_are_not_equally_far_apart_are_refused():
    x = torch.zeros((3, 4, 64), device=DEV)
    with pytest.raises(ValueError, match="equally far apart"):
        sv.logits_process(x[:, :2])
    with pytest.raises(ValueError, match="contiguous over V"):
        sv.logits_process(x[:, :1, ::2])
