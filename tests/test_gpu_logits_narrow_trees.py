"""Penalties over a tree's ancestors where the tree is narrow: up to R - 1 of them, whatever R is."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from oracle import logits as olog
from tests.test_gpu_logits_process import on_gpu, same

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("R", [2, 3, 4, 5, 6, 7, 8, 9, 16, 33, 64])
@pytest.mark.parametrize("wide", [0, 1, 2])
def test_narrow_trees(R, wide):
    """Parents at most `wide` rows further back than the row in front (0: a chain given as a tree), ids that repeat."""
    r = np.random.default_rng(R + wide)
    B, V = 40, 97
    kw = dict(history=r.integers(0, V, (B, 3)), prompt_len=r.integers(0, 4, B),
              block_tokens=r.integers(0, 5, (B, R)),
              parent=np.array([[-1] + [max(0, i - 1 - r.integers(0, wide + 1)) for i in range(1, R)] for _ in range(B)]),
              repetition=r.uniform(1, 2, B).astype(np.float32), frequency=r.normal(size=B).astype(np.float32),
              presence=r.normal(size=B).astype(np.float32))
    x = torch.from_numpy(r.normal(size=(B, R, V)).astype(np.float32))
    same(sv.logits_process(x.to(DEV), **on_gpu(kw)), olog.process(x.numpy(), fp=np.float32, **kw))
