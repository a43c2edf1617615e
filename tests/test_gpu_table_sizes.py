"""Block tables at the batch sizes where a launch needs more shared memory than it has by
default."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SIZES = """
import numpy as np, torch
import speculative_decoding_verification_76_gb300 as sv
from oracle import tables
rng = np.random.default_rng(0)
for B in (257, 6137, 6138, 6143, 6144, 8192):
    ctx, add = rng.integers(0, 30, B), rng.integers(0, 4, B)
    table = np.full((B, 3), 5)
    lst = np.arange(4 * B)
    t = lambda x: torch.as_tensor(x).int().cuda()
    tab = t(table)
    e = sv.extend_tables(t(ctx), t(add), tab, t(lst), t([4 * B]), 16, 4 * B)
    ref = tables.extend(ctx, add, table, lst, 4 * B, 16, 4 * B)
    np.testing.assert_array_equal(tab.cpu().numpy(), ref["block_table"])
    for k in ("slot_map", "positions", "cu_len", "new_len", "status"):
        np.testing.assert_array_equal(e[k].cpu().numpy(), ref[k], err_msg=f"{B} {k}")
    held, out = t(lst), e["new_len"]
    n, st = sv.release_pages(tab, out, t([0] * B), held, e["free_count"], 16)
    lref, nref, sref = tables.release(ref["block_table"], ref["new_len"], [0] * B, lst,
                                      ref["free_count"], 16)
    np.testing.assert_array_equal(held.cpu().numpy(), lref)
    assert n.item() == nref and st.tolist() == sref.tolist()
print("sizes ok")
"""


def test_table_batches_in_ascending_order_in_a_process_of_their_own():
    """The limit of a launch's shared memory counts the kernel's own static bytes, and once
    raised by a larger batch it stays: sizes around it, from small to large, in a process that
    has made no larger call."""
    r = subprocess.run([sys.executable, "-c", SIZES], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "sizes ok" in r.stdout, r.stderr[-2000:]
