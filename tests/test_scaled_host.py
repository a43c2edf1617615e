"""What the sources of the scaled cache's kernels have to hold, read without a GPU."""
import re

import pytest

from tests.test_cache_side_host import kernels


@pytest.mark.parametrize("name,count", [("rotate.cu", 1), ("append_scaled.cu", 3), ("logits.cu", 1),
                                        ("attn_scaled.cuh", 2)])
def test_no_chained_kernel_ends_without_waiting(name, count):
    """Programmatic dependents: a block that returns before the wait lets the next operation on the
    stream overtake the kernel in front."""
    found = list(kernels(name))
    assert len(found) == count
    for kernel, body in found:
        waits = [m.start() for m in re.finditer(r"chain_wait\(\);", body)]
        assert len(waits) == 1, kernel
        assert not re.search(r"\breturn;", body[:waits[0]]), kernel
        # the next one may only be let in by a block that has itself waited: it reads lengths early
        assert "chain_next" not in body[:waits[0]], kernel
