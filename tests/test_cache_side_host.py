"""Faults of the cache-side calls that show without a GPU: read from the sources, or from
what the host entry points answer before anything is launched."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_76_gb300", "csrc")


def kernels(name):
    """(name, body) of every kernel of a source file, comments taken out."""
    with open(os.path.join(CSRC, name)) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__ void __launch_bounds__\([^{;]*?\)\s*(\w+)\s*\(", src):
        at = src.index("{", m.end())
        end, depth = at, 0
        while True:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
            if depth == 0:
                break
        yield m.group(1), src[at:end]


@pytest.mark.parametrize("name,count", [("tables.cu", 2), ("append_tokens.cu", 1),
                                        ("decode.cu", 2)])
def test_no_chained_kernel_ends_without_waiting(name, count):
    """These kernels are programmatic dependents.  The next operation on the stream is ordered
    behind them alone, so a block that returns before the wait lets it overtake the kernel in
    front."""
    found = list(kernels(name))
    assert len(found) == count
    for kernel, body in found:
        waits = [m.start() for m in re.finditer(r"(?<!return )chain_wait\(\);", body)]
        assert len(waits) == 1, kernel
        # a bare return in front of the wait (a lambda's returns carry a value; an exit that
        # waits reads `return chain_wait();`)
        assert not re.search(r"\breturn;", body[:waits[0]]), kernel


# ------------------------------------------------------------------ sizes near 2^31
@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_verification_76_gb300 as sv
    from speculative_decoding_verification_76_gb300 import build
    build.build()
    return sv.load()


def test_decode_attn_refuses_rows_and_batches_near_two_to_the_31(lib):
    """The position loop looks up to two rounds of a block's warps past a sequence's end, in
    32 bits.  (The workspace is refused behind the sizes: nothing is ever launched here.)"""
    from tests.test_oracle_cache_side import DECODE

    def call(**change):
        return lib.spec_decode_attn(*dict(DECODE, pages=1, maxp=1, wsb=0, **change).values())
    top = 2 ** 31 - 1
    for n in (top, top - 1, top - 127, top - 511):
        assert call(B=1, P=n) == 2, n
        assert call(B=n, P=1) == 2, n
    assert call(B=1, P=top - 512) == 1
    assert call(B=top - 512, P=1) == 1


def test_tables_refuse_rows_near_two_to_the_31(lib):
    """Rows of page ids are walked eight blocks' widths at a time, in 32 bits."""
    import ctypes
    top = 2 ** 31 - 1
    p = [ctypes.c_void_p(1 << (33 + i)) for i in range(11)]   # apart by more than the sizes
    for maxp in (top, top - 1, top - 4095):
        assert lib.spec_extend_tables(p[0], p[1], 1, 1, p[10], maxp, p[2], 8, p[3], 0, p[4], p[5],
                                      p[6], p[7], p[8], p[9], None) == 2
        assert lib.spec_release_pages(p[10], maxp, p[1], p[2], 1, 1, p[3], 8, p[4], p[5], p[6],
                                      None) == 2


def test_append_refuses_tokens_that_no_grid_counts(lib):
    """Two rows to a block: T + 1 is counted in 32 bits."""
    from tests.test_oracle_cache_side import APPEND
    top = 2 ** 31 - 1
    assert lib.spec_append_tokens(*dict(APPEND, T=top, slots=None).values()) == 2
    assert lib.spec_append_tokens(*dict(APPEND, T=top - 1, slots=None).values()) == 1


def test_tables_refuse_outputs_that_overlap(lib):
    """No output may share memory with an input or with another output, in part either: some
    blocks would read what others have written.  (B 2, four pages a row, a pool of 8, 64 rows.)"""
    import ctypes
    at = {k: 1 << (20 + i) for i, k in enumerate(
        "ctx add table lst cnt slots pos cu new left status".split())}
    size = dict(ctx=8, add=8, table=32, lst=32, cnt=4, slots=512, pos=256, cu=12, new=8, left=4,
                status=8)
    outs = "table slots pos cu new left status".split()

    def extend(**move):
        a = {k: ctypes.c_void_p(v) for k, v in dict(at, **move).items()}
        return lib.spec_extend_tables(a["ctx"], a["add"], 2, 16, a["table"], 4, a["lst"], 8,
                                      a["cnt"], 64, a["slots"], a["pos"], a["cu"], a["new"],
                                      a["left"], a["status"], None)
    for o in outs:
        for other in at:
            if other != o:
                for by in (size[other] - 4, 4 - size[o]):   # the last word, the first word
                    assert extend(**{o: at[other] + by}) == 1, (o, other, by)
    rel = {k: 1 << (20 + i) for i, k in enumerate("table len keep lst cnt total status".split())}
    rsize = dict(table=32, len=8, keep=8, lst=32, cnt=4, total=4, status=8)

    def release(**move):
        a = {k: ctypes.c_void_p(v) for k, v in dict(rel, **move).items()}
        return lib.spec_release_pages(a["table"], 4, a["len"], a["keep"], 2, 16, a["lst"], 8,
                                      a["cnt"], a["total"], a["status"], None)
    for o in ("lst", "total", "status"):
        for other in rel:
            if other != o:
                for by in (rsize[other] - 4, 4 - rsize[o]):
                    assert release(**{o: rel[other] + by}) == 1, (o, other, by)
