"""Order on the stream: what follows a one-token attention sees all of it, whether or not
the joining kernel has anything to join."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_76_gb300 as sv
from tests.test_gpu_cache_side import DEV, TYPES, dev, make_cache

pytestmark = pytest.mark.gpu


# (KV heads, query heads to each, D, type, lengths): few KV heads and tables of more than 4096
# positions, so the joining kernel is launched; only the last two have a sequence for it
CASES = [
    (1, 8, 256, "bf16", [3000 - 97 * i for i in range(24)]),
    (2, 4, 128, "f16", [1 + 61 * i for i in range(33)]),
    (4, 4, 64, "e4m3", [2048, 7, 0, 1500, 900, 33] * 4),
    (1, 16, 128, "bf16", [700] * 40),
    (1, 4, 128, "f16", [20000, 300]),
    (1, 8, 64, "bf16", [30000]),
]


@pytest.fixture(scope="module")
def calls():
    """For each case: the arguments of a call, a sink for its output's rows, and what the call
    gives alone."""
    out = []
    for i, (Hkv, G, D, cache, lens) in enumerate(CASES):
        k, v, table, sc = make_cache(lens, Hkv, D, 16, cache, 70 + i, extra=300)
        qt = "f16" if cache == "e4m3" else cache
        q = torch.randn((len(lens), Hkv * G, D),
                        generator=torch.Generator().manual_seed(i)).to(TYPES[qt])
        kw = {} if sc[0] is None else dict(k_scale=sc[0].to(DEV), v_scale=sc[1].to(DEV))
        args = [q.to(DEV), k.to(DEV), v.to(DEV), dev(table), dev(lens)]
        torch.cuda.synchronize()
        o, lse = sv.decode_attn(*args, **kw)
        torch.cuda.synchronize()
        rows = dev(np.arange(len(lens)), torch.int64)
        out.append((args, kw, rows, o.clone(), lse.clone()))
    return out


def run_all(calls, ws, rounds):
    """The cases in turn, `rounds` times, nothing waited for; each output is read at once by
    a chained call.  Returns what that call stored, and the log-sum-exps."""
    got = []
    for _ in range(rounds):
        for args, kw, rows, o, _ in calls:
            out, lse = sv.decode_attn(*args, workspace=ws, **kw)
            sink = [torch.empty((o.shape[0], 1) + o.shape[1:], dtype=o.dtype, device=DEV)
                    for _ in range(2)]
            sv.append_tokens(out, out, *sink, rows, rope_base=0)
            out.fill_(-7.0)        # what comes next may overwrite the output
            got.append((sink[0][:, 0], lse))
    return got


def check(calls, got):
    for i, (o, lse) in enumerate(got):
        _, _, _, ref, lref = calls[i % len(calls)]
        assert torch.equal(o, ref) and torch.equal(lse, lref), i


def test_calls_back_to_back_on_one_workspace(calls):
    ws = sv.new_workspace(max(sv.decode_attn_workspace_size(1, Hkv * G, Hkv, D)
                              for Hkv, G, D, _, _ in CASES), DEV)
    check(calls, run_all(calls, ws, 10))
    # workspaces of their own: freed on return, other tensors' memory at once
    check(calls, run_all(calls, None, 10))


def test_calls_back_to_back_in_a_captured_graph(calls):
    ws = sv.new_workspace(max(sv.decode_attn_workspace_size(1, Hkv * G, Hkv, D)
                              for Hkv, G, D, _, _ in CASES), DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_all(calls, ws, 1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_all(calls, ws, 2)
    for _ in range(5):
        graph.replay()
        check(calls, [(o.clone(), lse.clone()) for o, lse in got])
        for o, lse in got:
            o.zero_()
            lse.zero_()
