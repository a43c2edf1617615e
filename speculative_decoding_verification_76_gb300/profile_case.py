"""One library call on a workload, for profilers (ncu -k ... -c ...).

    python -m speculative_decoding_verification_76_gb300.profile_case attn NAME B REPS
    python -m speculative_decoding_verification_76_gb300.profile_case sampler NAME B REPS
    python -m speculative_decoding_verification_76_gb300.profile_case decode NAME B REPS
    python -m speculative_decoding_verification_76_gb300.profile_case decode_e4m3 NAME B REPS
    python -m speculative_decoding_verification_76_gb300.profile_case append_e4m3 NAME B REPS

Builds the named synthetic workload with B sequences (same generator as the tests
and the bench) and makes REPS calls of the verify attention's partial pass, of the
acceptance sampler (no p returned), of the one-token attention over the same cache
(as it is or in e4m3) or of a packed append of 256 tokens a sequence into an e4m3
cache, then synchronises.
"""
import sys

import torch

from . import api as sv
from . import workloads as wl


def main(argv):
    what, name, B = argv[0], argv[1], int(argv[2])
    reps = int(argv[3]) if len(argv) > 3 else 3
    spec = wl.SPECS[name].with_(B=B)
    if what == "attn":
        w = wl.make_attention_inputs(spec, device="cuda")
        # a chain needs no mask (the causal block), as in the verify step
        anc = sv.tree_prepare(w.parent, w.ctx_len)[0] if spec.is_tree else None
        call = sv.AttnCall(w.q, w.k_cache, w.v_cache, w.block_table, w.ctx_len, anc,
                           num_splits=spec.num_splits)
        for _ in range(reps):
            call.partials()
    elif what == "sampler":
        w = wl.make_sampler_inputs(spec, seed=spec.seed, device="cuda")
        cfg = sv.SamplerConfig(temperature=spec.temperature, top_k=spec.top_k, top_p=spec.top_p,
                               greedy=spec.greedy)
        for _ in range(reps):
            if spec.is_tree:
                sv.accept_sample_tree(w.logits, w.draft_probs, w.draft_tokens, w.parent,
                                      w.uniforms, cfg)
            else:
                sv.accept_sample(w.logits, w.draft_probs, w.draft_tokens, w.uniforms, cfg)
    elif what in ("decode", "decode_e4m3"):
        w = wl.make_attention_inputs(spec, device="cuda")
        k, v, sc = w.k_cache, w.v_cache, None
        if what == "decode_e4m3":      # N(0, 1) values, stored under one scale
            sc = torch.full((spec.Hkv,), 0.0125, device="cuda")
            k, v = ((x / 0.0125).clamp(-448, 448).to(torch.float8_e4m3fn) for x in (k, v))
        q, seen = w.q[:, 0], w.ctx_len + spec.R
        ws = sv.new_workspace(sv.decode_attn_workspace_size(B, spec.Hq, spec.Hkv, spec.D), "cuda")
        for _ in range(reps):
            sv.decode_attn(q, k, v, w.block_table, seen, k_scale=sc, v_scale=sc, workspace=ws)
    elif what == "append_e4m3":
        T = 256 * B
        q, k, v = (torch.randn((T, h, spec.D), device="cuda").bfloat16()
                   for h in (spec.Hq, spec.Hkv, spec.Hkv))
        kc, vc = (torch.zeros((T // 16, 16, spec.Hkv, spec.D), dtype=torch.float8_e4m3fn,
                              device="cuda") for _ in range(2))
        sc = torch.full((spec.Hkv,), 0.0125, device="cuda")
        slots, out = torch.randperm(T, device="cuda"), torch.empty_like(q)
        pos = torch.arange(T, device="cuda", dtype=torch.int32)
        for _ in range(reps):
            sv.append_tokens(k, v, kc, vc, slots, pos, q=q, q_out=out, k_scale=sc, v_scale=sc)
    else:
        raise SystemExit(f"unknown case {what!r}")
    torch.cuda.synchronize()
    print("ok", what, name, B, reps)


if __name__ == "__main__":
    main(sys.argv[1:])
