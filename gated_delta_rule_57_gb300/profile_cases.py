"""Run the hot path on one named workload, for profilers.

    python -m gated_delta_rule_57_gb300.profile_cases prefill [--B 8] [--calls 4]
    python -m gated_delta_rule_57_gb300.profile_cases decode  [--calls 4]
    python -m gated_delta_rule_57_gb300.profile_cases spec    [--calls 4]
    python -m gated_delta_rule_57_gb300.profile_cases long    [--T 65536] [--nseg 5|decay] [--calls 4]
    python -m gated_delta_rule_57_gb300.profile_cases t4k     [--nseg 4|decay|1] [--calls 4]
    python -m gated_delta_rule_57_gb300.profile_cases prompt  [--B 2] [--calls 4]
    python -m gated_delta_rule_57_gb300.profile_cases paged   --T 4096 [--B 64] [--calls 4]
    python -m gated_delta_rule_57_gb300.profile_cases latent_prompt [--B 2] [--calls 4]
    python -m gated_delta_rule_57_gb300.profile_cases latent_paged --T 4096 [--B 64] [--calls 4]
    python -m gated_delta_rule_57_gb300.profile_cases rope    [--B 2] [--calls 4]

Draws the seeded synthetic inputs on the GPU, then makes `calls` back-to-back
calls of kda_chunk_fwd (prefill: B x 8192 tokens x 32 heads, d = 128, bf16)
or kda_decode_step (256 sequences x 32 heads, d = 128), or rounds of
kda_decode_multi (the same 256 x 32 states, 4 draft tokens: verify then
commit), or kda_chunk_fwd_segmented (long: one sequence of T tokens x 32 heads
split into nseg segments; three launches per call; --nseg decay plans the
split on the device from the decay probe: five launches; t4k: the same on
one sequence of 4096 tokens x 32 heads, half of them with g = -4.99), or
kda_attn_prompt (B prompts of 8192 tokens, 32 query and 8 key heads, d = 128) or
kda_attn_paged (one token of B requests over T cached tokens each, pages of 64;
the same heads), or their counterparts over latents (32 heads, 64 rotated channels), or
kda_kv_append_rope (B prompts of 8192 tokens, 32 query and 8 key heads, d = 128). Under a profiler,
skip the first calls as warm-up (e.g. ncu -s 2 -c 1 -k regex:kda_).
"""
import argparse

import torch

from . import inputs, kda, latent


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("which", choices=["prefill", "decode", "spec", "long", "t4k", "prompt", "paged", "latent_prompt", "latent_paged", "rope"])
    ap.add_argument("--B", type=int, default=8)
    ap.add_argument("--T", type=int, default=65536)
    ap.add_argument("--nseg", default="5", help="segment count, or 'decay'")
    ap.add_argument("--calls", type=int, default=4)
    args = ap.parse_args()
    dev = torch.device("cuda", 0)
    if args.which == "prefill":
        w = inputs.PREFILL_B8_T8K
        x = inputs.prefill_inputs(w, dev, B=args.B)
        o = torch.empty_like(x["v"])
        hT = torch.empty(args.B, w.H, w.dk, w.dv, device=dev)
        for _ in range(args.calls):
            kda.kda_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["h0"], o=o, hT=hT)
    elif args.which == "decode":
        w = inputs.DECODE_N256
        x = inputs.decode_inputs(w, dev, steps=args.calls)
        for s in range(args.calls):
            kda.kda_decode_step(x["q"][s], x["k"][s], x["v"][s], x["g"][s], x["beta"][s], x["S"])
    elif args.which in ("long", "t4k"):
        # t4k: B=1, T=4096, H=32 with the stress heads (g = -4.99); --T is ignored
        w = inputs.PREFILL_T1M if args.which == "long" else inputs.PREFILL_T4K
        if args.which == "t4k":
            args.T = w.T
        x = inputs.prefill_inputs(w, dev, T=args.T)
        o = torch.empty_like(x["v"])
        hT = torch.empty(w.B, w.H, w.dk, w.dv, device=dev)
        nseg = 0 if args.nseg == "decay" else int(args.nseg)  # 0: planned on the device
        ws = torch.empty(kda.kda_chunk_fwd_segmented_workspace_size(
            w.B, args.T, w.H, w.dk, w.dv, nseg=nseg), dtype=torch.uint8, device=dev)
        for _ in range(args.calls):
            kda.kda_chunk_fwd_segmented(x["q"], x["k"], x["v"], x["g"], x["beta"], None,
                                        nseg=nseg, o=o, hT=hT, workspace=ws)
    elif args.which == "prompt":
        qkv = torch.randn(args.B * 8192, 48, 128, device=dev).bfloat16()
        cu = torch.arange(args.B + 1, dtype=torch.int32, device=dev) * 8192
        for _ in range(args.calls):
            kda.kda_attn_prompt(qkv[:, :32], qkv[:, 32:40], qkv[:, 40:], cu, max_len=8192)
    elif args.which == "paged":
        per = -(-args.T // 64)
        kc, vc = (torch.randn(args.B * per, 8, 64, 128, device=dev).bfloat16() for _ in range(2))
        table = torch.randperm(args.B * per, device=dev).to(torch.int32).view(args.B, per)
        q = torch.randn(args.B, 32, 128, device=dev).bfloat16()
        cu = torch.arange(args.B + 1, dtype=torch.int32, device=dev)
        kv = torch.full((args.B,), args.T, dtype=torch.int32, device=dev)
        for _ in range(args.calls):
            kda.kda_attn_paged(q, kc, vc, table, cu, kv, max_q=1)
    elif args.which == "latent_prompt":
        t = args.B * 8192
        q, kv, k_r = (torch.randn(t, *s, device=dev).bfloat16() for s in ((32, 192), (32, 256), (64,)))
        cu = torch.arange(args.B + 1, dtype=torch.int32, device=dev) * 8192
        for _ in range(args.calls):
            latent.kda_attn_latent_prompt(q, kv[..., :128], k_r, kv[..., 128:], cu, max_len=8192)
    elif args.which == "latent_paged":
        per = -(-args.T // 64)
        cache = torch.randn(args.B * per, 64, 576, device=dev).bfloat16()
        table = torch.randperm(args.B * per, device=dev).to(torch.int32).view(args.B, per)
        q = torch.randn(args.B, 32, 576, device=dev).bfloat16()
        cu = torch.arange(args.B + 1, dtype=torch.int32, device=dev)
        kv = torch.full((args.B,), args.T, dtype=torch.int32, device=dev)
        for _ in range(args.calls):
            latent.kda_attn_latent_paged(q, cache, table, cu, kv, scale=192 ** -0.5, max_q=1)
    elif args.which == "rope":
        t = args.B * 8192
        qkv = torch.randn(t, 48, 128, device=dev).bfloat16()
        kc, vc = (torch.empty(t // 64, 8, 64, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
        i = torch.arange(t, dtype=torch.int32, device=dev)
        turns = latent.kda_rope_turns([10000.0 ** (-j / 64) for j in range(64)])
        out = torch.empty(t, 32, 128, dtype=torch.bfloat16, device=dev)
        for _ in range(args.calls):
            latent.kda_kv_append_rope(qkv[:, :32], qkv[:, 32:40], qkv[:, 40:], i, i % 8192, turns, kc, vc, q_out=out)
    else:
        w = inputs.DECODE_N256
        x = inputs.prefill_inputs(inputs.PrefillWorkload("draft", w.N, 4, w.H, w.dk, w.dv, w.io,
                                                         w.seed, h0_std=w.S_std), dev)
        for _ in range(args.calls):
            kda.kda_decode_multi(x["q"], x["k"], x["v"], x["g"], x["beta"], x["h0"])
            kda.kda_decode_multi(x["q"], x["k"], x["v"], x["g"], x["beta"], x["h0"], commit=True,
                                 want_o=False)
    torch.cuda.synchronize()
    print(f"{args.which}: {args.calls} calls done")


if __name__ == "__main__":
    main()
