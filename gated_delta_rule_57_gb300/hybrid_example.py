"""A small hybrid stack served end to end: three KDA layers to one softmax-
attention layer (the ratio of the orkas.ai page "Kimi K3 architecture", section
"Sequence: three quarters of the layers stopped reading everything"), random
weights.

    python -m gated_delta_rule_57_gb300.hybrid_example [--prompts 3] [--tokens 200] [--steps 20]

Prompts go through the stack whole: the KDA layers leave a state per head, the
attention layers their keys and values in the paged cache. Then every request
gains one token per step: kda_decode_step advances the states, kda_kv_plan takes
pages, kda_kv_append writes the new keys and values, kda_attn_paged attends
over the cache. The outputs of the steps are compared with one pass over the
whole sequences.
"""
from __future__ import annotations

import argparse

import torch

from . import kda

PAGE = 64


class Layer:
    def __init__(self, gen, dim, hq, hkv, d, softmax):
        self.softmax, self.hq, self.hkv, self.d = softmax, hq, hkv, d

        def w(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") * shape[0] ** -0.5).bfloat16()

        # attention: q, k, v; KDA: q, k, v, log-decay, beta (all heads alike)
        self.w_in = w(dim, (hq + 2 * hkv) * d if softmax else 4 * hq * d + hq)
        self.w_out = w(hq * d, dim)

    def project(self, x):
        y = x @ self.w_in
        if self.softmax:
            return y.view(-1, self.hq + 2 * self.hkv, self.d)
        h, d = self.hq, self.d
        q, k, v, g, b = y.split([h * d, h * d, h * d, h * d, h], -1)
        unit = lambda t: torch.nn.functional.normalize(t.float().unflatten(-1, (h, d)), dim=-1).bfloat16()  # noqa: E731
        g = -5.0 * torch.sigmoid(g.float().unflatten(-1, (h, d)) - 3.0)
        return unit(q), unit(k), v.unflatten(-1, (h, d)).contiguous(), g.contiguous(), torch.sigmoid(b.float()).contiguous()


def norm(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)


class Stack:
    """Layers, and what a batch of N requests keeps between calls."""

    def __init__(self, layers=4, dim=256, hq=4, hkv=2, d=64, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer(gen, dim, hq, hkv, d, softmax=i % 4 == 3) for i in range(layers)]

    def start(self, n, most):
        per = -(-most // PAGE)
        pages = n * per
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((n, per), -1, **i32)
        self.free = torch.arange(pages, **i32)
        self.ring = torch.tensor([0, pages], **i32)
        self.kv_len = torch.zeros(n, **i32)
        self.status = torch.zeros(1, **i32)
        # a layer's own caches; the plan of a step serves all layers
        self.caches = [tuple(torch.empty(pages, x.hkv, PAGE, x.d, dtype=torch.bfloat16, device="cuda")
                             for _ in range(2)) if x.softmax else None for x in self.layers]
        self.states = [None] * len(self.layers)

    def plan(self, lengths, tokens):
        self.kv_len, cu, slots, self.ring = kda.kda_kv_plan(
            self.kv_len, lengths, self.table, self.free, self.ring, page_size=PAGE, max_tokens=tokens, status=self.status)
        return cu, slots

    def prompt(self, x):
        """x [N, T, dim], from empty: hidden states of all tokens."""
        n, t, _ = x.shape
        cu, slots = self.plan(torch.full_like(self.kv_len, t), n * t)
        for i, layer in enumerate(self.layers):
            y = layer.project(norm(x))
            if layer.softmax:
                q, k, v = y.split([layer.hq, layer.hkv, layer.hkv], 1)
                kda.kda_kv_append(k, v, slots, *self.caches[i], status=self.status)
                o, _ = kda.kda_attn_prompt(q, k, v, cu, max_len=t, want_lse=False, status=self.status)
            else:
                o, self.states[i] = kda.kda_chunk_fwd(*y, status=self.status)
            x = x + o.reshape(n, t, -1) @ layer.w_out
        return x

    def step(self, x):
        """x [N, dim], one new token per request: its hidden states."""
        n = x.shape[0]
        cu, slots = self.plan(self.kv_len + 1, n)
        for i, layer in enumerate(self.layers):
            y = layer.project(norm(x))
            if layer.softmax:
                q, k, v = y.split([layer.hq, layer.hkv, layer.hkv], 1)
                kda.kda_kv_append(k, v, slots, *self.caches[i], status=self.status)
                o, _ = kda.kda_attn_paged(q, *self.caches[i], self.table, cu, self.kv_len, max_q=1, want_lse=False,
                                          status=self.status)
            else:
                o = kda.kda_decode_step(*y, self.states[i], status=self.status)
            x = x + o.reshape(n, -1) @ layer.w_out
        return x


def run(prompts=3, tokens=200, steps=20, layers=8, dim=256, hq=4, hkv=2, d=64, seed=0):
    """Largest difference between the steps and one pass, relative to the
    outputs' root mean square; and the status word."""
    stack = Stack(layers, dim, hq, hkv, d, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    x = torch.randn(prompts, tokens + steps, dim, generator=gen, device="cuda").bfloat16()
    stack.start(prompts, tokens + steps)
    stack.prompt(x[:, :tokens].contiguous())
    got = torch.stack([stack.step(x[:, tokens + s]) for s in range(steps)], 1)
    status = int(stack.status)
    stack.start(prompts, tokens + steps)
    want = stack.prompt(x)[:, tokens:]
    status |= int(stack.status)
    rms = want.float().square().mean().sqrt()
    return float((got.float() - want.float()).abs().max() / rms), status


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--prompts", type=int, default=3)
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    off, status = run(a.prompts, a.tokens, a.steps)
    print(f"{a.prompts} prompts of {a.tokens} tokens, {a.steps} steps: steps against one pass over everything: "
          f"largest difference {off:.3e} of the rms; status {status}")


if __name__ == "__main__":
    main()
