"""That every key counts, and only as much as it should, where a bound that grows with
the sum of all values would hide one: each channel's value is 1 at a single key and 0
elsewhere, so an output is that key's probability p, and its bound (attn_ref's, with
A = |o| = p) is a fraction of p. Also the attention layers of the hybrid example, each
call against the 64-bit definition on the layer's own operands."""
import pytest
import torch

import attn_ref
from gated_delta_rule_57_gb300 import hybrid_example, kda
from test_gpu_attn import BF, DEV, F32, cumulative, ints, randn

pytestmark = pytest.mark.gpu


def one_key_per_channel(kv, hkv, d, io, seed):
    """[kv, hkv, d]: channel c of head h is 1 at one key only, the channels' keys being
    the ends of the request and of its tiles and pages, and any others."""
    g = torch.Generator().manual_seed(seed)
    ends = sorted({x for t in (0, 16, 64, 128, kv // 2 // 128 * 128, kv // 128 * 128, kv // 16 * 16, kv) for x in (t - 1, t) if 0 <= x < kv})
    v = torch.zeros(kv, hkv, d)
    for h in range(hkv):
        keys = torch.cat([torch.tensor(ends), torch.randint(0, kv, (d,), generator=g)])[:d]
        v[keys, h, torch.arange(d)] = 1.0
    return v.to(io).to(DEV)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("kv,n,hq,hkv,d,page", [(4000, 1, 8, 2, 128, 64), (4099, 3, 8, 2, 64, 16), (2600, 70, 4, 1, 128, 128),
                                               (9001, 1, 16, 1, 128, 32), (1500, 300, 6, 3, 64, 1024)])
def test_every_cached_key_counts(kv, n, hq, hkv, d, page, io):
    g = torch.Generator(device=DEV).manual_seed(kv)
    per = -(-kv // page)
    table = torch.randperm(per, generator=g, device=DEV).to(torch.int32)[None].contiguous()
    k, v = randn(g, kv, hkv, d, io=io), one_key_per_channel(kv, hkv, d, io, kv)
    kc, vc = (torch.full((per, hkv, page, d), float("nan"), dtype=io, device=DEV) for _ in range(2))
    at = torch.arange(kv, device=DEV)
    slots = (table[0, at // page] * page + at % page).to(torch.int32)
    kda.kda_kv_append(k, v, slots, kc, vc)
    q = randn(g, n, hq, d, io=io)
    ref = attn_ref.attend(q, k, v, kv, d ** -0.5)
    for ws in (None, torch.empty(0, device=DEV)):
        o, lse = kda.kda_attn_paged(q, kc, vc, table, ints([0, n]), ints([kv]), max_q=n, workspace=ws)
        attn_ref.check(o, lse, ref)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("n,hq,hkv,d", [(1, 4, 2, 64), (129, 8, 2, 128), (1000, 4, 4, 64), (3000, 2, 1, 128)])
def test_every_key_of_a_prompt_counts(n, hq, hkv, d, io):
    g = torch.Generator(device=DEV).manual_seed(n)
    q, k, v = randn(g, n, hq, d, io=io), randn(g, n, hkv, d, io=io), one_key_per_channel(n, hkv, d, io, n)
    ref = attn_ref.attend(q, k, v, n, d ** -0.5)
    for ws in (None, torch.empty(0, device=DEV)):
        o, lse = kda.kda_attn_prompt(q, k, v, ints([0, n]), workspace=ws)
        attn_ref.check(o, lse, ref)


@pytest.mark.parametrize("kw", [dict(prompts=3, tokens=5, steps=70), dict(prompts=2, tokens=63, steps=4, d=128, hq=8)])
def test_attention_layers_of_the_hybrid_example(kw, monkeypatch):
    """Keys and values that each layer hands over, kept here in order, and every output
    of its attention against the definition over them."""
    prompts, checked = kw["prompts"], [0]
    kept = {}  # by cache: keys, values [request][tokens so far]
    last = {}
    append, prompt, paged = kda.kda_kv_append, kda.kda_attn_prompt, kda.kda_attn_paged

    def per_request(x):
        return x.unflatten(0, (prompts, -1))

    def on_append(k, v, slots, kc, vc, **a):
        new = [per_request(x).clone() for x in (k, v)]
        # a prompt starts the caches anew
        kept[id(kc)] = new if k.shape[0] > prompts else [torch.cat([x, y], 1) for x, y in zip(kept[id(kc)], new)]
        last["cache"] = id(kc)
        return append(k, v, slots, kc, vc, **a)

    def held_to(q, o):
        ks, vs = kept[last["cache"]]
        for r in range(prompts):
            rows = per_request(q)[r]
            ref = attn_ref.attend(rows, ks[r], vs[r], ks.shape[1], q.shape[2] ** -0.5)
            attn_ref.check(per_request(o)[r], None, ref)
            checked[0] += 1

    def on_prompt(q, k, v, cu, **a):
        o, lse = prompt(q, k, v, cu, **a)
        held_to(q, o)
        return o, lse

    def on_paged(q, kc, vc, *a, **b):
        assert id(kc) == last["cache"]
        o, lse = paged(q, kc, vc, *a, **b)
        held_to(q, o)
        return o, lse

    monkeypatch.setattr(kda, "kda_kv_append", on_append)
    monkeypatch.setattr(kda, "kda_attn_prompt", on_prompt)
    monkeypatch.setattr(kda, "kda_attn_paged", on_paged)
    _, status = hybrid_example.run(**kw)
    assert status == 0 and checked[0] == 2 * prompts * (kw["steps"] + 2)
