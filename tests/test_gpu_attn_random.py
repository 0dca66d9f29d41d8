"""Drawn attention calls against the 64-bit definition: types, groups, lengths, pages,
table widths, with and without a workspace, some with values that are not finite."""
import math
import random

import pytest
import torch

import attn_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_attn import BF, DEV, F32, cached, cumulative, ints, packed

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
GROUPS = [1, 2, 3, 4, 5, 6, 7, 8, 9, 16, 20, 33, 64]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case small enough for the definition: (paged, q_lens, kv_lens, hq, hkv, d, page, io)."""
    while True:
        io, d, hkv = rng.choice([BF, BF, BF, F32]), rng.choice([64, 128]), rng.choice([1, 2, 3, 5, 8])
        hq, n, paged = hkv * rng.choice(GROUPS), rng.choice([1, 2, 3, rng.randint(1, 40)]), rng.random() < 0.6
        page = rng.choice([16, 32, 64, 128, 256, 1024])
        longest = rng.choice([40, 300, 3000, 9000] if paged else [5, 100, 700, 2500])
        kv = [max(0, log_int(rng, 1, longest) - rng.choice([0, 0, 1])) for _ in range(n)]
        q = [rng.choice([1, 1, 0, rng.randint(0, 12), log_int(rng, 1, 400)]) for _ in range(n)] if paged else kv
        if rng.random() < 0.9:
            q = [min(a, b) for a, b in zip(q, kv)]
        if hq <= 128 and 0 < sum(q) and sum(a * b for a, b in zip(q, kv)) * hq <= 2e8 and sum(kv) * hkv * d <= 1e8:
            return paged, q, kv, hq, hkv, d, page, io


@pytest.mark.parametrize("seed", range(120))
def test_drawn_calls(seed):
    rng = random.Random(seed)
    paged, q_lens, kv_lens, hq, hkv, d, page, io = draw(rng)
    scale, n, total = d ** -0.5, len(q_lens), sum(q_lens)
    most = rng.choice([max(q_lens), max(q_lens), None, max(q_lens) + rng.randint(0, 300)])
    if paged:
        q, kc, vc, table = cached(q_lens, kv_lens, hq, hkv, d, page, io, seed=seed)
        width = rng.choice([3000, 20000, 0]) // page
        if width > table.shape[1]:
            wide = torch.full((n, width), -1, dtype=torch.int32, device=DEV)
            wide[:, :table.shape[1]] = table
            table = wide
        ref = attn_ref.paged(q, kc, vc, table, q_lens, kv_lens, scale)
    else:
        most = rng.choice([max(q_lens), None])
        q, k, v = (x.contiguous() for x in packed(q_lens, hq, hkv, d, io, seed=seed))
        ref = attn_ref.prompt(q, k, v, q_lens, scale)
    hit = torch.zeros(q.shape, dtype=torch.bool, device=DEV)
    bad = 0 if rng.random() < 0.5 else rng.randint(1, 6)
    starts = cumulative(q_lens).tolist()
    for _ in range(bad):  # mostly near a request's end, where some tokens do not see it
        r = rng.randrange(n)
        if kv_lens[r] == 0:
            continue
        j = kv_lens[r] - 1 - rng.randint(0, min(kv_lens[r], max(q_lens[r], 1) + 2) - 1)
        h, c, x = rng.randrange(hkv), rng.randrange(d), rng.choice([NAN, NAN, INF, -INF])
        if paged:
            vc[table[r, j // page].long(), h, j % page, c] = x
        else:
            v[starts[r] + j, h, c] = x
        first = starts[r] + max(0, j - (kv_lens[r] - q_lens[r]))
        hit[first:starts[r + 1], h * (hq // hkv):(h + 1) * (hq // hkv), c] = True
    need = kda.kda_attn_workspace_size(n, total, total if most is None else most, hq, hkv, d, io)
    ws, status = rng.choice([None, torch.full((max(need, 4) // 4,), NAN, device=DEV), torch.empty(0, device=DEV)]), ints([0])
    if paged:
        o, lse = kda.kda_attn_paged(q, kc, vc, table, cumulative(q_lens), ints(kv_lens), max_q=most, workspace=ws, status=status)
    else:
        o, lse = kda.kda_attn_prompt(q, k, v, cumulative(q_lens), max_len=most, workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status) == (kda.KDA_DEV_NONFINITE if hit.any() else 0)
    assert torch.equal(~torch.isfinite(o), hit)
    attn_ref.check(torch.where(hit, ref[0].to(io), o), lse, ref)
