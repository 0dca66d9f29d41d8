"""Latent attention over the paged cache against its definition in 64 bits."""
import random

import pytest
import torch

import attn_ref
import latent_ref
import gated_delta_rule_57_gb300 as pkg
from gated_delta_rule_57_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float32]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def case(q_lens, kv_lens, hq, dr, page, io, seed=0, spare=0):
    """Queries, a cache whose unused slots hold NaN, and its block table."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    held = [-(-x // page) for x in kv_lens]
    pages = sum(held) + 2
    ids = list(range(pages))
    rng.shuffle(ids)
    cache = torch.full((pages, page, 512 + dr), float("nan"), dtype=io, device=DEV)
    table, at = [], 0
    for h, kv in zip(held, kv_lens):
        row = ids[at:at + h]
        at += h
        table.append(row + [-1] * (max(held) + spare - h))
        rows = torch.randn(kv, 512 + dr, generator=g, device=DEV).to(io)
        for j, i in enumerate(row):
            part = rows[j * page:(j + 1) * page]
            cache[i, :len(part)] = part
    q = torch.randn(sum(q_lens), hq, 512 + dr, generator=g, device=DEV).to(io)
    cu = [0]
    for x in q_lens:
        cu.append(cu[-1] + x)
    return q, cache, ints(table).view(len(q_lens), -1), ints(cu), ints(kv_lens)


def run(q, cache, table, cu, kv, q_lens, scale=0.07, **kw):
    status = ints([0])
    o, lse = pkg.kda_attn_latent_paged(q, cache, table, cu, kv, scale=scale, max_q=max(q_lens), status=status, **kw)
    torch.cuda.synchronize()
    return o, lse, int(status)


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("q_lens,kv_lens,hq,dr,page", [
    ([1], [1], 1, 64, 16),
    ([1], [63], 32, 64, 16),
    ([1], [64], 32, 0, 64),
    ([1], [65], 16, 64, 32),
    ([1, 1, 1], [700, 5, 129], 8, 64, 16),
    ([2], [130], 32, 64, 64),
    ([3, 1, 4], [70, 200, 4], 5, 64, 128),
    ([1, 1], [300, 17], 64, 0, 16),
    ([1], [200], 128, 64, 64),
    ([2, 1], [100, 90], 40, 64, 32),
    ([1, 2], [33, 50], 67, 64, 16),
    ([65, 7], [300, 64], 3, 64, 1024),
    ([33], [33], 1, 0, 16),
    ([129, 1], [129, 500], 2, 64, 32),
])
def test_against_definition(io, q_lens, kv_lens, hq, dr, page):
    q, cache, table, cu, kv = case(q_lens, kv_lens, hq, dr, page, io)
    o, lse, status = run(q, cache, table, cu, kv, q_lens)
    attn_ref.check(o, lse, latent_ref.paged(q, cache, table, q_lens, kv_lens, 0.07))
    assert status == 0


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("q_lens,kv_lens,hq", [
    ([1], [9000], 32), ([4, 4], [5001, 3003], 32), ([1] * 40, list(range(1, 2001, 50)), 8), ([200, 1, 3], [1999, 3000, 700], 8),
])
def test_long_rows_are_split(io, q_lens, kv_lens, hq):
    q, cache, table, cu, kv = case(q_lens, kv_lens, hq, 64, 64, io, seed=3)
    ref = latent_ref.paged(q, cache, table, q_lens, kv_lens, 0.07)
    o, lse, status = run(q, cache, table, cu, kv, q_lens)
    attn_ref.check(o, lse, ref)
    whole, lw, _ = run(q, cache, table, cu, kv, q_lens, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    attn_ref.check(whole, lw, ref)
    assert status == 0
