"""Lengths, tables and pages that are wrong: what is reported, what is left unwritten,
and that the other requests of the call are right."""
import pytest
import torch

import attn_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_attn import BF, DEV, F32, cached, cumulative, ints, packed, randn

pytestmark = pytest.mark.gpu


def sentinels(total, hq, d, io):
    return torch.full((total, hq, d), 7.0, dtype=io, device=DEV), torch.full((total, hq), 7.0, device=DEV)


# cu_seqlens, max_len, the rows left alone, the prompts that are right
PROMPTS = [
    ([0, 30, 60], 50, (30, 50), [(0, 30)]),
    ([-4, 10, 50], 50, (0, 10), [(10, 50)]),
    ([0, 30, 50], 25, (0, 30), [(30, 50)]),
    ([20, 11, 50], 50, (0, 11), [(11, 50)]),
    ([0] + list(range(20, 1000, 7)) + [1400, 1500], 399, (993, 1400), [(0, 20), (20, 27), (986, 993), (1400, 1500)]),
    ([0, 3000, 5000], 2999, (0, 3000), [(3000, 5000)]),
    ([0, 3000, 5001], 3000, (3000, 5000), [(0, 3000)]),
]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
@pytest.mark.parametrize("hq,hkv", [(4, 2), (2, 2)])
def test_wrong_prompt_lengths(case, hq, hkv, io):
    cu, most, alone, right = PROMPTS[case]
    total, d = right[-1][1] if alone[1] <= right[-1][1] else alone[1], 64
    q, k, v = packed([total], hq, hkv, d, io, seed=case)
    need = kda.kda_attn_workspace_size(len(cu) - 1, total, most, hq, hkv, d, io)
    for ws in (torch.empty(0, device=DEV), torch.full((max(need, 4) // 4,), float("nan"), device=DEV)):
        o, lse = sentinels(total, hq, d, io)
        status = ints([0])
        kda.kda_attn_prompt(q, k, v, ints(cu), max_len=most, o=o, lse=lse, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status) == kda.KDA_DEV_LENGTH
        assert (o[alone[0]:alone[1]] == 7).all() and (lse[alone[0]:alone[1]] == 7).all()
        for a, b in right:
            attn_ref.check(o[a:b], lse[a:b], attn_ref.prompt(q[a:b], k[a:b], v[a:b], [b - a], d ** -0.5))


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("wide", [1, 8])
def test_wrong_cache_lengths_are_clamped(io, wide):
    """Below zero: nothing is seen; past the table's row: all of the row is."""
    hq, hkv, d, page, per = 4, 2, 64, 64, 40 * wide
    g = torch.Generator(device=DEV).manual_seed(wide)
    kc, vc = (randn(g, 3 * per, hkv, page, d, io=io) for _ in range(2))
    table = torch.randperm(3 * per, generator=g, device=DEV).to(torch.int32).view(3, per)
    q_lens, kv = [1, 3, 2], [per * page + 1, 700, -1]
    q = randn(g, sum(q_lens), hq, d, io=io)
    ref = attn_ref.paged(q, kc, vc, table, q_lens, [per * page, 700, 0], d ** -0.5)
    for ws in (None, torch.empty(0, device=DEV)):
        status = ints([0])
        o, lse = kda.kda_attn_paged(q, kc, vc, table, cumulative(q_lens), ints(kv), max_q=3, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status) == kda.KDA_DEV_LENGTH
        attn_ref.check(o, lse, ref)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("bad", [-1, 1 << 30, None])
@pytest.mark.parametrize("page", [16, 128, 256])
def test_pages_out_of_range_read_as_zeros(io, bad, page):
    q_lens, kv_lens = [1, 5, 200], [700, 611, 900]
    q, kc, vc, table = cached(q_lens, kv_lens, 8, 2, 128, page, io, seed=page, stale=0.0)
    pages = kc.shape[0]
    zero = torch.zeros_like(kc[:1])
    want = table.clone()
    for r, j in ((0, 0), (1, 2), (2, 1)):
        table[r, j] = pages if bad is None else bad
        want[r, j] = pages  # a page of zeros at the end
    ref = attn_ref.paged(q, torch.cat([kc, zero]), torch.cat([vc, zero]), want, q_lens, kv_lens, 128 ** -0.5)
    for ws in (None, torch.empty(0, device=DEV)):
        status = ints([0])
        o, lse = kda.kda_attn_paged(q, kc, vc, table, cumulative(q_lens), ints(kv_lens), max_q=200, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status) == kda.KDA_DEV_PAGES
        attn_ref.check(o, lse, ref)


@pytest.mark.parametrize("io", [BF, F32])
def test_more_new_tokens_than_announced(io):
    q_lens, kv_lens = [3, 9, 1], [800, 3000, 44]
    q, kc, vc, table = cached(q_lens, kv_lens, 8, 2, 128, 32, io)
    ref = attn_ref.paged(q, kc, vc, table, q_lens, kv_lens, 128 ** -0.5)
    for ws in (None, torch.empty(0, device=DEV)):
        o, lse = sentinels(13, 8, 128, io)
        status = ints([0])
        kda.kda_attn_paged(q, kc, vc, table, cumulative(q_lens), ints(kv_lens), max_q=5, o=o, lse=lse, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status) == kda.KDA_DEV_LENGTH
        assert (o[3:12] == 7).all() and (lse[3:12] == 7).all()
        for s in (slice(0, 3), slice(12, 13)):
            attn_ref.check(o[s], lse[s], tuple(x[s] for x in ref))


@pytest.mark.parametrize("io", [BF, F32])
def test_lengths_near_2_to_31(io):
    """A table of 2^31 slots and a length at its end: clamped to 2^30 and reported, and
    key numbers past the end stay positive. No page of it exists, so every score and
    value is 0."""
    kc, vc = (torch.ones(1, 1, 1024, 64, dtype=io, device=DEV) for _ in range(2))
    table = torch.full((1, 1 << 21), -1, dtype=torch.int32, device=DEV)
    q = torch.ones(1, 1, 64, device=DEV).to(io)
    for kv in ((1 << 31) - 1, (1 << 31) - 128, (1 << 31) - 200):
        status = ints([0])
        o, lse = kda.kda_attn_paged(q, kc, vc, table, ints([0, 1]), ints([kv]), max_q=1, status=status)
        torch.cuda.synchronize()
        assert int(status) == kda.KDA_DEV_LENGTH | kda.KDA_DEV_PAGES
        assert not o.any() and abs(float(lse) - 30 * 0.6931471805599453) <= 1e-4
