"""Values that are not finite in the attention operators: a NaN or Inf in q, k or v
reaches the rows that see it, and no others."""
import pytest
import torch

import attn_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_attn import BF, DEV, F32, cached, cumulative, ints, packed

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def rows_match(o, lse, ref, rows):
    attn_ref.check(o[rows], lse[rows], tuple(x[rows] for x in ref))


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("key,later", [(0, 20), (0, 1), (3, 20), (0, 299)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64)])
def test_nan_scores_beside_a_bad_later_value(io, bad, key, later, hq, hkv, d):
    """A NaN key that rows see is not lost where a later value is taken out of the
    same rows: o and lse are NaN from that key on."""
    lens = [300, 40]
    q, k, v = (x.contiguous() for x in packed(lens, hq, hkv, d, io, seed=later))
    ref = attn_ref.prompt(q, k, v, lens, d ** -0.5)
    k[key], v[later] = NAN, bad
    status = ints([0])
    o, lse = kda.kda_attn_prompt(q, k, v, cumulative(lens), status=status)
    torch.cuda.synchronize()
    hit = torch.zeros(340, dtype=torch.bool, device=DEV)
    hit[key:300] = True
    rows_match(o, lse, ref, ~hit)
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert int(status) == kda.KDA_DEV_NONFINITE


@pytest.mark.parametrize("io", [BF, F32])
def test_nan_query_beside_a_bad_later_value(io):
    lens = [300, 40]
    q, k, v = (x.contiguous() for x in packed(lens, 8, 2, 128, io, seed=1))
    ref = attn_ref.prompt(q, k, v, lens, 128 ** -0.5)
    q[5], v[310] = NAN, NAN  # the bad value is the other prompt's
    q[305] = NAN
    status = ints([0])
    o, lse = kda.kda_attn_prompt(q, k, v, cumulative(lens), status=status)
    torch.cuda.synchronize()
    hit = torch.zeros(340, dtype=torch.bool, device=DEV)
    hit[[5, 305]] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    hit[310:] = True  # these see it
    assert torch.isnan(o[310:]).all()
    rows_match(o, lse, ref, ~hit)
    assert int(status) == kda.KDA_DEV_NONFINITE


def far_apart(n, hq, hkv, d, io, low):
    """Keys whose scores are 128, those of `low` -128: e^-256 of the others' weight, zero in
    32 bits but not by the definition."""
    q = torch.full((n, hq, d), 4.0, device=DEV).to(io)
    k = torch.full((n, hkv, d), 32.0 / d, device=DEV).to(io)
    k[low] = -32.0 / d
    return q, k, torch.randn(n, hkv, d, generator=torch.Generator(device=DEV).manual_seed(n), device=DEV).to(io)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("n,low,at", [(60, slice(5, 6), 5), (60, slice(0, 1), 0), (250, slice(0, 128), 70), (250, slice(128, 250), 130),
                                      (900, slice(0, 512), 500)])
def test_a_bad_value_of_no_weight_reaches_its_rows(io, bad, n, low, at):
    """The weight of a seen key is positive, however small: what its value holds
    stays, in a prompt and for single tokens over a cache."""
    hq, hkv, d, page = 4, 2, 64, 64
    q, k, v = far_apart(n, hq, hkv, d, io, low)
    v[at, 1, 3] = bad
    hit = torch.zeros(n, hq, d, dtype=torch.bool, device=DEV)
    hit[at:, 2:, 3] = True
    status = ints([0])
    o, _ = kda.kda_attn_prompt(q, k, v, ints([0, n]), scale=1.0, status=status)
    torch.cuda.synchronize()
    assert torch.equal(~torch.isfinite(o), hit) and int(status) == kda.KDA_DEV_NONFINITE
    per = -(-n // page)
    kc, vc = (torch.zeros(per, hkv, page, d, dtype=io, device=DEV) for _ in range(2))
    kda.kda_kv_append(k, v, torch.arange(n, dtype=torch.int32, device=DEV), kc, vc)
    table = torch.arange(64, dtype=torch.int32, device=DEV)[None].contiguous()  # wide: cut into ranges
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        status.zero_()
        o, _ = kda.kda_attn_paged(q[-1:], kc, vc, table, ints([0, 1]), ints([n]), scale=1.0, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert torch.equal(~torch.isfinite(o), hit[-1:]) and int(status) == kda.KDA_DEV_NONFINITE


def visible(q_lens, kv_lens, at):
    """Per packed token, whether it sees key at[r] of its request r (None: no such key)."""
    out = []
    for n, kv, j in zip(q_lens, kv_lens, at):
        out += [j is not None and j <= kv - n + i for i in range(n)]
    return torch.tensor(out, device=DEV)


LATE = [  # q_lens, kv_lens, hq, hkv, d, page, bad keys (from the end)
    ([4, 70, 1], [4100, 4500, 300], 8, 2, 128, 64, [1, 1, None]),
    ([4, 70], [4223, 4096], 8, 2, 128, 16, [3, 33]),
    ([2, 31], [5000, 2600], 32, 2, 64, 128, [1, 30]),
    ([130, 3], [3000, 4097], 4, 1, 64, 1024, [127, 2]),
    ([255, 8], [2304, 4224], 2, 2, 128, 32, [254, 1]),
    ([300, 1, 513], [300, 2100, 2561], 1, 1, 128, 16, [299, None, 200]),
    ([5, 200], [2, 130], 8, 2, 128, 16, [1, 40]),
]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("one_channel", [False, True])
@pytest.mark.parametrize("case", range(len(LATE)))
def test_bad_late_values_over_a_cache(case, one_channel, bad, io):
    """A bad value among the new tokens of a request, in requests cut into ranges and
    whole, single row tiles and pairs: rows before it are as if it were not there."""
    q_lens, kv_lens, hq, hkv, d, page, back = LATE[case]
    q, kc, vc, table = cached(q_lens, kv_lens, hq, hkv, d, page, io, seed=case)
    ref = attn_ref.paged(q, kc, vc, table, q_lens, kv_lens, d ** -0.5)
    at = [None if b is None else kv - b for b, kv in zip(back, kv_lens)]
    head, chan = hkv - 1, slice(7, 8) if one_channel else slice(0, d)
    for r, j in enumerate(at):
        if j is not None:
            vc[table[r, j // page].long(), head, j % page, chan] = bad
    hit = torch.zeros(q.shape, dtype=torch.bool, device=DEV)
    hit[:, head * (hq // hkv):, chan] = visible(q_lens, kv_lens, at)[:, None, None]
    wide = torch.full((len(q_lens), 6144 // page), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    most = max(q_lens)
    need = kda.kda_attn_workspace_size(len(q_lens), sum(q_lens), most, hq, hkv, d, io)
    assert need > 0
    for ws in (torch.full((need // 4,), NAN, device=DEV), torch.empty(0, device=DEV)):
        status = ints([0])
        o, lse = kda.kda_attn_paged(q, kc, vc, wide, cumulative(q_lens), ints(kv_lens), max_q=most, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert torch.equal(~torch.isfinite(o), hit)
        attn_ref.check(torch.where(hit, ref[0].to(io), o), lse, ref)
        assert int(status) == kda.KDA_DEV_NONFINITE


def test_infinite_values_keep_their_signs():
    """Two Inf of one sign stay Inf, two of different signs are NaN, a row between them
    has the first."""
    q, k, v = (x.contiguous() for x in packed([60], 4, 2, 64, BF))
    v[20, 1, 3], v[40, 1, 3] = INF, -INF
    v[20, 0, 9], v[40, 0, 9] = -INF, -INF
    o, _ = kda.kda_attn_prompt(q, k, v, ints([0, 60]))
    torch.cuda.synchronize()
    assert (o[20:40, 2:, 3] == INF).all() and torch.isnan(o[40:, 2:, 3]).all()
    assert (o[20:, :2, 9] == -INF).all()
    o[20:, 2:, 3], o[20:, :2, 9] = 0, 0
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("lens,hq,hkv,at", [([5000], 4, 1, [4999]), ([5000], 4, 1, [4993, 4970]), ([3000, 2900, 17], 2, 1, [2999, 5899, 5916]),
                                            ([2500, 1, 2600], 6, 2, [2300, 2500, 5100])])
def test_bad_late_values_in_prompts_cut_into_ranges(lens, hq, hkv, at):
    d, total = 128, sum(lens)
    q, k, v = (x.contiguous() for x in packed(lens, hq, hkv, d, BF, seed=total))
    ref = attn_ref.prompt(q, k, v, lens, d ** -0.5)
    v[at], k[at] = NAN, NAN
    hit = torch.zeros(total, dtype=torch.bool, device=DEV)
    end = torch.tensor(lens, device=DEV).cumsum(0)
    for j in at:
        hit[j:int(end[end > j][0])] = True
    need = kda.kda_attn_workspace_size(len(lens), total, max(lens), hq, hkv, d)
    for ws in (torch.full((need // 4,), NAN, device=DEV), torch.empty(0, device=DEV)):
        status = ints([0])
        o, lse = kda.kda_attn_prompt(q, k, v, cumulative(lens), max_len=max(lens), workspace=ws, status=status)
        torch.cuda.synchronize()
        rows_match(o, lse, ref, ~hit)
        assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all() and int(status) == kda.KDA_DEV_NONFINITE


@pytest.mark.parametrize("split", [True, False])
def test_bad_late_value_over_a_very_long_context(split):
    """300 thousand keys, 64 new tokens, a NaN in the last one: no wait runs out and
    every row before it is written (pages are shared to keep the cache small)."""
    hq, hkv, d, page, n, kv = 4, 1, 128, 1024, 64, 300 * 1024
    g = torch.Generator(device=DEV).manual_seed(0)
    kc, vc = (torch.randn(9, hkv, page, d, generator=g, device=DEV).to(BF) for _ in range(2))
    table = torch.randint(0, 8, (1, kv // page), generator=g, device=DEV).to(torch.int32)
    table[0, -1] = 8
    q = torch.randn(n, hq, d, generator=g, device=DEV).to(BF)
    ref = attn_ref.paged(q, kc, vc, table, [n], [kv], d ** -0.5)
    vc[8, 0, page - 1] = NAN
    status = ints([0])
    ws = None if split else torch.empty(0, device=DEV)
    o, lse = kda.kda_attn_paged(q, kc, vc, table, ints([0, n]), ints([kv]), max_q=n, workspace=ws, status=status)
    torch.cuda.synchronize()
    assert int(status) == kda.KDA_DEV_NONFINITE
    assert torch.isnan(o[-1]).all()
    attn_ref.check(o[:-1], lse, (ref[0][:-1], ref[1], ref[2][:-1]))
