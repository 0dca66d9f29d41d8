"""Values that are not finite in the attention operators: a NaN or Inf in q, k or v
reaches the rows that see it, and no others."""
import pytest
import torch

import attn_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_attn import BF, DEV, F32, cumulative, ints, packed

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
