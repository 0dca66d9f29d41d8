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
