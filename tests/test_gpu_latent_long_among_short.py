"""One long request among many short ones is cut into ranges, whatever their number: a workspace
is asked for, and results are right with it and without."""
import pytest
import torch

import attn_ref
import latent_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_latent_paged import DEV, DTYPES, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1216, 5000, 100000])
def test_a_workspace_is_asked_for(n):
    assert kda.kda_attn_latent_workspace_size(n, n, 1, 16) > 0


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("n,at,heads", [(1300, 0, 4), (1300, 700, 4), (1300, 1299, 4), (8500, 8400, 1)])
def test_long_among_short(io, n, at, heads):
    kv_lens = [1 + i * 7 % 40 for i in range(n)]
    kv_lens[at] = 9000
    q, cache, table, cu, kv = case([1] * n, kv_lens, heads, 64, 64, io, seed=at)
    ref = latent_ref.paged(q, cache, table, [1] * n, kv_lens, 0.07)
    need = kda.kda_attn_latent_workspace_size(n, n, 1, heads, 512, 64, io)
    for ws in (torch.full((need // 4,), float("nan"), device=DEV), torch.empty(0, device=DEV), None):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        o, lse = kda.kda_attn_latent_paged(q, cache, table, cu, kv, scale=0.07, max_q=1, workspace=ws, status=status)
        torch.cuda.synchronize()
        attn_ref.check(o, lse, ref)
        assert int(status) == 0
