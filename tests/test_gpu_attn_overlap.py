"""Offsets that decrease so that a request starts inside the second one before it: the rows are
the earlier one's, whichever of the two ends first, and the later one is left out."""
import pytest
import torch

import attn_ref
import latent_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_attn import cached, packed
from test_gpu_latent_paged import DEV, DTYPES, case, ints
from test_gpu_latent_prompt import case as latent_prompt

pytestmark = pytest.mark.gpu


def outputs(total, heads, d, io):
    return (torch.full((total, heads, d), 7.0, dtype=io, device=DEV), torch.full((total, heads), 7.0, device=DEV),
            ints([0]))


def check(o, lse, status, ref, right):
    torch.cuda.synchronize()
    assert int(status) == kda.KDA_DEV_LENGTH
    attn_ref.check(o[:right], lse[:right], ref)
    assert (o[right:] == 7).all() and (lse[right:] == 7).all()


def spaces(need):
    return torch.empty(0, device=DEV), torch.full((max(need, 4) // 4,), float("nan"), device=DEV)


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("kv_lens", [[800, 3000, 44], [20, 5, 3000]])
def test_paged(io, kv_lens):
    q, kc, vc, table = cached([3, 9, 3], kv_lens, 8, 2, 128, 32, io)
    for ws in spaces(kda.kda_attn_workspace_size(3, 13, 20, 8, 2, 128, io)):
        o, lse, status = outputs(13, 8, 128, io)
        kda.kda_attn_paged(q[:13], kc, vc, table, ints([0, 3, 2, 13]), ints(kv_lens), max_q=20, o=o, lse=lse, workspace=ws, status=status)
        check(o, lse, status, attn_ref.paged(q[:3], kc, vc, table[:1], [3], kv_lens[:1], 128 ** -0.5), 3)


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("kv_lens", [[800, 3000, 44], [20, 5, 3000]])
def test_latent_paged(io, kv_lens):
    q, cache, table, _, kv = case([3, 9, 3], kv_lens, 8, 64, 32, io)
    for ws in spaces(kda.kda_attn_latent_workspace_size(3, 13, 20, 8, 512, 64, io)):
        o, lse, status = outputs(13, 8, 512, io)
        kda.kda_attn_latent_paged(q[:13], cache, table, ints([0, 3, 2, 13]), kv, scale=0.07, max_q=20, o=o, lse=lse, workspace=ws, status=status)
        check(o, lse, status, latent_ref.paged(q[:3], cache, table[:1], [3], kv_lens[:1], 0.07), 3)


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("cu", [[0, 40, 20, 500], [0, 400, 399, 500], [0, 400, 0, 500]])
def test_prompts(io, cu):
    n = cu[1]
    q, k, v = packed([500], 4, 2, 64, io)
    for ws in spaces(kda.kda_attn_workspace_size(3, 500, 500, 4, 2, 64, io)):
        o, lse, status = outputs(500, 4, 64, io)
        kda.kda_attn_prompt(q, k, v, ints(cu), max_len=500, o=o, lse=lse, workspace=ws, status=status)
        check(o, lse, status, attn_ref.prompt(q[:n], k[:n], v[:n], [n], 0.125), n)
    q, k, k_r, v, _ = latent_prompt([500], 4, 64, io)
    for ws in spaces(kda.kda_attn_workspace_size(3, 500, 500, 4, 4, 128, io)):
        o, lse, status = outputs(500, 4, 128, io)
        kda.kda_attn_latent_prompt(q, k, k_r, v, ints(cu), max_len=500, o=o, lse=lse, workspace=ws, status=status)
        check(o, lse, status, latent_ref.prompt(q[:n], k[:n], k_r[:n], v[:n], [n], 192 ** -0.5), n)
