"""Latent attention over cached rows that hold Inf: a score of -Inf has weight 0, and 0 x Inf
leaves NaN in the channel of that Inf, for every row that sees it and has other scores; a row
of no other scores counts as one that sees no key. The same whole and in ranges."""
import math

import pytest
import torch

import attn_ref
import latent_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_latent_paged import DEV, DTYPES, ints

pytestmark = pytest.mark.gpu
INF = float("inf")
SCALE, CHANNEL = 0.07, 7


def call(q, cache, kv, ws):
    n, page = q.shape[0], cache.shape[1]
    table = torch.arange(cache.shape[0], dtype=torch.int32, device=DEV)[None]
    need = kda.kda_attn_latent_workspace_size(1, n, n, q.shape[1], 512, q.shape[2] - 512, q.dtype)
    assert kv <= table.shape[1] * page and need > 0
    space = torch.full((need // 4,), float("nan"), device=DEV) if ws else torch.empty(0, device=DEV)
    status = ints([0])
    o, lse = kda.kda_attn_latent_paged(q, cache, table, ints([0, n]), ints([kv]), scale=SCALE, max_q=n, workspace=space, status=status)
    torch.cuda.synchronize()
    return o, lse, int(status)


def inputs(n, heads, kv, dr, io, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    cache = torch.randn(-(-kv // 64), 64, 512 + dr, generator=g, device=DEV).to(io)
    q = torch.randn(n, heads, 512 + dr, generator=g, device=DEV).to(io)
    q[..., CHANNEL] = -1  # +Inf there: a score of -Inf
    return q, cache, cache.view(-1, 512 + dr)


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("kv,heads,dr", [(1500, 4, 64), (1500, 40, 0), (9000, 4, 64), (9000, 64, 0)])  # few parts, and many
def test_a_part_of_vanishing_weight_keeps_its_nan(io, ws, kv, heads, dr):
    """One key has all the weight: every other's is below 2^-300, so that o is its row to the
    last bit, but for the channel in which a key far away from it holds Inf."""
    q, cache, rows = inputs(1, 1, kv, dr, io, kv)
    q = q.expand(1, heads, 512 + dr).contiguous()
    rows[10] = 8 * q[0, 0]
    rows[kv - 200, CHANNEL] = INF
    score = SCALE * float((q[0, 0].double() * rows[10].double()).sum())
    others = SCALE * (rows.double() @ q[0, 0].double())
    others[10] = -INF
    assert (score - float(others[:kv].max())) / math.log(2) > 300
    o, lse, status = call(q, cache, kv, ws)
    assert torch.isnan(o[..., CHANNEL]).all() and status == kda.KDA_DEV_NONFINITE
    keep = torch.arange(512, device=DEV) != CHANNEL
    assert torch.equal(o[..., keep], rows[10, :512][keep].expand(1, heads, 511))
    # an fp32 sum of 576 products, most at the last one's size: 576 half units at worst
    assert ((lse.double() - score).abs() <= 576 * 2.0 ** -24 * score).all()


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("kv,lo,hi", [(1500, 400, 1000), (9000, 1000, 5000), (1500, 0, 700), (1500, 700, 1500)])
def test_a_stretch_of_minus_infinity_leaves_nan_in_its_channel(io, ws, kv, lo, hi):
    """Ranges all of whose scores are -Inf. The other keys have one value a channel, so that
    any weighting of them gives it: o is that value, off by the sum's rounding and its own."""
    q, cache, rows = inputs(1, 8, kv, 64, io, hi)
    rows[:, :512] = rows[0, :512].clone()
    rows[lo:hi, CHANNEL] = INF
    o, lse, status = call(q, cache, kv, ws)
    assert torch.isnan(o[..., CHANNEL]).all() and status == kda.KDA_DEV_NONFINITE
    keep = torch.arange(512, device=DEV) != CHANNEL
    want = rows[0, :512].double()[keep].expand(1, 8, 511)
    # two fp32 sums of up to 9000 terms, each term a unit off at worst; bf16: the weights and o rounded once each
    off = 2 * 9000 * 2.0 ** -23 + (2 * 2.0 ** -8 if io == torch.bfloat16 else 0)
    assert ((o[..., keep].double() - want).abs() <= off * want.abs()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("n,kv,heads", [(1, 3, 4), (2, 2, 1), (3, 40, 8), (4, 900, 8), (2, 4, 64), (64, 900, 1), (4, 9000, 5)])
def test_tokens_of_no_other_scores_see_nothing(io, ws, n, kv, heads):
    """Every key of theirs scores -Inf, those that only the later ones see too."""
    q, cache, rows = inputs(n, heads, kv, 64, io, n)
    rows[:kv, CHANNEL] = INF
    o, lse, status = call(q, cache, kv, ws)
    assert not o.any() and (lse == -INF).all() and status == 0


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("kv", [5, 900, 9000])
def test_infinity_among_the_last_keys_reaches_the_tokens_from_it_on(io, ws, kv):
    """Four tokens; the last key but one holds Inf, with a score of -Inf for all heads but one."""
    q, cache, rows = inputs(4, 6, kv, 64, io, kv)
    table = torch.arange(cache.shape[0], dtype=torch.int32, device=DEV)[None]
    ref = latent_ref.paged(q, cache, table, [4], [kv], SCALE)
    rows[kv - 2, CHANNEL] = INF
    q2 = q.clone()
    q2[:, 3, CHANNEL] = 1
    o, lse, status = call(q2, cache, kv, ws)
    heads = [0, 1, 2, 4, 5]
    attn_ref.check(o[:2, heads], lse[:2, heads], tuple(x[:2, heads] for x in ref))
    assert torch.isfinite(o[:2]).all()
    assert torch.isnan(o[2:, 3]).all() and not torch.isfinite(o[2:, heads, CHANNEL]).any()
    keep = torch.arange(512, device=DEV) != CHANNEL
    assert torch.isfinite(o[2:, heads][..., keep]).all() and torch.isfinite(lse[2:, heads]).all()
    assert status == kda.KDA_DEV_NONFINITE


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("ws", [False, True])
def test_a_token_whose_only_other_key_is_its_own(io, ws):
    """Two tokens over two keys: key 0 scores -Inf, so token 0 sees nothing; token 1 sees its own."""
    q, cache, rows = inputs(2, 4, 2, 64, io, 5)
    rows[0, CHANNEL] = INF
    o, lse, status = call(q, cache, 2, ws)
    assert not o[0].any() and (lse[0] == -INF).all() and status == kda.KDA_DEV_NONFINITE
    keep = torch.arange(512, device=DEV) != CHANNEL
    assert torch.isnan(o[1, :, CHANNEL]).all() and torch.equal(o[1][:, keep], rows[1, :512][keep].expand(4, 511))
