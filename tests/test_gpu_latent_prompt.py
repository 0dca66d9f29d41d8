"""Latent attention over packed prompts (expanded heads) against its definition in 64 bits."""
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


def case(lens, h, dr, io, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = sum(lens)
    q = torch.randn(t, h, 128 + dr, generator=g, device=DEV).mul(1.5).to(io)
    kv = torch.randn(t, h, 256, generator=g, device=DEV).to(io)
    k_r = torch.randn(t, dr, generator=g, device=DEV).to(io) if dr else None
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return q, kv[..., :128], k_r, kv[..., 128:], ints(cu)


def run(q, k, k_r, v, cu, lens, **kw):
    status = ints([0])
    o, lse = pkg.kda_attn_latent_prompt(q, k, k_r, v, cu, max_len=max(lens), status=status, **kw)
    torch.cuda.synchronize()
    return o, lse, int(status)


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("lens,h,dr", [
    ([1], 1, 64), ([1, 0, 2], 3, 64), ([64], 2, 64), ([65, 63], 2, 0), ([127, 128, 129], 4, 64), ([255, 3, 200, 17], 4, 64),
    ([256, 257], 5, 64), ([511, 1, 513], 3, 64), ([700, 0, 40], 2, 0), ([1021], 8, 64), ([385, 384, 383], 1, 64),
])
def test_against_definition(io, lens, h, dr):
    q, k, k_r, v, cu = case(lens, h, dr, io)
    o, lse, status = run(q, k, k_r, v, cu, lens)
    attn_ref.check(o, lse, latent_ref.prompt(q, k, k_r, v, lens, (128 + dr) ** -0.5))
    assert status == 0


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("lens,h", [([2500], 1), ([3000, 100], 2), ([2049, 2051], 8)])
def test_long_prompts_with_and_without_workspace(io, lens, h):
    q, k, k_r, v, cu = case(lens, h, 64, io, seed=5)
    ref = latent_ref.prompt(q, k, k_r, v, lens, 192 ** -0.5)
    o, lse, status = run(q, k, k_r, v, cu, lens)
    attn_ref.check(o, lse, ref)
    whole, lw, _ = run(q, k, k_r, v, cu, lens, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    attn_ref.check(whole, lw, ref)
    assert status == 0


@pytest.mark.parametrize("io", DTYPES)
def test_orders_and_strides(io):
    """Heads inside tokens, tokens inside heads, and padded rows give the same bits."""
    lens, h = [200, 61], 3
    q, k, k_r, v, cu = case(lens, h, 64, io, seed=7)
    o, lse, _ = run(*(x.contiguous() for x in (q, k, k_r, v)), cu, lens)

    def head_major(x):
        return x.transpose(0, 1).contiguous().transpose(0, 1)

    def padded(x):
        y = torch.full((*x.shape[:-1], x.shape[-1] + 24), float("nan"), dtype=io, device=DEV)
        y[..., 8:-16] = x
        return y[..., 8:-16]

    for f in (head_major, padded):
        o2, lse2, _ = run(f(q), f(k), padded(k_r), f(v), cu, lens)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
