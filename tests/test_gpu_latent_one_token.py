"""One token's views of buffers with tokens inside heads: as contiguous ones, to the bit."""
import pytest
import torch

from gated_delta_rule_57_gb300 import kda
from test_gpu_latent_paged import DEV, ints

pytestmark = pytest.mark.gpu
H, ROOM = 64, 30000  # H x ROOM x 576: heads 2^30 elements and more from one another in all


def test_one_token_of_a_large_buffer():
    g = torch.Generator(device=DEV).manual_seed(0)
    wide = torch.empty(H, ROOM, 576, dtype=torch.bfloat16, device=DEV)
    wide[:, ROOM - 1] = torch.randn(H, 576, generator=g, device=DEV).bfloat16()
    q = wide.transpose(0, 1)[ROOM - 1:]
    assert q.shape == (1, H, 576) and H * q.stride(1) > 1 << 30
    cache = torch.randn(9, 16, 576, generator=g, device=DEV).bfloat16()
    table, cu, kv = torch.arange(9, dtype=torch.int32, device=DEV)[None], ints([0, 1]), ints([140])

    def paged(x):
        return kda.kda_attn_latent_paged(x, cache, table, cu, kv, scale=0.07)

    def prompt(x):
        k, v = x[..., 192:320], x[..., 320:448]
        return kda.kda_attn_latent_prompt(x[..., :192], k, cache[0, :1, :64].contiguous(), v, cu)

    for f in (paged, prompt):
        for a, b in zip(f(q), f(q.contiguous())):
            assert torch.equal(a, b) and torch.isfinite(a).all()

    c, k_r, pos = cache[0, :1, :512].clone(), cache[0, :1, 512:].clone(), ints([77])
    turns = kda.kda_rope_turns([10000.0 ** (-i / 32) for i in range(32)])
    got = kda.kda_latent_append(c, k_r, ints([0]), cache, positions=pos, turns=turns, q_r=q[..., 512:])
    want = kda.kda_latent_append(c, k_r, ints([0]), cache, positions=pos, turns=turns, q_r=q[..., 512:].contiguous())
    assert torch.equal(got, want)
    rest = q[..., :512].clone()
    kda.kda_latent_append(c, k_r, ints([0]), cache, positions=pos, turns=turns, q_r=q[..., 512:], q_out=q[..., 512:])
    torch.cuda.synchronize()
    assert torch.equal(q[..., 512:], want) and torch.equal(q[..., :512], rest)
