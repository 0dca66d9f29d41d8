"""One token's views of buffers with tokens inside heads: the token stride has no meaning, and
any head stride that is right for more tokens is right for it. Without a GPU: each call here has
another fault, which the library finds after it has looked at the strides."""
import pytest
import torch

from gated_delta_rule_57_gb300 import kda, latent

H, HEAD = 64, (1 << 24) + 64  # H heads of this stride: past 2^30 elements


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def token(d, n=1):
    """[n, H, d], n tokens inside heads (memory that is never touched)."""
    return torch.empty(H * HEAD, dtype=torch.bfloat16).as_strided((n, H, d), (d, HEAD, 1))


@pytest.fixture(autouse=True)
def host(monkeypatch):
    monkeypatch.setattr(latent, "_device", lambda t: t.get_device())
    monkeypatch.setattr(kda, "_stream", lambda s: 0)


@pytest.mark.parametrize("n", [1, 2])
def test_paged(n):
    cache, kw = torch.zeros(9, 16, 576, dtype=torch.bfloat16), dict(want_lse=False, workspace=torch.empty(0))
    with pytest.raises(kda.KdaError, match="scale"):
        kda.kda_attn_latent_paged(token(576, n), cache, i32(1, 9), i32(2), i32(1), scale=-1.0, **kw)


@pytest.mark.parametrize("n", [1, 2])
def test_prompt(n):
    q, kv = token(192, n), token(256, n)
    with pytest.raises(kda.KdaError, match="scale"):
        kda.kda_attn_latent_prompt(q, kv[..., :128], torch.zeros(n, 64, dtype=torch.bfloat16), kv[..., 128:], i32(2), scale=-1.0, want_lse=False,
                                   workspace=torch.empty(0))


@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("inside", [True, False])
def test_append(n, inside):
    cache = torch.zeros(1, 16, 576, dtype=torch.bfloat16)
    q = token(64, n)
    with pytest.raises(kda.KdaError, match="the cache, q_out or k_out overlaps an input"):
        kda.kda_latent_append(cache[0, :n, :512], torch.zeros(n, 64, dtype=torch.bfloat16), i32(n), cache, positions=i32(n),
                              turns=torch.zeros(32, dtype=torch.int64), q_r=q, q_out=q if inside else None)
