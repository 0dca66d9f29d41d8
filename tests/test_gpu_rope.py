"""Rotated appends against the rotation in 64 bits; what is copied, exactly."""
import pytest
import torch

import latent_ref
import gated_delta_rule_57_gb300 as pkg
from gated_delta_rule_57_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float32]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def slots_of(t, pages, page, gen):
    slot = torch.randperm(pages * page, generator=gen, device=DEV)[:t].to(torch.int32)
    slot[::3] = -1
    if t > 4:
        slot[4] = pages * page  # past the cache
    return slot, [(i, s // page, s % page) for i, s in enumerate(slot.tolist()) if 0 <= s < pages * page]


def positions_of(t, gen):
    """Near, far, at the ends of the type, negative."""
    pos = torch.randint(0, 1 << 20, (t,), generator=gen, device=DEV).to(torch.int32)
    pos[:5] = ints([2 ** 31 - 1, 0, -7, -2 ** 31, 1])[:t]
    return pos


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("t,hq,hkv,d,rot,page", [
    (1, 1, 1, 64, 64, 16), (7, 4, 2, 128, 128, 16), (300, 32, 8, 128, 128, 64), (65, 5, 5, 64, 48, 7), (1000, 3, 1, 128, 16, 48),
    (129, 40, 8, 128, 96, 32), (33, 200, 1, 64, 32, 16), (20, 0, 3, 64, 64, 16), (20, 3, 0, 64, 64, 16),
])
def test_kv_append_rope(io, neighbours, t, hq, hkv, d, rot, page):
    g = torch.Generator(device=DEV).manual_seed(t + rot)
    pages = -(-2 * t // page) + 1
    kc, vc = (torch.randn(pages, hkv, page, d, generator=g, device=DEV).to(io) for _ in range(2))
    qkv = torch.randn(t, hq + 2 * hkv, d, generator=g, device=DEV).to(io)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    pos, freq = positions_of(t, g), latent_ref.frequencies(rot)
    slot, live = slots_of(t, pages, page, g)
    turns, status = pkg.kda_rope_turns(freq, device=DEV), ints([0])
    (rk, sk), rv = latent_ref.rotate(k, pos, freq, neighbours), vc.clone()
    want, size = kc.double(), torch.zeros(kc.shape, dtype=torch.float64, device=DEV)
    for i, p, r in live:
        want[p, :, r], size[p, :, r], rv[p, :, r] = rk[i], sk[i], v[i]
    ref_q = latent_ref.rotate(q, pos, freq, neighbours)
    again = torch.empty(t, hkv, d, dtype=io, device=DEV)
    out = pkg.kda_kv_append_rope(q, k, v, slot, pos, turns, kc, vc, neighbours=neighbours, k_out=again, status=status)
    torch.cuda.synchronize()
    latent_ref.check_rotated(again, (rk, sk))
    latent_ref.check_rotated(out, ref_q)
    latent_ref.check_rotated(kc, (want, size))
    assert torch.equal(vc, rv)
    assert int(status) == (kda.KDA_DEV_PAGES if t > 4 else 0)
    # in place, in the projection itself
    back = pkg.kda_kv_append_rope(q, k, v, slot, pos, turns, kc, vc, neighbours=neighbours, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert back is q and torch.equal(q, out) and torch.equal(k, again)


def test_append_without_queries():
    x = torch.randn(5, 2, 64, device=DEV)
    kc, vc = (torch.zeros(1, 2, 16, 64, device=DEV) for _ in range(2))
    i = torch.arange(5, dtype=torch.int32, device=DEV)
    assert pkg.kda_kv_append_rope(None, x, x, i, i, pkg.kda_rope_turns(latent_ref.frequencies(64)), kc, vc) is None
    torch.cuda.synchronize()
    latent_ref.check_rotated(kc[0, :, :5].transpose(0, 1), latent_ref.rotate(x, i, latent_ref.frequencies(64), False))
    assert torch.equal(vc[0, :, :5].transpose(0, 1), x) and not kc[0, :, 5:].any()


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("t,hq,dr,page,order", [(1, 1, 64, 16, "token"), (257, 32, 64, 64, "token"), (70, 8, 64, 7, "head"),
                                                (999, 3, 64, 48, "token"), (40, 0, 64, 16, "token"), (100, 0, 0, 32, "token")])
def test_latent_append(io, neighbours, t, hq, dr, page, order):
    g = torch.Generator(device=DEV).manual_seed(t + hq)
    pages = -(-2 * t // page) + 1
    cache = torch.randn(pages, page, 512 + dr, generator=g, device=DEV).to(io)
    down = torch.randn(t, 512 + 64, generator=g, device=DEV).to(io)
    c, k_r = down[:, :512], down[:, 512:] if dr else None
    pos, freq = positions_of(t, g), latent_ref.frequencies(64)
    slot, live = slots_of(t, pages, page, g)
    status = ints([0])
    want, size = cache.double(), torch.zeros(cache.shape, dtype=torch.float64, device=DEV)
    kw = {}
    if dr:
        rk, sk = (x[:, 0] for x in latent_ref.rotate(k_r[:, None], pos, freq, neighbours))
        kw = dict(positions=pos, turns=pkg.kda_rope_turns(freq, device=DEV), k_out=torch.empty(t, 64, dtype=io, device=DEV))
    for i, p, r in live:
        want[p, r, :512] = c[i].double()
        if dr:
            want[p, r, 512:], size[p, r, 512:] = rk[i], sk[i]
    if hq:
        # a projection's last channels; to beside the absorbed queries, heads inside tokens or tokens inside heads
        q_r = torch.randn(t, hq, 192, generator=g, device=DEV).to(io)[..., 128:]
        q = torch.zeros((t, hq, 576) if order == "token" else (hq, t, 576), dtype=io, device=DEV)
        q = q if order == "token" else q.transpose(0, 1)
        kw.update(q_r=q_r, q_out=q[..., 512:])
    out = pkg.kda_latent_append(c, k_r, slot, cache, neighbours=neighbours, status=status, **kw)
    torch.cuda.synchronize()
    latent_ref.check_rotated(cache, (want, size))
    if dr:
        latent_ref.check_rotated(kw["k_out"], (rk, sk))
    if hq:
        latent_ref.check_rotated(out, latent_ref.rotate(q_r, pos, freq, neighbours))
        assert not q[..., :512].any()
        # in place
        pkg.kda_latent_append(c, k_r, slot, cache, positions=pos, turns=kw["turns"], q_r=q_r, q_out=q_r, k_out=k_r, neighbours=neighbours)
        torch.cuda.synchronize()
        assert torch.equal(q_r, out) and torch.equal(k_r, kw["k_out"])
    assert int(status) == (kda.KDA_DEV_PAGES if t > 4 else 0)
