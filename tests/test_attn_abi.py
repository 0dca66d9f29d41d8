"""Refusals of the paged-cache and attention entry points: every argument set
here is invalid (or empty), so nothing is launched and no GPU is needed."""
import ctypes

import pytest
import torch

from gated_delta_rule_57_gb300 import kda

BAD, UNS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK
A = [0x100000 * (i + 1) for i in range(12)]  # never dereferenced


@pytest.fixture(scope="module")
def L():
    return kda.lib()


def plan(L, **kw):
    a = dict(old=A[0], new=A[1], table=A[2], ring=A[3], ring_in=A[4], ring_out=A[5], kv=A[6], cu=A[7], slot=A[8],
             N=4, max_pages=8, num_pages=64, page=16, room=32, status=None)
    a.update(kw)
    return L.kda_kv_plan(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(max_pages=-1), BAD), (dict(num_pages=0), BAD), (dict(page=0), BAD), (dict(room=-1), BAD),
    (dict(num_pages=1 << 20, page=1 << 11), BAD), (dict(room=(1 << 30) + 1), BAD), (dict(N=16385), UNS),
    (dict(old=None), BAD), (dict(table=None), BAD), (dict(ring_in=None), BAD), (dict(cu=None), BAD), (dict(slot=None), BAD),
    (dict(new=A[1] + 2), BAD), (dict(status=A[9] + 1), BAD),
    (dict(kv=A[0]), BAD), (dict(ring_out=A[4]), BAD), (dict(slot=A[3] + 64), BAD), (dict(table=A[7]), BAD),
])
def test_plan_refuses(L, kw, code):
    assert plan(L, **kw) == code
    assert L.kda_last_error_string()


def append(L, **kw):
    a = dict(k=A[0], v=A[1], slot=A[2], kc=A[3], vc=A[4], T=4, Hkv=2, d=64, ks=128, vs=128, pages=16, page=16,
             io=kda.KDA_BF16, status=None)
    a.update(kw)
    return L.kda_kv_append(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(Hkv=-1), BAD), (dict(pages=-1), BAD), (dict(page=0), BAD), (dict(io=2), BAD),
    (dict(d=96, ks=192, vs=192), UNS), (dict(ks=127), BAD), (dict(vs=132), BAD), (dict(ks=-128), BAD),
    (dict(k=None), BAD), (dict(slot=None), BAD), (dict(vc=None), BAD), (dict(k=A[0] + 8), BAD), (dict(kc=A[3] + 4), BAD),
    (dict(slot=A[2] + 2), BAD), (dict(kc=A[0]), BAD), (dict(vc=A[3] + 1024), BAD), (dict(pages=1 << 20, page=1 << 11), BAD),
    (dict(T=0, k=None), OK), (dict(Hkv=0, k=None), OK),
])
def test_append_refuses(L, kw, code):
    assert append(L, **kw) == code


def prompt(L, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], cu=A[3], o=A[4], lse=A[5], N=2, total=16, most=16, Hq=4, Hkv=2, d=64, qs=256, ks=128,
             vs=128, scale=0.125, io=kda.KDA_BF16, ws=None, ws_bytes=0, status=None)
    a.update(kw)
    return L.kda_attn_prompt(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(total=-1), BAD), (dict(most=-1), BAD), (dict(io=7), BAD), (dict(d=80), UNS),
    (dict(Hq=5), BAD), (dict(Hq=130), UNS), (dict(Hkv=0), BAD), (dict(Hkv=-2), BAD), (dict(qs=255), BAD), (dict(ks=64), BAD),
    (dict(vs=130), BAD), (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD), (dict(q=None), BAD), (dict(k=None), BAD), (dict(cu=None), BAD), (dict(o=None), BAD),
    (dict(q=A[0] + 8), BAD), (dict(o=A[4] + 2), BAD), (dict(cu=A[3] + 1), BAD), (dict(lse=A[5] + 2), BAD), (dict(o=A[0]), BAD),
    (dict(lse=A[1]), BAD), (dict(lse=A[4] + 256), BAD), (dict(ws=A[4], ws_bytes=64), BAD), (dict(ws=A[6] + 4, ws_bytes=64), BAD),
    (dict(N=0, q=None), OK), (dict(total=0, k=None), OK), (dict(most=0), OK), (dict(Hq=0, Hkv=0), OK),
])
def test_prompt_refuses(L, kw, code):
    assert prompt(L, **kw) == code


def paged(L, **kw):
    a = dict(q=A[0], kc=A[1], vc=A[2], table=A[3], cu=A[4], kv=A[5], o=A[6], lse=None, N=2, total=2, most=1, Hq=4, Hkv=2,
             d=64, qs=256, pages=16, page=16, max_pages=8, scale=0.125, io=kda.KDA_BF16, ws=None, ws_bytes=0, status=None)
    a.update(kw)
    return L.kda_attn_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(total=-1), BAD), (dict(most=-1), BAD), (dict(pages=-1), BAD), (dict(max_pages=-1), BAD),
    (dict(page=8), UNS), (dict(page=48), UNS), (dict(page=2048), UNS), (dict(page=0), BAD), (dict(d=32), UNS), (dict(Hq=3), BAD),
    (dict(pages=1 << 21, page=1 << 10), BAD), (dict(scale=0.0), BAD), (dict(q=None), BAD), (dict(kc=None), BAD),
    (dict(table=None), BAD), (dict(kv=None), BAD), (dict(cu=None), BAD), (dict(vc=A[2] + 8), BAD), (dict(kv=A[5] + 2), BAD),
    (dict(o=A[1]), BAD), (dict(lse=A[3]), BAD), (dict(qs=252), BAD), (dict(N=0), OK), (dict(total=0), OK), (dict(most=0), OK),
])
def test_paged_refuses(L, kw, code):
    assert paged(L, **kw) == code


def test_workspace_size_refuses(L):
    bad = ctypes.c_size_t(-1).value
    f = L.kda_attn_workspace_size
    assert f(-1, 1, 1, 4, 2, 64, kda.KDA_BF16) == bad
    assert f(1, 1, 1, 4, 2, 96, kda.KDA_BF16) == bad
    assert f(1, 1, 1, 5, 2, 64, kda.KDA_BF16) == bad
    assert f(1, 1, 1, 4, 2, 64, 9) == bad
    assert f(0, 0, 0, 4, 2, 64, kda.KDA_BF16) == 0


def test_binding_refuses():
    i = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a GPU
        kda.kda_attn_prompt(x, x[:, :2], x[:, :2], i)
    with pytest.raises(TypeError):
        kda.kda_attn_prompt(x.half(), x.half(), x.half(), i)
    with pytest.raises(ValueError):
        kda.kda_attn_prompt(x, x[:3], x[:3], i)
    with pytest.raises(ValueError):
        kda.kda_attn_paged(x, torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64), i[None], i, i)
    with pytest.raises(ValueError):
        kda.kda_kv_append(x, x[:2], i, x[None], x[None])
    with pytest.raises(ValueError):
        kda.kda_kv_plan(i.long(), i, i[:, None], i, i[:2], page_size=16, max_tokens=4)


def test_short_keys_matches_header():
    import re
    from gated_delta_rule_57_gb300 import build
    text = open(build.INCLUDE + "/kda.h").read()
    assert kda.KDA_ATTN_SHORT_KEYS == int(re.search(r"#define KDA_ATTN_SHORT_KEYS (\d+)", text).group(1))
