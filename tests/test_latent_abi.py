"""Refusals of the rotated appends and of latent attention: every argument set here is
invalid (or empty), so nothing is launched and no GPU is needed."""
import ctypes

import pytest

from gated_delta_rule_57_gb300 import kda

BAD, UNS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK
A = [0x1000000 * (i + 1) for i in range(14)]  # never dereferenced


@pytest.fixture(scope="module")
def L():
    return kda.lib()


def rope(L, **kw):
    a = dict(q=A[0], k=A[1], v=A[2], slot=A[3], pos=A[4], turns=A[5], kc=A[6], vc=A[7], out=A[8], ko=A[10], T=4, Hq=4, Hkv=2, d=64, rot=64,
             neighbours=0, qs=256, ks=128, vs=128, os=256, kos=128, pages=16, page=16, io=kda.KDA_BF16, status=None)
    a.update(kw)
    return L.kda_kv_append_rope(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(Hq=-1), BAD), (dict(Hkv=-1), BAD), (dict(pages=-1), BAD), (dict(page=0), BAD), (dict(io=2), BAD),
    (dict(d=96), UNS), (dict(rot=0), UNS), (dict(rot=8), UNS), (dict(rot=24), UNS), (dict(rot=80), UNS), (dict(T=(1 << 30) + 1), BAD),
    (dict(Hq=65537), BAD), (dict(pages=1 << 20, page=1 << 11), BAD), (dict(qs=255), BAD), (dict(qs=260), BAD), (dict(ks=64), BAD),
    (dict(vs=-128), BAD), (dict(os=128), BAD), (dict(os=1 << 31), BAD), (dict(q=None), BAD), (dict(out=None), BAD), (dict(k=None), BAD),
    (dict(slot=None), BAD), (dict(pos=None), BAD), (dict(turns=None), BAD), (dict(vc=None), BAD), (dict(q=A[0] + 8), BAD),
    (dict(kc=A[6] + 4), BAD), (dict(turns=A[5] + 4), BAD), (dict(pos=A[4] + 2), BAD), (dict(status=A[9] + 1), BAD),
    (dict(kc=A[0]), BAD), (dict(vc=A[6] + 1024), BAD), (dict(out=A[1]), BAD), (dict(out=A[4]), BAD), (dict(out=A[0] + 16), BAD),
    (dict(out=A[0], os=512), BAD), (dict(out=A[6]), BAD), (dict(ko=A[2]), BAD), (dict(ko=A[8]), BAD), (dict(ko=A[1] + 16), BAD), (dict(kos=64), BAD),
    (dict(ko=A[10] + 8), BAD), (dict(ko=A[7]), BAD),
    (dict(T=0, k=None), OK), (dict(Hq=0, Hkv=0, q=None, k=None), OK),
])
def test_kv_append_rope_refuses(L, kw, code):
    assert rope(L, **kw) == code
    assert code == OK or L.kda_last_error_string()


def append(L, **kw):
    a = dict(c=A[0], kr=A[1], qr=A[2], slot=A[3], pos=A[4], turns=A[5], cache=A[6], qo=A[7], ko=A[8], T=4, Hq=4, dl=512, dr=64, neighbours=0,
             cs=576, krs=576, qrs=768, qrh=192, qos=2304, qoh=576, kos=64, pages=16, page=16, io=kda.KDA_BF16, status=None)
    a.update(kw)
    return L.kda_latent_append(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), BAD), (dict(Hq=-1), BAD), (dict(pages=-1), BAD), (dict(page=0), BAD), (dict(io=5), BAD), (dict(dl=256), UNS), (dict(dr=32), UNS),
    (dict(dr=-64), UNS), (dict(dr=0), BAD), (dict(T=(1 << 30) + 1), BAD), (dict(pages=1 << 20, page=1 << 11), BAD), (dict(c=None), BAD),
    (dict(kr=None), BAD), (dict(qr=None), BAD), (dict(qo=None), BAD), (dict(slot=None), BAD), (dict(pos=None), BAD), (dict(turns=None), BAD),
    (dict(cache=None), BAD), (dict(c=A[0] + 8), BAD), (dict(ko=A[8] + 2), BAD), (dict(turns=A[5] + 4), BAD), (dict(cs=508), BAD), (dict(cs=516), BAD),
    (dict(krs=32), BAD), (dict(kos=60), BAD), (dict(qrh=32), BAD), (dict(qrs=384), BAD), (dict(qos=576), BAD), (dict(qoh=580), BAD),
    (dict(cache=A[0]), BAD), (dict(qo=A[1]), BAD), (dict(ko=A[4]), BAD), (dict(qo=A[2], qos=768), BAD), (dict(ko=A[7]), BAD), (dict(qo=A[6]), BAD),
    (dict(status=A[9] + 2), BAD), (dict(T=0, c=None), OK),
    (dict(T=0, Hq=0, dr=0, ko=None, c=None), OK),
])
def test_latent_append_refuses(L, kw, code):
    assert append(L, **kw) == code


def prompt(L, **kw):
    a = dict(q=A[0], k=A[1], kr=A[2], v=A[3], cu=A[4], o=A[5], lse=A[6], N=2, total=16, most=16, H=4, d=128, dr=64, qs=768, qh=192, ks=1024, kh=256,
             krs=64, vs=1024, vh=256, scale=0.07, io=kda.KDA_BF16, ws=None, ws_bytes=0, status=None)
    a.update(kw)
    return L.kda_attn_latent_prompt(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(total=-1), BAD), (dict(most=-1), BAD), (dict(io=7), BAD), (dict(H=-1), BAD), (dict(H=65537), BAD), (dict(d=64), UNS),
    (dict(dr=32), UNS), (dict(scale=0.0), BAD), (dict(scale=float("nan")), BAD), (dict(q=None), BAD), (dict(k=None), BAD), (dict(kr=None), BAD),
    (dict(v=None), BAD), (dict(cu=None), BAD), (dict(o=None), BAD), (dict(q=A[0] + 8), BAD), (dict(kr=A[2] + 4), BAD), (dict(lse=A[6] + 2), BAD),
    (dict(qs=764), BAD), (dict(qs=384), BAD), (dict(qh=128), BAD), (dict(kh=64), BAD), (dict(ks=512), BAD), (dict(vs=1028), BAD), (dict(krs=56), BAD),
    (dict(krs=68), BAD), (dict(o=A[0]), BAD), (dict(o=A[2]), BAD), (dict(lse=A[3]), BAD), (dict(ws=A[5], ws_bytes=64), BAD), (dict(vs=1 << 31), BAD),
    (dict(N=0, q=None), OK), (dict(total=0, k=None), OK), (dict(most=0), OK), (dict(H=0), OK),
])
def test_latent_prompt_refuses(L, kw, code):
    assert prompt(L, **kw) == code


def paged(L, **kw):
    a = dict(q=A[0], cache=A[1], table=A[2], cu=A[3], kv=A[4], o=A[5], lse=None, N=2, total=2, most=1, Hq=4, dl=512, dr=64, qs=2304, qh=576, pages=16,
             page=16, max_pages=8, scale=0.07, io=kda.KDA_BF16, ws=None, ws_bytes=0, status=None)
    a.update(kw)
    return L.kda_attn_latent_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), BAD), (dict(total=-1), BAD), (dict(most=-1), BAD), (dict(pages=0), BAD), (dict(max_pages=-1), BAD), (dict(page=8), UNS),
    (dict(page=48), UNS), (dict(page=2048), UNS), (dict(page=0), BAD), (dict(dl=128), UNS), (dict(dr=128), UNS), (dict(Hq=-1), BAD), (dict(Hq=65537), BAD),
    (dict(pages=1 << 21, page=1 << 10), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("inf")), BAD), (dict(q=None), BAD), (dict(cache=None), BAD),
    (dict(table=None), BAD), (dict(kv=None), BAD), (dict(cu=None), BAD), (dict(o=None), BAD), (dict(cache=A[1] + 8), BAD), (dict(kv=A[4] + 2), BAD),
    (dict(o=A[1]), BAD), (dict(lse=A[2]), BAD), (dict(qs=2300), BAD), (dict(qs=1152), BAD), (dict(qh=512), BAD), (dict(io=3), BAD),
    (dict(ws=A[6] + 4, ws_bytes=64), BAD), (dict(N=0), OK), (dict(total=0), OK), (dict(most=0), OK), (dict(Hq=0), OK),
])
def test_latent_paged_refuses(L, kw, code):
    assert paged(L, **kw) == code


def test_workspace_size_refuses(L):
    bad = ctypes.c_size_t(-1).value
    f = L.kda_attn_latent_workspace_size
    assert f(-1, 1, 1, 4, 512, 64, kda.KDA_BF16) == bad
    assert f(1, 1, 1, 4, 256, 64, kda.KDA_BF16) == bad
    assert f(1, 1, 1, -4, 512, 64, kda.KDA_BF16) == bad
    assert f(1, 1, 1, 4, 512, 64, 9) == bad
    assert f(0, 0, 0, 4, 512, 64, kda.KDA_F32) == 0
