"""Page planning and cache writes against their serial definitions; whole
numbers and copies, so every comparison is exact."""
import random

import pytest
import torch

import attn_ref
from gated_delta_rule_57_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def state(rng, old, page, max_pages, spare):
    """A table that holds the requests' pages and a ring of the free ones."""
    held = [-(-x // page) for x in old]
    pages = sum(held) + spare
    ids = list(range(pages))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-7] * (max_pages - h))
        at += h
    head = rng.randrange(pages)
    ring = [-9] * pages
    for i in range(spare):
        ring[(head + i) % pages] = ids[at + i]
    return table, ring, [head, spare]


def run(old, new, table, ring, at, page, room):
    t = ints(table) if table else torch.empty(0, 3, dtype=torch.int32, device=DEV)
    r, status = ints(ring), ints([0])
    kv, cu, slot, out = kda.kda_kv_plan(ints(old), ints(new), t, r, ints(at), page_size=page,
                                        max_tokens=room, status=status)
    torch.cuda.synchronize()
    return [x.tolist() for x in (kv, cu, slot, t, r, out)], int(status)


@pytest.mark.parametrize("n,page,longest", [(1, 16, 40), (2, 1, 9), (31, 7, 100), (33, 48, 1000),
                                            (256, 64, 3000), (513, 16, 700), (2049, 128, 4000)])
@pytest.mark.parametrize("short", ["", "pages", "row", "tokens"])
def test_plan(n, page, longest, short):
    rng = random.Random(n * 7 + len(short))
    old = [rng.choice([0, rng.randint(0, longest)]) for _ in range(n)]
    new = [rng.choice([x, x + 1, min(longest, x + rng.randint(0, 3 * page)), max(0, x - rng.randint(0, page)), 0])
           for x in old]
    max_pages = max(-(-max(old + new) // page), 1)
    table, ring, at = state(rng, old, page, max_pages, spare=max(2, n * 4))
    room = sum(max(0, b - a) for a, b in zip(old, new)) + rng.choice([0, 5])
    if short == "pages":
        at[1] = min(at[1], 1 + n // 5)
    elif short == "row":
        r = rng.randrange(n)
        new[r] = max_pages * page + 1
        room += new[r]
    elif short == "tokens":
        room = room // 2
    got, status = run(old, new, table, ring, at, page, room)
    want = attn_ref.plan(old, new, table, ring, at, page, room)
    assert got == list(want[:6])
    assert status == (kda.KDA_DEV_PAGES if want[6] else 0)


def test_plan_steps_reuse_pages():
    """Many steps over one cache: no page is ever held twice, none is lost."""
    rng = random.Random(3)
    n, page, max_pages = 40, 16, 20
    table, ring, at = state(rng, [0] * n, page, max_pages, spare=500)
    old = [0] * n
    t, r, a = ints(table), ints(ring), ints(at)
    kv = ints(old)
    for step in range(40):
        new = [0 if rng.random() < 0.1 else min(page * max_pages, x + rng.choice([1, 1, 1, 40])) for x in kv.tolist()]
        kv, cu, slot, a = kda.kda_kv_plan(kv, ints(new), t, r, a, page_size=page, max_tokens=40 * n)
        head, count = a.tolist()
        held = [i for x, row in zip(kv.tolist(), t.tolist()) for i in row[:-(-x // page)]]
        free = [r.tolist()[(head + i) % 500] for i in range(count)]
        assert sorted(held + free) == list(range(500))


def test_plan_most_requests_and_none():
    old, new = [1] * 16384, [2] * 16384
    table = [[i, -1] for i in range(16384)]
    got, status = run(old, new, table, list(range(16384)) + [0], [0, 1], 1, 16384)
    want = attn_ref.plan(old, new, table, list(range(16384)) + [0], [0, 1], 1, 16384)
    assert got == list(want[:6]) and status == kda.KDA_DEV_PAGES
    got, status = run([], [], [], [5, 4, 3], [2, 2], 16, 4)
    assert got == [[], [0], [-1] * 4, [], [5, 4, 3], [2, 2]] and status == 0
    with pytest.raises(kda.KdaError) as e:
        run([0] * 16385, [0] * 16385, [[0]] * 16385, [0], [0, 0], 16, 4)
    assert e.value.code == kda.KDA_ERR_UNSUPPORTED


def test_plan_reports_bad_lengths_ring_and_ids():
    # a negative length counts as 0; a ring state out of range is clamped; a
    # page id out of range gives no slot
    got, status = run([-3, 5], [1, 6], [[0, 0], [9, 0]], [1, 2, 3], [4, 9], 4, 3)
    assert status & kda.KDA_DEV_LENGTH and status & kda.KDA_DEV_PAGES
    got, status = run([5], [6], [[1, 99]], [0, 2, 3], [0, 1], 4, 2)
    assert status == kda.KDA_DEV_PAGES and got[2] == [-1, -1]


@pytest.mark.parametrize("t,hkv,d,page,io", [(1, 1, 64, 16, torch.bfloat16), (7, 3, 128, 16, torch.float32),
                                             (256, 8, 128, 64, torch.bfloat16), (1000, 5, 64, 48, torch.float32),
                                             (333, 40, 128, 7, torch.bfloat16)])
@pytest.mark.parametrize("fused", [False, True])
def test_append(t, hkv, d, page, io, fused):
    g = torch.Generator(device=DEV).manual_seed(t)
    pages = -(-2 * t // page) + 1
    kc, vc = (torch.randn(pages, hkv, page, d, generator=g, device=DEV).to(io) for _ in range(2))
    qkv = torch.randn(t, 4 * hkv, d, generator=g, device=DEV).to(io)
    k, v = qkv[:, 2 * hkv:3 * hkv], qkv[:, 3 * hkv:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    slot = torch.randperm(pages * page, generator=g, device=DEV)[:t].to(torch.int32)
    slot[::3] = -1
    if t > 4:
        slot[4] = pages * page
    rk, rv = kc.clone(), vc.clone()
    for i, s in enumerate(slot.tolist()):
        if 0 <= s < pages * page:
            rk[s // page, :, s % page] = k[i]
            rv[s // page, :, s % page] = v[i]
    status = ints([0])
    kda.kda_kv_append(k, v, slot, kc, vc, status=status)
    torch.cuda.synchronize()
    assert torch.equal(kc, rk) and torch.equal(vc, rv)
    assert int(status) == (kda.KDA_DEV_PAGES if t > 4 else 0)


def test_append_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: its last page."""
    pages, hkv, page, d = (1 << 31) // (8 * 64 * 128) + 3, 8, 64, 128
    kc, vc = (torch.empty(pages, hkv, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kc[-2:], vc[-2:] = 0, 0
    k, v = (torch.randn(page, hkv, d, device=DEV).bfloat16() for _ in range(2))
    kda.kda_kv_append(k, v, ints([(pages - 1) * page + i for i in range(page)]), kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc[-1], k.transpose(0, 1)) and torch.equal(vc[-1], v.transpose(0, 1))
    assert not kc[-2].any() and not vc[-2].any()
