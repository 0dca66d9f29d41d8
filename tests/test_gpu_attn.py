"""Softmax attention over packed prompts and over the paged cache against the
64-bit definition (attn_ref.py: definitions and derived tolerances)."""
import pytest
import torch

import attn_ref
from gated_delta_rule_57_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cumulative(lens):
    return ints([0] + torch.cumsum(torch.tensor(lens), 0).tolist())


def randn(g, *shape, io, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(io)


def packed(lens, hq, hkv, d, io, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = randn(g, sum(lens), hq + 2 * hkv, d, io=io)
    return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]


def cached(q_lens, kv_lens, hq, hkv, d, page, io, seed=0, spare=2, stale=float("nan")):
    """A cache whose unwritten slots hold `stale`, its pages in any order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    held = [-(-x // page) for x in kv_lens]
    pages = sum(held) + spare
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(held), max(held + [1]) + 1), -1, dtype=torch.int32, device=DEV)
    kc = torch.full((pages, hkv, page, d), stale, dtype=io, device=DEV)
    vc = torch.full_like(kc, stale)
    at = 0
    for r, (h, x) in enumerate(zip(held, kv_lens)):
        table[r, :h] = ids[at:at + h]
        for j in range(h):
            n = min(page, x - j * page)
            kc[ids[at + j], :, :n] = randn(g, hkv, n, d, io=io)
            vc[ids[at + j], :, :n] = randn(g, hkv, n, d, io=io)
        at += h
    return randn(g, sum(q_lens), hq, d, io=io, std=1.5), kc, vc, table


LENS = [[1], [0, 1, 0, 2, 0], [127, 128, 129], [63, 64, 65, 1], [255, 256, 257], [1000, 3, 517], [2049]]
HEADS = [(1, 1, 64), (2, 1, 128), (6, 2, 128), (5, 1, 64), (16, 2, 128), (32, 2, 64), (64, 1, 128), (3, 3, 128)]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("case", range(len(LENS) + len(HEADS) - 1))
def test_prompt(case, io):
    lens = LENS[case] if case < len(LENS) else [200, 77]
    hq, hkv, d = HEADS[case - len(LENS) + 1] if case >= len(LENS) else HEADS[case % 3 + 1]
    q, k, v = packed(lens, hq, hkv, d, io, seed=case)
    status = ints([0])
    o, lse = kda.kda_attn_prompt(q, k, v, cumulative(lens), max_len=max(lens), status=status)
    torch.cuda.synchronize()
    attn_ref.check(o, lse, attn_ref.prompt(q, k, v, lens, d ** -0.5))
    assert int(status) == 0


@pytest.mark.parametrize("io", [BF, F32])
def test_prompt_scale_lse_and_unknown_longest(io):
    lens = [90, 300]
    q, k, v = packed(lens, 4, 2, 64, io)
    o, lse = kda.kda_attn_prompt(q.contiguous(), k.contiguous(), v.contiguous(), cumulative(lens), scale=0.31,
                                 want_lse=False)
    assert lse is None
    attn_ref.check(o, None, attn_ref.prompt(q, k, v, lens, 0.31))


@pytest.mark.parametrize("io", [BF, F32])
def test_prompt_large_scores(io):
    """Scores in the hundreds: the running maximum rises by more than the
    exponent's range between key tiles."""
    lens = [700]
    q, k, v = packed(lens, 2, 1, 128, io, seed=5)
    k = k.contiguous()
    k *= torch.linspace(0.1, 3.0, lens[0], device=DEV)[:, None, None].to(io)
    q = (q.float() * 4).to(io)
    o, lse = kda.kda_attn_prompt(q, k, v, cumulative(lens))
    ro, rl, a = attn_ref.prompt(q, k, v, lens, 128 ** -0.5)
    # scores to 250: their fp32 error (250 sqrt(128) 2^-24 = 1.7e-4) is the tolerance's
    tol = 1e-3 * a + (1.01 * attn_ref.U * (a + ro.abs()) if io == BF else 0)
    assert ((o.double() - ro).abs() <= tol).all()
    assert float((lse.double() - rl).abs().max()) <= 1e-3


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 5, 130, 299])
def test_prompt_later_tokens_do_not_reach_earlier_ones(io, bad, at):
    lens = [300, 40]
    q, k, v = (x.contiguous() for x in packed(lens, 8, 2, 128, io, seed=at))
    ref = attn_ref.prompt(q, k, v, lens, 128 ** -0.5)
    v[at], k[at] = bad, bad
    status = ints([0])
    o, lse = kda.kda_attn_prompt(q, k, v, cumulative(lens), status=status)
    torch.cuda.synchronize()
    ok = torch.ones(340, dtype=torch.bool, device=DEV)
    ok[at:300] = False
    attn_ref.check(o[ok], lse[ok], tuple(x[ok] for x in ref))
    assert not torch.isfinite(o[~ok]).any()
    assert int(status) == kda.KDA_DEV_NONFINITE


@pytest.mark.parametrize("io", [BF, F32])
def test_prompt_rows_of_no_prompt_are_left(io):
    q, k, v = packed([50], 4, 4, 64, io)
    o = torch.full((50, 4, 64), 7.0, dtype=io, device=DEV)
    lse = torch.full((50, 4), 7.0, device=DEV)
    kda.kda_attn_prompt(q, k, v, ints([3, 20, 20, 41]), o=o, lse=lse)
    torch.cuda.synchronize()
    for a, b in ((0, 3), (41, 50)):
        assert (o[a:b] == 7).all() and (lse[a:b] == 7).all()
    ref = attn_ref.prompt(q[3:41], k[3:41], v[3:41], [17, 21], 0.125)
    attn_ref.check(o[3:41], lse[3:41], ref)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("cu,most", [([0, 40, 20, 50], 50), ([0, 30, 60], 50), ([-4, 10], 50), ([0, 30, 50], 25)])
def test_prompt_bad_lengths_are_reported(io, cu, most):
    q, k, v = packed([50], 4, 2, 64, io)
    status = ints([0])
    kda.kda_attn_prompt(q, k, v, ints(cu), max_len=most, status=status)
    torch.cuda.synchronize()
    assert int(status) == kda.KDA_DEV_LENGTH


PAGED = [  # q_lens, kv_lens, hq, hkv, d, page
    ([1], [1], 1, 1, 64, 16),
    ([1, 1, 1], [700, 16, 17], 8, 2, 64, 16),
    ([1] * 33, [1 + 37 * i for i in range(33)], 8, 1, 128, 32),
    ([1, 1], [5000, 4999], 32, 2, 128, 64),
    ([4, 1, 3], [257, 128, 3], 6, 2, 128, 128),
    ([130, 1, 0, 64], [130, 513, 40, 1000], 8, 2, 128, 16),
    ([300], [2300], 4, 1, 64, 1024),
    ([17, 5], [600, 255], 64, 1, 128, 256),
    ([1, 40], [3000, 900], 5, 5, 64, 512),
]


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("case", range(len(PAGED)))
def test_paged(case, io):
    q_lens, kv_lens, hq, hkv, d, page = PAGED[case]
    q, kc, vc, table = cached(q_lens, kv_lens, hq, hkv, d, page, io, seed=case)
    status = ints([0])
    o, lse = kda.kda_attn_paged(q, kc, vc, table, cumulative(q_lens), ints(kv_lens), max_q=max(q_lens), status=status)
    torch.cuda.synchronize()
    ref = attn_ref.paged(q, kc, vc, table, q_lens, kv_lens, d ** -0.5)
    attn_ref.check(o, lse, ref)
    assert int(status) == 0
    # unsplit, and with a view of a fused projection
    wide = torch.zeros(q.shape[0], hq + 3, d, dtype=io, device=DEV)
    wide[:, :hq] = q
    o2, lse2 = kda.kda_attn_paged(wide[:, :hq], kc, vc, table, cumulative(q_lens), ints(kv_lens),
                                  workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    attn_ref.check(o2, lse2, ref)


@pytest.mark.parametrize("io", [BF, F32])
def test_paged_rows_that_see_nothing(io):
    """More new tokens than cached ones: the first rows see no key."""
    q_lens, kv_lens = [5, 200, 3], [2, 130, 0]
    q, kc, vc, table = cached(q_lens, kv_lens, 8, 2, 128, 16, io)
    o, lse = kda.kda_attn_paged(q, kc, vc, table, cumulative(q_lens), ints(kv_lens))
    torch.cuda.synchronize()
    ref = attn_ref.paged(q, kc, vc, table, q_lens, kv_lens, 128 ** -0.5)
    attn_ref.check(o, lse, ref)
    assert torch.isinf(lse[:3]).all() and not o[:3].any() and not o[205:].any()


@pytest.mark.parametrize("io", [BF, F32])
def test_paged_bad_tables_and_lengths_are_reported(io):
    q, kc, vc, table = cached([1, 1], [100, 60], 4, 2, 64, 16, io, stale=0.0)
    for change, want in ((lambda t, n: t.__setitem__((0, 2), 99), kda.KDA_DEV_PAGES),
                         (lambda t, n: t.__setitem__((1, 0), -5), kda.KDA_DEV_PAGES),
                         (lambda t, n: n.__setitem__(0, 16 * 8 + 1), kda.KDA_DEV_LENGTH),
                         (lambda t, n: n.__setitem__(1, -1), kda.KDA_DEV_LENGTH)):
        t, n, status = table.clone(), ints([100, 60]), ints([0])
        change(t, n)
        kda.kda_attn_paged(q, kc, vc, t, ints([0, 1, 2]), n, status=status)
        torch.cuda.synchronize()
        assert int(status) & want


@pytest.mark.parametrize("io", [BF, F32])
def test_paged_past_32_bits(io):
    """Pages beyond 2^31 elements of a cache."""
    hkv, page, d = 8, 64, 128
    pages = (1 << 31) // (hkv * page * d) + 40
    kc, vc = (torch.empty(pages, hkv, page, d, dtype=io, device=DEV) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(1)
    kc[-20:], vc[-20:] = (randn(g, 20, hkv, page, d, io=io) for _ in range(2))
    table = torch.arange(pages - 20, pages, device=DEV, dtype=torch.int32).flip(0)[None].contiguous()
    q = randn(g, 2, 16, d, io=io)
    o, lse = kda.kda_attn_paged(q, kc, vc, table, ints([0, 2]), ints([20 * page - 3]))
    attn_ref.check(o, lse, attn_ref.paged(q, kc[-20:], vc[-20:], table - (pages - 20), [2], [20 * page - 3], d ** -0.5))


@pytest.mark.parametrize("io", [BF, F32])
def test_repeats_streams_and_graphs_give_the_same_bits(io):
    q_lens, kv_lens = [1, 70, 1], [2000, 900, 33]
    q, kc, vc, table = cached(q_lens, kv_lens, 8, 2, 128, 64, io)
    cu, kv = cumulative(q_lens), ints(kv_lens)
    p = packed([300, 5, 600], 8, 2, 128, io)
    pcu = cumulative([300, 5, 600])

    def both():
        return kda.kda_attn_paged(q, kc, vc, table, cu, kv, max_q=70) + kda.kda_attn_prompt(*p, pcu, max_len=600)

    first = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = both()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        replayed = both()
    for x in replayed:
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(first, other, replayed):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("io", [BF, F32])
def test_cache_built_step_by_step_equals_the_prompt(io):
    """plan, append and paged attention over chunks and single tokens give what
    attention over the whole prompt gives."""
    lens, hq, hkv, d, page = [150, 61, 7], 8, 2, 128, 16
    q, k, v = packed(lens, hq, hkv, d, io, seed=11)
    whole, whole_lse = kda.kda_attn_prompt(q, k, v, cumulative(lens))
    starts = [0, 150, 211]
    n, pages = 3, 40
    table = torch.full((n, 12), -1, dtype=torch.int32, device=DEV)
    ring, at = torch.randperm(pages, device=DEV).to(torch.int32), ints([7, pages])
    kc, vc = (torch.full((pages, hkv, page, d), float("nan"), dtype=io, device=DEV) for _ in range(2))
    have = [0, 0, 0]
    kv = ints(have)
    status = ints([0])
    for step in [100, 1, 1, 30, 1, 1, 64]:
        new = [min(a + step, b) for a, b in zip(have, lens)]
        rows = [starts[r] + i for r in range(n) for i in range(have[r], new[r])]
        kv, cu, slot, at = kda.kda_kv_plan(kv, ints(new), table, ring, at, page_size=page,
                                           max_tokens=len(rows) + 2, status=status)
        rows = torch.tensor(rows, device=DEV)
        kda.kda_kv_append(k[rows], v[rows], slot, kc, vc, status=status)
        o, lse = kda.kda_attn_paged(q[rows], kc, vc, table, cu, kv, max_q=step, status=status)
        have = new
        ref = attn_ref.prompt(q, k, v, lens, d ** -0.5)
        attn_ref.check(o, lse, tuple(x[rows] for x in ref))
    torch.cuda.synchronize()
    assert have == lens and int(status) == 0
    attn_ref.check(whole, whole_lse, ref)


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,d,page", [([300], [2300], 4, 1, 64, 1024), ([70, 1], [1200, 1100], 8, 2, 128, 32),
                                                         ([40, 260, 1], [1111, 1500, 3], 6, 1, 128, 16)])
def test_ranges_of_few_key_tiles(q_lens, kv_lens, hq, hkv, d, page):
    """Ranges so short that a softmax group gets pieces without key tiles: every
    part is written before it is joined (the workspace starts as NaN), no wait
    runs out, and repeats give the same bits."""
    q, kc, vc, table = cached(q_lens, kv_lens, hq, hkv, d, page, BF, seed=d)
    ref = attn_ref.paged(q, kc, vc, table, q_lens, kv_lens, d ** -0.5)
    need = kda.kda_attn_workspace_size(len(q_lens), sum(q_lens), max(q_lens), hq, hkv, d)
    assert need > 0
    status, first = ints([0]), None
    for _ in range(30):
        ws = torch.full((need // 4,), float("nan"), device=DEV)
        o, lse = kda.kda_attn_paged(q, kc, vc, table, cumulative(q_lens), ints(kv_lens), max_q=max(q_lens),
                                    workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status) == 0
        if first is None:
            first = (o, lse)
            attn_ref.check(o, lse, ref)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("at", [3, 140, 256])
def test_one_bad_value_reaches_only_its_column(io, at):
    """A NaN in one channel of one token's value: that channel of the rows that
    see it, and nothing else."""
    lens = [300, 70]
    q, k, v = (x.contiguous() for x in packed(lens, 8, 2, 128, io, seed=at))
    ref = attn_ref.prompt(q, k, v, lens, 128 ** -0.5)
    v[at, 1, 5] = float("nan")
    status = ints([0])
    o, lse = kda.kda_attn_prompt(q, k, v, cumulative(lens), status=status)
    torch.cuda.synchronize()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[at:300, 4:, 5] = True
    assert torch.isnan(o[hit]).all() and int(status) == kda.KDA_DEV_NONFINITE
    attn_ref.check(torch.where(hit, ref[0].to(io), o), lse, ref)


@pytest.mark.parametrize("io", [BF, F32])
def test_a_call_on_a_stream_of_its_own(io):
    """stream= given while another stream is current: the workspace made by the
    call is not reused before that stream is done."""
    q_lens, kv_lens = [1, 3], [4000, 2500]
    q, kc, vc, table = cached(q_lens, kv_lens, 8, 2, 128, 64, io)
    cu, kv = cumulative(q_lens), ints(kv_lens)
    ref = attn_ref.paged(q, kc, vc, table, q_lens, kv_lens, 128 ** -0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        outs.append(kda.kda_attn_paged(q, kc, vc, table, cu, kv, max_q=3, stream=s))
        torch.full((1 << 22,), float("nan"), device=DEV)  # takes what the allocator thinks is free
    s.synchronize()
    for o, lse in outs:
        attn_ref.check(o, lse, ref)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,d,page", [([70, 1], [1200, 1100], 8, 2, 128, 32), ([40, 260, 1], [1111, 1500, 3], 6, 1, 128, 16),
                                                          ([1, 1, 1], [700, 588, 83], 8, 2, 64, 16), ([33] * 9, [33, 300, 129, 64, 1000, 95, 40, 511, 77], 4, 4, 64, 64)])
def test_short_requests_in_wide_tables(io, q_lens, kv_lens, hq, hkv, d, page):
    """Tables with room for long requests, so that the work is cut into ranges
    whatever the lengths are; the workspace starts as NaN."""
    q, kc, vc, table = cached(q_lens, kv_lens, hq, hkv, d, page, io, seed=page)
    wide = torch.full((table.shape[0], 9000 // page), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    ref = attn_ref.paged(q, kc, vc, table, q_lens, kv_lens, d ** -0.5)
    need = kda.kda_attn_workspace_size(len(q_lens), sum(q_lens), max(q_lens), hq, hkv, d, io)
    status, first = ints([0]), None
    for _ in range(10):
        ws = torch.full((need // 4,), float("nan"), device=DEV)
        o, lse = kda.kda_attn_paged(q, kc, vc, wide, cumulative(q_lens), ints(kv_lens), max_q=max(q_lens),
                                    workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status) == 0
        if first is None:
            first = (o, lse)
            attn_ref.check(o, lse, ref)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("lens,hq,hkv", [([5000], 4, 1), ([3000, 2900, 17], 2, 1), ([2500, 1, 2600], 6, 2)])
def test_prompts_cut_into_ranges(lens, hq, hkv):
    """Few long prompts of few heads, whose items are cut."""
    q, k, v = packed(lens, hq, hkv, 128, BF, seed=sum(lens))
    need = kda.kda_attn_workspace_size(len(lens), sum(lens), max(lens), hq, hkv, 128)
    ws, status = torch.full((need // 4,), float("nan"), device=DEV), ints([0])
    o, lse = kda.kda_attn_prompt(q, k, v, cumulative(lens), max_len=max(lens), workspace=ws, status=status)
    torch.cuda.synchronize()
    attn_ref.check(o, lse, attn_ref.prompt(q, k, v, lens, 128 ** -0.5))
    assert int(status) == 0
