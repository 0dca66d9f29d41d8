"""Latent attention where rows hold NaN or Inf, lengths and pages are wrong, or a call is
repeated, captured, on another stream or far into a cache."""
import math
import random

import pytest
import torch

import attn_ref
import gated_delta_rule_57_gb300 as pkg
import latent_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_latent_paged import DEV, DTYPES, case, ints
from test_gpu_latent_prompt import case as prompt_case

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
BF, F32 = DTYPES
SCALE = 0.07


def paged(q, cache, table, cu, kv, most=None, **kw):
    status = ints([0])
    o, lse = pkg.kda_attn_latent_paged(q, cache, table, cu, kv, scale=SCALE, max_q=most, status=status, **kw)
    torch.cuda.synchronize()
    return o, lse, int(status)


def widened(table, slots, page):
    wide = torch.full((table.shape[0], max(slots // page, table.shape[1])), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    return wide


def workspaces(n, total, most, hq, dr, io):
    """Made by the call, full of NaN, and none (whole rows)."""
    need = pkg.kda_attn_latent_workspace_size(n, total, most, hq, 512, dr, io)
    return None, torch.full((max(need, 4) // 4,), NAN, device=DEV), torch.empty(0, device=DEV)


def spoil(q, cache, table, q_lens, kv_lens, dr, io, bad):
    """Puts bad values (request, key, channel, value) into the cache. Returns which of o is
    not finite by the definition, and which rows' lse. A row that sees a bad row has a score
    that is NaN or +-Inf (its sign that of the query's channel): a row of NaN, but for a
    score of -Inf, which has weight 0 and leaves NaN in its channel alone."""
    starts = [0]
    for n in q_lens:
        starts.append(starts[-1] + n)
    page = cache.shape[1]
    hit = torch.zeros(q.shape[0], q.shape[1], 512, dtype=torch.bool, device=DEV)
    gone = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    for r, j, c, x in bad:
        cache[table[r, j // page].long(), j % page, c] = x
    for r, j, c, x in bad:
        first = starts[r] + max(0, j - (kv_lens[r] - q_lens[r]))
        rows = slice(first, starts[r + 1])
        low = (q[rows, :, c].float() * x) == -INF
        hit[rows] |= ~low[..., None]
        gone[rows] |= ~low
        if c < 512:
            hit[rows, :, c] = True
    return hit, gone


def check_spoiled(o, lse, ref, hit, gone, status):
    """Against the reference of the unspoiled cache, where a row sees nothing bad."""
    assert torch.equal(~torch.isfinite(o), hit)
    assert not torch.isfinite(lse[gone]).any()
    ro, rl, a = ref
    seen = hit.any(-1)
    attn_ref.check(torch.where(seen[..., None], ro.to(o.dtype), o), torch.where(seen, rl.float(), lse), ref)
    assert status == (kda.KDA_DEV_NONFINITE if hit.any() else 0)


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("x", [NAN, INF])
@pytest.mark.parametrize("q_lens,kv_lens,hq,dr,back", [
    ([4], [300], 8, 64, 1), ([4], [300], 8, 64, 4), ([40, 2], [2100, 130], 3, 0, 33), ([2, 1], [65, 40], 32, 64, 2), ([1], [97], 64, 64, 5),
    ([64], [64], 1, 64, 63), ([64], [2090], 1, 64, 40), ([3], [700], 128, 0, 2),
])
def test_bad_rows_reach_what_sees_them(io, x, q_lens, kv_lens, hq, dr, back):
    """A NaN or Inf among a request's last keys: tokens before it are as if it were
    not there (a latent counts as key and as value). Inf: some heads' scores are +Inf,
    others' -Inf."""
    q, cache, table, cu, kv = case(q_lens, kv_lens, hq, dr, 32, io, seed=back)
    ref = latent_ref.paged(q, cache, table, q_lens, kv_lens, SCALE)
    hit, gone = spoil(q, cache, table, q_lens, kv_lens, dr, io, [(0, kv_lens[0] - back, 77, x)])
    for t in (table, widened(table, 6000, 32)):
        for ws in workspaces(len(q_lens), sum(q_lens), max(q_lens), hq, dr, io):
            o, lse, status = paged(q, cache, t, cu, kv, max(q_lens), workspace=ws)
            check_spoiled(o, lse, ref, hit, gone, status)


@pytest.mark.parametrize("io", DTYPES)
def test_rows_of_scores_of_minus_infinity_see_nothing(io):
    cache = torch.zeros(1, 16, 576, dtype=io, device=DEV)
    cache[0, :3, 7], cache[0, :3, 570] = INF, 1.0
    q = torch.ones(1, 4, 576, device=DEV).to(io)
    q[0, 1:, 7] = -1.0
    o, lse, status = paged(q, cache, ints([[0]]), ints([0, 1]), ints([3]), 1)
    assert torch.isnan(o[0, 0]).all() and not o[0, 1:].any()
    assert not torch.isfinite(lse[0, 0]) and (lse[0, 1:] == -INF).all() and status == kda.KDA_DEV_NONFINITE


@pytest.mark.parametrize("io", DTYPES)
def test_a_bad_rotated_channel_is_a_key_only(io):
    q, cache, table, cu, kv = case([3], [200], 8, 64, 16, io, seed=9)
    ref = latent_ref.paged(q, cache, table, [3], [200], SCALE)
    hit, gone = spoil(q, cache, table, [3], [200], 64, io, [(0, 198, 512 + 5, INF)])
    o, lse, status = paged(q, cache, table, cu, kv, 3)
    ro, rl, a = ref
    low = ~hit.any(-1)
    low[0] = False  # the first token does not see it; the others' heads with a score of -Inf lose its weight
    assert torch.equal(~torch.isfinite(o), hit)
    cache[table[0, 198 // 16].long(), 198 % 16] = 0
    cache[table[0, 198 // 16].long(), 198 % 16, 512 + 5] = 0
    rows = latent_ref.attn_ref.gather(cache[:, None], table[0], 200)
    for t, h in low.nonzero().tolist():
        n = 198 + t  # keys it sees, of which key 198 has no weight
        s = (q[t, h].double() @ rows[:n, 0].double().t()) * SCALE
        s[198] = -INF
        p = torch.softmax(s, 0)
        y, size = p @ rows[:n, 0, :512].double(), p @ rows[:n, 0, :512].double().abs()
        tol = 1e-4 * size + (1.01 * attn_ref.U * (size + y.abs()) if io == BF else 0)
        assert ((o[t, h].double() - y).abs() <= tol).all() and abs(float(lse[t, h]) - float(torch.logsumexp(s, 0))) <= 1e-4
    attn_ref.check(o[:1], lse[:1], tuple(y[:1] for y in ref))


@pytest.mark.parametrize("io", DTYPES)
def test_wrong_lengths_and_pages(io):
    hq, dr, page, per = 5, 64, 64, 70
    g = torch.Generator(device=DEV).manual_seed(1)
    cache = torch.randn(3 * per, page, 576, generator=g, device=DEV).to(io)
    table = torch.randperm(3 * per, generator=g, device=DEV).to(torch.int32).view(3, per)
    q_lens, kv = [1, 3, 2], [per * page + 1, 700, -1]
    q = torch.randn(6, hq, 576, generator=g, device=DEV).to(io)
    cu = ints([0, 1, 4, 6])
    ref = latent_ref.paged(q, cache, table, q_lens, [per * page, 700, 0], SCALE)
    for ws in workspaces(3, 6, 3, hq, dr, io):
        o, lse, status = paged(q, cache, table, cu, ints(kv), 3, workspace=ws)
        assert status == kda.KDA_DEV_LENGTH
        attn_ref.check(o, lse, ref)
    # pages out of range read as zeros
    zeros, want = torch.cat([cache, torch.zeros_like(cache[:1])]), table.clone()
    for r, j, bad in ((0, 0, -1), (1, 2, 1 << 30), (1, 10, 3 * per)):
        table[r, j], want[r, j] = bad, 3 * per
    kv = [4000, 700, 90]
    ref = latent_ref.paged(q, zeros, want, q_lens, kv, SCALE)
    for ws in workspaces(3, 6, 3, hq, dr, io):
        o, lse, status = paged(q, cache, table, cu, ints(kv), 3, workspace=ws)
        assert status == kda.KDA_DEV_PAGES
        attn_ref.check(o, lse, ref)


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("cu,most,alone,right", [
    ([0, 3, 12, 13], 5, (3, 12), [0, 2]), ([0, 3, 2, 13], 20, (0, 0), [0]), ([-2, 3, 12, 13], 20, (0, 3), [1, 2]), ([0, 3, 12, 14], 20, (12, 13), [0, 1]),
])
def test_rows_of_wrong_requests_are_left_alone(io, cu, most, alone, right):
    """More new tokens than announced, offsets that decrease, start below zero or end past
    the rows; rows behind the last request."""
    kv_lens, hq = [800, 3000, 44], 8
    q, cache, table, _, kv = case([3, 9, 3], kv_lens, hq, 64, 32, io)
    q = q[:13].contiguous()
    for ws in workspaces(3, 13, most, hq, 64, io):
        o, lse = torch.full((13, hq, 512), 7.0, dtype=io, device=DEV), torch.full((13, hq), 7.0, device=DEV)
        _, _, status = paged(q, cache, table, ints(cu), kv, most, workspace=ws, o=o, lse=lse)
        assert status == kda.KDA_DEV_LENGTH
        assert (o[alone[0]:alone[1]] == 7).all() and (lse[alone[0]:alone[1]] == 7).all()
        for r in right:
            a, b = cu[r], cu[r + 1]
            attn_ref.check(o[a:b], lse[a:b], latent_ref.paged(q[a:b], cache, table[r:r + 1], [b - a], kv_lens[r:r + 1], SCALE))


@pytest.mark.parametrize("io", DTYPES)
def test_empty_requests_and_rows_that_see_nothing(io):
    q_lens, kv_lens = [0, 5, 0, 3, 1], [40, 2, 0, 0, 70]
    q, cache, table, cu, kv = case(q_lens, kv_lens, 6, 64, 16, io)
    ref = latent_ref.paged(q, cache, table, q_lens, kv_lens, SCALE)
    o, lse = torch.full((12, 6, 512), 7.0, dtype=io, device=DEV), torch.full((12, 6), 7.0, device=DEV)
    q = torch.cat([q, q[:3]])  # and rows of no request
    for ws in workspaces(5, 12, 5, 6, 64, io):
        _, _, status = paged(q, cache, widened(table, 5000, 16), cu, kv, 5, workspace=ws, o=o, lse=lse)
        assert status == 0
        attn_ref.check(o[:9], lse[:9], ref)
        assert (o[9:] == 7).all() and (lse[9:] == 7).all()
    assert not o[:3].any() and not o[5:8].any()


@pytest.mark.parametrize("io", DTYPES)
def test_past_32_bits(io):
    """A cache of more than 2^31 elements and, its table's ids, at its end."""
    page = 1024
    pages = (1 << 31) // (page * 576) + 4
    cache = torch.empty(pages, page, 576, dtype=io, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(2)
    cache[-3:] = torch.randn(3, page, 576, generator=g, device=DEV).to(io)
    table = ints([[pages - 1, pages - 3, pages - 2]])
    q = torch.randn(2, 8, 576, generator=g, device=DEV).to(io)
    o, lse, status = paged(q, cache, table, ints([0, 2]), ints([3 * page - 3]), 2)
    attn_ref.check(o, lse, latent_ref.paged(q, cache[-3:], table - (pages - 3), [2], [3 * page - 3], SCALE))
    k_r, c, i = cache[-1, :40, 512:].clone(), cache[-1, :40, :512].clone(), torch.arange(40, dtype=torch.int32, device=DEV)
    turns = pkg.kda_rope_turns([0.0] * 32)  # no rotation: copies
    pkg.kda_latent_append(c, k_r, i + (pages - 2) * page + 7, cache, positions=i, turns=turns)
    torch.cuda.synchronize()
    assert torch.equal(cache[-2, 7:47, :512], c) and torch.equal(cache[-2, 7:47, 512:], k_r) and status == 0


@pytest.mark.parametrize("io", DTYPES)
def test_length_near_2_to_31(io):
    cache = torch.ones(1, 1024, 576, dtype=io, device=DEV)
    table = torch.full((1, 1 << 21), -1, dtype=torch.int32, device=DEV)
    q = torch.ones(1, 1, 576, device=DEV).to(io)
    o, lse, status = paged(q, cache, table, ints([0, 1]), ints([(1 << 31) - 1]), 1)
    assert status == kda.KDA_DEV_LENGTH | kda.KDA_DEV_PAGES
    assert not o.any() and abs(float(lse) - 30 * 0.6931471805599453) <= 1e-4


@pytest.mark.parametrize("io", DTYPES)
def test_repeats_streams_and_graphs_give_the_same_bits(io):
    q_lens, kv_lens = [1, 30, 1], [2000, 900, 33]
    q, cache, table, cu, kv = case(q_lens, kv_lens, 8, 64, 64, io)
    lens = [300, 5, 600]
    p = prompt_case(lens, 3, 64, io)

    def both():
        return pkg.kda_attn_latent_paged(q, cache, table, cu, kv, scale=SCALE, max_q=30) + pkg.kda_attn_latent_prompt(*p, max_len=600)

    first = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = both()
    s.synchronize()
    own = pkg.kda_attn_latent_paged(q, cache, table, cu, kv, scale=SCALE, max_q=30, stream=s) + \
        pkg.kda_attn_latent_prompt(*p, max_len=600, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        replayed = both()
    for x in replayed:
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    for x, y, z, w in zip(first, other, own, replayed):
        assert torch.equal(x, y) and torch.equal(x, z) and torch.equal(x, w)


def test_appends_in_a_graph():
    """Captured once, replayed for another step's positions and slots."""
    g = torch.Generator(device=DEV).manual_seed(0)
    down, q = torch.randn(6, 576, generator=g, device=DEV).to(BF), torch.randn(6, 4, 192, generator=g, device=DEV).to(BF)
    qkv = torch.randn(6, 8, 64, generator=g, device=DEV).to(BF)
    freq = latent_ref.frequencies(64)
    turns, slot, pos = pkg.kda_rope_turns(freq), ints(list(range(6))), ints([5] * 6)
    cache, kc, vc = (torch.zeros(s, dtype=BF, device=DEV) for s in ((2, 16, 576), (2, 2, 16, 64), (2, 2, 16, 64)))

    def step():
        return (pkg.kda_latent_append(down[:, :512], down[:, 512:], slot, cache, positions=pos, turns=turns, q_r=q[..., 128:]),
                pkg.kda_kv_append_rope(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], slot, pos, turns, kc, vc))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = step()
    pos.copy_(ints([1000, 2, 3, 70000, 5, 6]))
    slot.copy_(ints([20, 21, -1, 22, 23, 24]))
    graph.replay()
    torch.cuda.synchronize()
    latent_ref.check_rotated(a, latent_ref.rotate(q[..., 128:], pos, freq, False))
    latent_ref.check_rotated(b, latent_ref.rotate(qkv[:, :4], pos, freq, False))
    kr, size = latent_ref.rotate(down[:, None, 512:], pos, freq, False)
    latent_ref.check_rotated(cache[1, 4:6, 512:], (kr[:2, 0], size[:2, 0]))
    assert torch.equal(vc[1, :, 6:9], qkv[3:, 6:].transpose(0, 1))


# ------------------------------------------------------------------------- prompts
@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("lens,at", [([300, 40], 256), ([300, 40], 299), ([70], 3), ([2600, 30], 2590)])
def test_prompt_bad_values(io, lens, at):
    """A NaN in k, k_r or v reaches the tokens from it on and no others; in v, one channel."""
    q, k, k_r, v, cu = prompt_case(lens, 2, 64, io, seed=at)
    ref = latent_ref.prompt(q, k, k_r, v, lens, 192 ** -0.5)
    for which in ("k", "k_r", "v"):
        k2, r2, v2 = k.clone(), k_r.clone(), v.clone()
        hit = torch.zeros(sum(lens), 2, 128, dtype=torch.bool, device=DEV)
        if which == "v":
            v2[at, 1, 5] = NAN
            hit[at:lens[0], 1, 5] = True
        elif which == "k":
            k2[at, 1, 5] = NAN
            hit[at:lens[0], 1] = True
        else:
            r2[at, 5] = NAN
            hit[at:lens[0]] = True
        status = ints([0])
        o, lse = pkg.kda_attn_latent_prompt(q, k2, r2, v2, cu, max_len=max(lens), status=status)
        torch.cuda.synchronize()
        assert torch.equal(torch.isnan(o), hit) and int(status) == kda.KDA_DEV_NONFINITE
        gone = hit.all(-1)
        assert torch.equal(torch.isnan(lse), gone)
        attn_ref.check(torch.where(hit, ref[0].to(io), o), torch.where(gone, ref[1].float(), lse), ref)


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("cu,most,alone,right", [
    ([0, 30, 60], 50, (30, 50), [(0, 30)]), ([-4, 10, 50], 50, (0, 10), [(10, 50)]), ([0, 30, 50], 25, (0, 30), [(30, 50)]),
    ([0, 3000, 5000], 2999, (0, 3000), [(3000, 5000)]), ([0, 20, 20, 45], 50, (45, 50), [(0, 20), (20, 45)]),
])
def test_prompt_wrong_lengths(io, cu, most, alone, right):
    total = max(alone[1], right[-1][1])
    q, k, k_r, v, _ = prompt_case([total], 2, 64, io, seed=most)
    bad = cu != [0, 20, 20, 45]
    for ws in (None, torch.empty(0, device=DEV)):
        o, lse = torch.full((total, 2, 128), 7.0, dtype=io, device=DEV), torch.full((total, 2), 7.0, device=DEV)
        status = ints([0])
        pkg.kda_attn_latent_prompt(q, k, k_r, v, ints(cu), max_len=most, o=o, lse=lse, workspace=ws, status=status)
        torch.cuda.synchronize()
        assert int(status) == (kda.KDA_DEV_LENGTH if bad else 0)
        assert (o[alone[0]:alone[1]] == 7).all() and (lse[alone[0]:alone[1]] == 7).all()
        for a, b in right:
            attn_ref.check(o[a:b], lse[a:b], latent_ref.prompt(q[a:b], k[a:b], k_r[a:b], v[a:b], [b - a], 192 ** -0.5))


# ------------------------------------------------------------------------- drawn calls
def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        io, dr, hq = rng.choice([BF, BF, BF, F32]), rng.choice([0, 64]), rng.choice([1, 2, 3, 5, 8, 16, 20, 31, 32, 33, 40, 64, 66, 128])
        n, page = rng.choice([1, 2, 3, rng.randint(1, 40)]), rng.choice([16, 32, 64, 128, 256, 1024])
        longest = rng.choice([40, 300, 3000, 9000])
        kv = [max(0, log_int(rng, 1, longest) - rng.choice([0, 0, 1])) for _ in range(n)]
        q = [rng.choice([1, 1, 0, rng.randint(0, 12), log_int(rng, 1, 200)]) for _ in range(n)]
        if rng.random() < 0.9:
            q = [min(a, b) for a, b in zip(q, kv)]
        if 0 < sum(q) and sum(a * b for a, b in zip(q, kv)) * hq <= 3e7 and sum(kv) <= 60000:
            return q, kv, hq, dr, page, io


@pytest.mark.parametrize("seed", range(100))
def test_drawn_calls(seed):
    rng = random.Random(seed)
    q_lens, kv_lens, hq, dr, page, io = draw(rng)
    n, total = len(q_lens), sum(q_lens)
    q, cache, table, cu, kv = case(q_lens, kv_lens, hq, dr, page, io, seed=seed)
    most = rng.choice([max(q_lens), max(q_lens), None, max(q_lens) + rng.randint(0, 300)])
    if rng.random() < 0.5:
        table = widened(table, rng.choice([3000, 20000]), page)
    if rng.random() < 0.5:  # tokens inside heads
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    ref = latent_ref.paged(q, cache, table, q_lens, kv_lens, SCALE)
    bad, used = [], set()
    for _ in range(0 if rng.random() < 0.5 else rng.randint(1, 4)):  # mostly near a request's end
        r = rng.randrange(n)
        if kv_lens[r] == 0:
            continue
        j = kv_lens[r] - 1 - rng.randint(0, min(kv_lens[r], max(q_lens[r], 1) + 2) - 1)
        if (r, j) not in used:
            used.add((r, j))
            # (a score of -Inf takes a key's weight away, which the reference does not know: NaN only)
            bad.append((r, j, rng.randrange(512), NAN))
    hit, gone = spoil(q, cache, table, q_lens, kv_lens, dr, io, bad)
    ws = rng.choice(workspaces(n, total, total if most is None else most, hq, dr, io))
    o, lse, status = paged(q, cache, table, cu, kv, most, workspace=ws)
    check_spoiled(o, lse, ref, hit, gone, status)


@pytest.mark.parametrize("seed", range(60))
def test_drawn_prompts(seed):
    rng = random.Random(1000 + seed)
    while True:
        io, dr, h = rng.choice([BF, BF, BF, F32]), rng.choice([0, 64, 64]), rng.choice([1, 2, 3, 5, 8, 16])
        lens = [max(0, log_int(rng, 1, rng.choice([5, 100, 700, 2600])) - rng.choice([0, 0, 1])) for _ in range(rng.choice([1, 2, 3, rng.randint(1, 30)]))]
        if 0 < sum(lens) and sum(x * x for x in lens) * h <= 3e7:
            break
    q, k, k_r, v, cu = prompt_case(lens, h, dr, io, seed=seed)
    if rng.random() < 0.5:  # tokens inside heads
        q, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, v))
    ref = latent_ref.prompt(q, k, k_r, v, lens, (128 + dr) ** -0.5)
    hit, gone = torch.zeros(sum(lens), h, 128, dtype=torch.bool, device=DEV), torch.zeros(sum(lens), h, dtype=torch.bool, device=DEV)
    starts = cu.tolist()
    for _ in range(0 if rng.random() < 0.5 else rng.randint(1, 4)):
        r = rng.randrange(len(lens))
        if lens[r] == 0:
            continue
        at, head, c = starts[r] + rng.randrange(lens[r]), rng.randrange(h), rng.randrange(128)
        rows = slice(at, starts[r + 1])
        if rng.random() < 0.5:
            v[at, head, c] = NAN
            hit[rows, head, c] = True
        elif dr and rng.random() < 0.5:
            k_r[at, c % dr] = NAN
            hit[rows], gone[rows] = True, True
        else:
            k[at, head, c] = NAN
            hit[rows, head], gone[rows, head] = True, True
    need = kda.kda_attn_workspace_size(len(lens), sum(lens), max(lens), h, h, 128, io)
    ws = rng.choice([None, torch.full((max(need, 4) // 4,), NAN, device=DEV), torch.empty(0, device=DEV)])
    status = ints([0])
    o, lse = pkg.kda_attn_latent_prompt(q, k, k_r, v, cu, max_len=rng.choice([None, max(lens)]), workspace=ws, status=status)
    torch.cuda.synchronize()
    assert torch.equal(~torch.isfinite(o), hit) and torch.equal(torch.isnan(lse), gone)
    attn_ref.check(torch.where(hit, ref[0].to(io), o), torch.where(gone, ref[1].float(), lse), ref)
    assert int(status) == (kda.KDA_DEV_NONFINITE if hit.any() else 0)


@pytest.mark.parametrize("io", DTYPES)
def test_calls_at_once_on_two_streams(io):
    """Each with the workspace that it makes: the bits of calls alone."""
    cases = [case([1, 3], [5000, 4000], 8, 64, 64, io, seed=1), case([2] * 9, [700] * 9, 40, 0, 16, io, seed=2)]
    prompts = [prompt_case([2500, 3], 2, 64, io, seed=3), prompt_case([100, 900], 5, 0, io, seed=4)]

    def calls(i):
        return (*pkg.kda_attn_latent_paged(*cases[i], scale=SCALE, max_q=3), *pkg.kda_attn_latent_prompt(*prompts[i]))

    alone = [calls(i) for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, calls(i)))
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(x, y) for x, y in zip(alone[i], out))


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("n,longest,hq", [(800, 64, 4), (400, 60, 1), (350, 500, 3), (320, 700, 2)])
def test_many_requests(io, n, longest, hq):
    """More items than SMs, whole or in ranges, of requests of any length and none."""
    rng = random.Random(n + longest)
    kv_lens = [rng.choice([longest, 0, 1, rng.randint(1, longest)]) for _ in range(n)]
    q_lens = [rng.choice([1, 1, 1, 0, 2]) for _ in range(n)]
    q, cache, table, cu, kv = case(q_lens, kv_lens, hq, 64, 16, io)
    o, lse, status = paged(q, cache, table, cu, kv, 2)
    attn_ref.check(o, lse, latent_ref.paged(q, cache, table, q_lens, kv_lens, SCALE))
    assert int(status) == 0


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("n,longest,h", [(65, 64, 3), (300, 40, 2), (200, 380, 1), (70, 400, 1)])
def test_many_prompts(io, n, longest, h):
    rng = random.Random(n + longest)
    lens = [rng.choice([longest, 0, 1, rng.randint(1, longest)]) for _ in range(n)]
    q, k, k_r, v, cu = prompt_case(lens, h, 64, io)
    o, lse = pkg.kda_attn_latent_prompt(q, k, k_r, v, cu, max_len=longest)
    attn_ref.check(o, lse, latent_ref.prompt(q, k, k_r, v, lens, 192 ** -0.5))


@pytest.mark.parametrize("io", DTYPES)
def test_calls_without_work(io):
    """No tokens, no requests, no heads: nothing is read or written, outputs have their shapes."""
    def x(*shape):
        return torch.zeros(shape, dtype=io, device=DEV)
    cache, kc, turns = x(4, 16, 576).fill_(3), x(4, 2, 16, 64).fill_(3), pkg.kda_rope_turns([1.0] * 32)
    status, none = ints([0]), ints([])
    for t, n, h in [(0, 0, 4), (0, 3, 4), (5, 0, 4), (5, 1, 0)]:
        cu = ints([0] * n + [t])
        o, lse = pkg.kda_attn_latent_paged(x(t, h, 576), cache, ints([[0]] * n).view(n, 1), cu, ints([1] * n), scale=1.0, status=status)
        assert o.shape == (t, h, 512) and lse.shape == (t, h)
        o, lse = pkg.kda_attn_latent_prompt(x(t, h, 192), x(t, h, 128), x(t, 64), x(t, h, 128), cu, status=status)
        assert o.shape == (t, h, 128) and lse.shape == (t, h)
    assert pkg.kda_latent_append(x(0, 512), x(0, 64), none, cache, positions=none, turns=turns, q_r=x(0, 2, 64)).shape == (0, 2, 64)
    assert pkg.kda_kv_append_rope(x(0, 3, 64), x(0, 2, 64), x(0, 2, 64), none, none, turns, kc, kc.clone()).shape == (0, 3, 64)
    torch.cuda.synchronize()
    assert int(status) == 0 and (cache == 3).all() and (kc == 3).all()


@pytest.mark.parametrize("io", DTYPES)
def test_queries_or_keys_alone(io):
    """A call that rotates only queries, and one that only appends."""
    q, k, v = (torch.randn(7, 2, 64, device=DEV).to(io) for _ in range(3))
    freq = latent_ref.frequencies(64)
    turns, at, slots = pkg.kda_rope_turns(freq), ints(list(range(50, 57))), ints(list(range(7)))
    kc, vc = (torch.full((1, 2, 16, 64), 5.0, dtype=io, device=DEV) for _ in range(2))
    assert pkg.kda_kv_append_rope(None, k, v, slots, at, turns, kc, vc) is None
    torch.cuda.synchronize()
    latent_ref.check_rotated(kc[0, :, :7].transpose(0, 1), latent_ref.rotate(k, at, freq, False))
    assert torch.equal(vc[0, :, :7].transpose(0, 1), v) and (kc[0, :, 7:] == 5).all() and (vc[0, :, 7:] == 5).all()
    none = torch.empty(7, 0, 64, dtype=io, device=DEV)
    empty = torch.empty(1, 0, 16, 64, dtype=io, device=DEV)
    out = pkg.kda_kv_append_rope(q, none, none, slots, at, turns, empty, empty)
    torch.cuda.synchronize()
    latent_ref.check_rotated(out, latent_ref.rotate(q, at, freq, False))


@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("x", [NAN, INF])
def test_a_bad_query_is_its_own_rows(io, x):
    """NaN or Inf in a head's query: that head's row of that token and no other, whole and in ranges.
    (Inf: among the keys that such a row sees here there is one whose score is +Inf.)"""
    q_lens, kv_lens, hq = [3, 1, 2], [700, 3000, 40], 20
    q, cache, table, cu, kv = case(q_lens, kv_lens, hq, 64, 64, io)
    ref = latent_ref.paged(q, cache, table, q_lens, kv_lens, SCALE)
    hit = torch.zeros(6, hq, dtype=torch.bool, device=DEV)
    for t, h, c in [(0, 3, 0), (2, 19, 511), (3, 7, 570), (5, 0, 100)]:
        q[t, h, c] = x
        hit[t, h] = True
    for ws in workspaces(3, 6, 3, hq, 64, io):
        o, lse, status = paged(q, cache, table, cu, kv, 3, workspace=ws)
        check_spoiled(o, lse, ref, hit[..., None].expand(-1, -1, 512), hit, status)
    lens = [300, 70, 2500]
    q, k, k_r, v, cu = prompt_case(lens, 2, 64, io)
    ref = latent_ref.prompt(q, k, k_r, v, lens, 192 ** -0.5)
    hit = torch.zeros(sum(lens), 2, dtype=torch.bool, device=DEV)
    for t, h, c in [(299, 0, 5), (100, 1, 191), (310, 1, 127), (2000, 0, 130)]:
        q[t, h, c] = x
        hit[t, h] = True
    o, lse = pkg.kda_attn_latent_prompt(q, k, k_r, v, cu, max_len=2500)
    torch.cuda.synchronize()
    assert torch.equal(~torch.isfinite(o), hit[..., None].expand_as(o)) and torch.equal(torch.isnan(lse), hit)
    attn_ref.check(torch.where(hit[..., None], ref[0].to(io), o), torch.where(hit, ref[1].float(), lse), ref)
