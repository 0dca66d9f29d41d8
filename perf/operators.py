"""Measured cases of the attention and paged-cache operators.

A stack that mixes Kimi Delta Attention layers with softmax-attention layers
keeps, for the latter, a paged key/value cache next to the fixed-size
recurrent states. Four operators serve it:

  plan    block tables, slot map and free list built on the GPU from lengths
  append  new keys and values written to their slots of the paged cache
  prompt  causal attention over packed prompts of different lengths, grouped heads
  paged   causal attention of a chunk of new tokens (one or many) over the paged cache

Each has a plain form below (elementary torch operations in 32 bits) and its
call through the package. Layouts: q [T, Hq, d], k and v [T, Hkv, d] (views of
one fused projection where a case says so), caches [pages, Hkv, page, d].
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCORES = 1 << 31  # largest score tensor of the plain form, in elements


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one scheduling step of a decode batch: every request gains one token
        {"name": "plan_decode_n256", "op": "plan", "n": 256, "page": 64, "longest": 8192, "chunk": 1, "lengths": 1},
        # a large mixed step with small pages: prompts' chunks, single tokens, drafts taken back, requests that end
        {"name": "plan_mixed_n2048", "op": "plan", "n": 2048, "page": 16, "longest": 32768, "chunk": 2048, "lengths": 2},
        # one token each of a decode batch goes to the cache: latency counts
        {"name": "append_decode_t256", "op": "append", "tokens": 256, "hkv": 8, "d": 128, "page": 64, "io": "bf16"},
        # eight prompts of 8192 tokens go to the cache
        {"name": "append_prompt_t65536", "op": "append", "tokens": 65536, "hkv": 8, "d": 128, "page": 64, "io": "bf16"},
        # a handful of short prompts on a small model: latency counts
        {"name": "prompt_short_d64", "op": "prompt", "n": 5, "longest": 255, "hq": 4, "hkv": 2, "d": 64, "io": "bf16", "lengths": 3},
        # the accuracy path, in 32 bits
        {"name": "prompt_f32_d64", "op": "prompt", "n": 3, "longest": 1021, "hq": 8, "hkv": 2, "d": 64, "io": "f32", "lengths": 4},
        # a packed batch of prompts of very different lengths
        {"name": "prompt_ragged_n24", "op": "prompt", "n": 24, "longest": 4096, "hq": 32, "hkv": 8, "d": 128, "io": "bf16", "lengths": 5},
        # the prefill batch of the benchmark: eight prompts of 8192 tokens
        {"name": "prompt_b8_t8192", "op": "prompt", "n": 8, "longest": 8192, "hq": 32, "hkv": 8, "d": 128, "io": "bf16", "lengths": 0},
        # single tokens of three short conversations: latency counts
        {"name": "paged_decode_n3_d64", "op": "paged", "n": 3, "longest": 700, "chunk": 1, "chunks": 0, "hq": 8, "hkv": 2, "d": 64, "page": 16, "io": "bf16", "lengths": 6},
        # the decode batch of the benchmark: 256 requests, one token each
        {"name": "paged_decode_n256", "op": "paged", "n": 256, "longest": 8192, "chunk": 1, "chunks": 0, "hq": 32, "hkv": 8, "d": 128, "page": 64, "io": "bf16", "lengths": 7},
        # four draft tokens of two very long contexts, verified in one pass
        {"name": "paged_draft_long", "op": "paged", "n": 2, "longest": 262147, "chunk": 4, "chunks": 2, "hq": 32, "hkv": 8, "d": 128, "page": 128, "io": "bf16", "lengths": 0},
        # a mixed step: two prompts' chunks over their caches among single tokens
        {"name": "paged_mixed_n33", "op": "paged", "n": 33, "longest": 16384, "chunk": 2048, "chunks": 2, "hq": 32, "hkv": 4, "d": 128, "page": 32, "io": "bf16", "lengths": 8},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["plan", "append", "prompt", "paged"])
    while True:
        page = rng.choice([16, 32, 64, 128])
        hkv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        d = rng.choice([64, 128])
        io = rng.choice(["bf16", "bf16", "bf16", "f32"])
        seed = rng.randrange(1, 1 << 30)
        if op == "plan":
            c = {"op": op, "n": _log_int(rng, 1, 2048), "page": page, "longest": _log_int(rng, 64, 32768),
                 "chunk": _log_int(rng, 1, 2048), "lengths": seed}
        elif op == "append":
            c = {"op": op, "tokens": _log_int(rng, 1, 65536), "hkv": hkv, "d": d, "page": page, "io": io}
        elif op == "prompt":
            c = {"op": op, "n": _log_int(rng, 1, 32), "longest": _log_int(rng, 1, 1021 if io == "f32" else 8192),
                 "hq": hkv * group, "hkv": hkv, "d": d, "io": io, "lengths": seed}
        else:
            n = _log_int(rng, 1, 256)
            c = {"op": op, "n": n, "longest": _log_int(rng, 1, 4099 if io == "f32" else 65536),
                 "chunk": _log_int(rng, 1, 64 if io == "f32" else 2048), "chunks": rng.choice([0, 1, min(n, 2), n]),
                 "hq": hkv * group, "hkv": hkv, "d": d, "page": page, "io": io, "lengths": seed}
        w = work(c)
        if 3072 in c.values() or (c.get("hq", 0) + 2 * c.get("hkv", 0)) * d == 3072:
            continue
        # no dearer than the largest listed cases, for either form
        if w["bytes"] <= 5e9 and w["flops"] <= (3e10 if io == "f32" else 2e12) and _padded(c) <= 8e11:
            return c


def _lengths(case):
    """(old, new) lengths per request, or prompt lengths: by the case alone."""
    rng = random.Random(case["lengths"])
    n, longest = case["n"], case["longest"]
    if case["op"] == "prompt":
        if case["lengths"] == 0:
            return [longest] * n
        return [longest if i == 0 else max(0, _log_int(rng, 1, longest) - rng.choice([0, 0, 0, 1])) for i in range(n)]
    if case["op"] == "paged":
        kv = [longest - 5 * i if case["lengths"] == 0 else longest if i == 0 else rng.randint(1, longest) for i in range(n)]
        kv = [max(1, x) for x in kv]
        q = [1] * n
        for i in range(case["chunks"]):
            q[i] = case["chunk"] if i % 2 == 0 or case["lengths"] == 0 else rng.randint(1, case["chunk"])
        return [min(a, b) for a, b in zip(q, kv)], kv
    old, new = [], []
    for _ in range(n):
        x = rng.randint(0, longest)
        kind = rng.random() if case["chunk"] > 1 else 1.0
        if kind < 0.1:  # a prompt's chunk
            y = min(longest, x + rng.randint(1, case["chunk"]))
        elif kind < 0.2:  # drafts taken back
            y = max(0, x - rng.randint(1, 8))
        elif kind < 0.25:  # the request ends
            y = 0
        else:
            y = min(longest, x + 1)
        old.append(x)
        new.append(y)
    return old, new


def _ceil(a, b):
    return -(-a // b)


def _padded(case):
    """Score elements x d that the plain form computes."""
    if case["op"] == "prompt":
        return sum(x * x for x in _lengths(case)) * case["hq"] * case["d"]
    if case["op"] == "paged":
        q, kv = _lengths(case)
        return max(q) * sum(kv) * case["hq"] * case["d"] if max(q) * max(kv) * case["n"] * case["hq"] <= SCORES else \
            sum(a * b for a, b in zip(q, kv)) * case["hq"] * case["d"]
    return 0


def work(case):
    if case["op"] == "plan":
        old, new = _lengths(case)
        grown = sum(max(0, b - a) for a, b in zip(old, new))
        pages = sum(abs(_ceil(b, case["page"]) - _ceil(a, case["page"])) for a, b in zip(old, new))
        # two lengths in, one length and one offset out; a page id read and written; a slot written
        return {"bytes": 16 * case["n"] + 8 * pages + 4 * grown + 20, "flops": 0}
    es = 2 if case["io"] == "bf16" else 4
    if case["op"] == "append":
        return {"bytes": case["tokens"] * (4 + 4 * case["hkv"] * case["d"] * es), "flops": 0}
    if case["op"] == "prompt":
        lens = _lengths(case)
        row = case["hq"] * case["d"] * es
        pairs = sum(x * (x + 1) // 2 for x in lens)
        return {"bytes": sum(lens) * (2 * row + 2 * case["hkv"] * case["d"] * es + 4 * case["hq"]) + 4 * len(lens) + 4,
                "flops": 4 * pairs * case["hq"] * case["d"]}
    q, kv = _lengths(case)
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, kv))
    return {"bytes": sum(q) * (2 * case["hq"] * case["d"] * es + 4 * case["hq"]) + sum(kv) * 2 * case["hkv"] * case["d"] * es
            + sum(4 * _ceil(x, case["page"]) for x in kv) + 8 * case["n"] + 4, "flops": 4 * pairs * case["hq"] * case["d"]}


# --------------------------------------------------------------------------- inputs
def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _randn(gen, shape, dtype, std=1.0):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEV).mul_(std))
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": case, "op": case["op"]}
    if case["op"] == "plan":
        old, new = _lengths(case)
        n, page = case["n"], case["page"]
        max_pages = _ceil(case["longest"], page) + 1
        held = [_ceil(x, page) for x in old]
        grow = sum(max(0, _ceil(b, page) - h) for b, h in zip(new, held))
        free = grow + 17  # pages to spare
        pages = sum(held) + free
        perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        first = torch.zeros(n + 1, dtype=torch.int64)
        first[1:] = torch.cumsum(torch.tensor(held), 0)
        col = torch.arange(max_pages, device=DEV)
        at = first[:-1].to(DEV)[:, None] + col[None, :]
        table = torch.where(col[None, :] < _ints(held)[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32)
        head = int(seed) % pages
        ring = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        ring[(head + torch.arange(free, device=DEV)) % pages] = perm[sum(held):]
        tokens = sum(max(0, b - a) for a, b in zip(old, new))
        # room for a few tokens more than this step has, as a fixed-size step keeps
        s.update(old=_ints(old), new=_ints(new), table=table, ring=ring, at=_ints([head, free]), page=page, room=tokens + 8)
        return s
    dt, hkv, d = DTYPES[case["io"]], case["hkv"], case["d"]
    if case["op"] == "append":
        t, page = case["tokens"], case["page"]
        pages = _ceil(t + t // 4, page) + 1
        # every token's slot: whole pages in any order, and each 64th token has none
        order = torch.randperm(pages, generator=gen, device=DEV)
        i = torch.arange(t, device=DEV)
        slot = order[i // page] * page + i % page
        slot = torch.where(i % 64 == 63, -1, slot).to(torch.int32)
        qkv = _randn(gen, (t, 4 * hkv, d), dt)  # the fused projection, two query heads to a key head
        s.update(k=qkv[:, 2 * hkv:3 * hkv], v=qkv[:, 3 * hkv:], slot=slot, live=i[i % 64 != 63], kc=_randn(gen, (pages, hkv, page, d), dt),
                 vc=_randn(gen, (pages, hkv, page, d), dt))
        return s
    hq = case["hq"]
    s["scale"] = d ** -0.5
    if case["op"] == "prompt":
        lens = _lengths(case)
        total = sum(lens)
        qkv = _randn(gen, (total, hq + 2 * hkv, d), dt)
        qkv[:, :hq] *= 1.5  # scores with a spread of 1.5
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], q_lens=lens, kv_lens=lens, most=max(lens))
    else:
        q, kv = _lengths(case)
        page = case["page"]
        held = [_ceil(x, page) for x in kv]
        pages = sum(held) + 3
        perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
        first = [0]
        for h in held:
            first.append(first[-1] + h)
        col = torch.arange(max(held) + 1, device=DEV)
        at = _ints(first[:-1])[:, None] + col[None, :]
        table = torch.where(col[None, :] < _ints(held)[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32)
        kc, vc = (_randn(gen, (pages, hkv, page, d), dt) for _ in range(2))
        # what was never written holds anything at all
        used = torch.zeros(pages, dtype=torch.int64, device=DEV)
        fill = torch.tensor([min(page, x - j * page) for x, h in zip(kv, held) for j in range(h)], device=DEV)
        used[perm[:sum(held)].long()] = fill
        stale = torch.arange(page, device=DEV)[None, :] >= used[:, None]
        p, r = stale.nonzero(as_tuple=True)
        kc[p, :, r] = float("nan")
        vc[p, :, r] = float("nan")
        s.update(q=_randn(gen, (sum(q), hq, d), dt, 1.5), kc=kc, vc=vc, table=table, q_lens=q, kv_lens=kv, kv_len=_ints(kv), most=max(q))
    cu = [0]
    for x in s["q_lens"]:
        cu.append(cu[-1] + x)
    s.update(cu=_ints(cu), starts=cu)
    return s


# --------------------------------------------------------------------------- the operators
def run(s):
    if own:
        return _framework(s)
    return {"plan": _plan, "append": _append, "prompt": _attend, "paged": _attend}[s["op"]](s)


def _framework(s):
    from gated_delta_rule_57_gb300 import kda
    if s["op"] == "plan":
        kv_len, cu, slot, ring_at = kda.kda_kv_plan(s["old"], s["new"], s["table"], s["ring"], s["at"], page_size=s["page"],
                                                    max_tokens=s["room"])
        return {"kv_len": kv_len, "cu": cu, "slot": slot, "table": s["table"], "ring": s["ring"], "ring_at": ring_at}
    if s["op"] == "append":
        kda.kda_kv_append(s["k"], s["v"], s["slot"], s["kc"], s["vc"])
        return {"kc": s["kc"], "vc": s["vc"]}
    if s["op"] == "prompt":
        o, lse = kda.kda_attn_prompt(s["q"], s["k"], s["v"], s["cu"], max_len=s["most"], scale=s["scale"])
    else:
        o, lse = kda.kda_attn_paged(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv_len"], max_q=s["most"], scale=s["scale"])
    return {"o": o, "lse": lse}


def _plan(s):
    """A request grows from old to new tokens and takes pages from the head of
    the ring of free pages, in the requests' order, or shrinks and gives the
    pages it no longer needs back at the ring's end. It is left as it was where
    the free pages, its table row or the room for tokens run out."""
    old, new, table, ring, page = s["old"].long(), s["new"].long(), s["table"], s["ring"], s["page"]
    pages, max_pages = ring.numel(), table.shape[1]
    head, count = s["at"].long().unbind()
    held, want, q = (old + page - 1) // page, (new + page - 1) // page, (new - old).clamp(min=0)
    fits = want <= max_pages
    grow = torch.where(fits, (want - held).clamp(min=0), 0)
    gi, ti = torch.cumsum(grow, 0), torch.cumsum(q, 0)
    ok = fits & ((grow == 0) | (gi <= count)) & ((q == 0) | (ti <= s["room"]))
    back = torch.where(ok, (held - want).clamp(min=0), 0)
    bi = torch.cumsum(back, 0)
    col = torch.arange(max_pages, device=DEV)[None, :]
    take = ok[:, None] & (col >= held[:, None]) & (col < want[:, None])
    from_ring = ring[(head + (gi - grow)[:, None] + col - held[:, None]) % pages]
    table = torch.where(take, from_ring, table)
    give = ok[:, None] & (col >= want[:, None]) & (col < held[:, None])
    to = torch.where(give, (head + count + (bi - back)[:, None] + col - want[:, None]) % pages, pages)
    ring = torch.cat([ring, ring[:1]]).scatter(0, to.flatten(), table.flatten())[:pages]
    cu = torch.cat([ti[:1] * 0, ti]).to(torch.int32)
    t = torch.arange(s["room"], device=DEV)
    r = torch.searchsorted(ti, t, right=True)
    live = r < old.numel()
    r = r.clamp(max=old.numel() - 1)
    at = (old[r] + t - (ti - q)[r]).clamp(max=max_pages * page - 1)
    slot = torch.where(live & ok[r], table[r, at // page] * page + at % page, -1).to(torch.int32)
    taken = torch.where(ok, grow, 0).sum()
    ring_at = torch.stack([(head + taken) % pages, count - taken + back.sum()]).to(torch.int32)
    return {"kv_len": torch.where(ok, new, old).to(torch.int32), "cu": cu, "slot": slot, "table": table, "ring": ring, "ring_at": ring_at}


def _append(s):
    page, live = s["kc"].shape[2], s["live"]
    slot = s["slot"][live].long()
    s["kc"][slot // page, :, slot % page] = s["k"][live]
    s["vc"][slot // page, :, slot % page] = s["v"][live]
    return {"kc": s["kc"], "vc": s["vc"]}


def _groups(s):
    """Runs of requests whose padded scores fit, as (first, last + 1, padded new tokens, padded keys)."""
    hq, out, a = s["q"].shape[1], [], 0
    for b in range(1, len(s["q_lens"]) + 1):
        most = lambda to: max(s["q_lens"][a:to]) * max(s["kv_lens"][a:to]) * (to - a) * hq  # noqa: E731
        if b == len(s["q_lens"]) or most(b + 1) > SCORES:
            out.append((a, b, max(s["q_lens"][a:b]), max(s["kv_lens"][a:b])))
            a = b
    return [g for g in out if g[2] > 0]


def _attend(s):
    """softmax(scale q k^T) v over the keys at or before each token, the new
    tokens being the last of their request's; also the log of the softmax's sum."""
    total, hq, d = s["q"].shape
    hkv = s["kc"].shape[1] if "kc" in s else s["k"].shape[1]
    o = torch.empty((total + 1, hq, d), dtype=s["q"].dtype, device=DEV)  # the last row takes what pads
    lse = torch.empty((total + 1, hq), dtype=torch.float32, device=DEV)
    cu = s["cu"].long()
    for a, b, nq, nk in _groups(s):
        i, j = torch.arange(nq, device=DEV), torch.arange(nk, device=DEV)
        ql = (cu[a + 1:b + 1] - cu[a:b])[:, None]
        kl = s["kv_len"].long()[a:b, None] if "kc" in s else ql
        rows = cu[a:b, None] + i
        q = s["q"][rows.clamp(max=total - 1)].float()  # [n, nq, hq, d]
        if "kc" in s:
            page = s["kc"].shape[2]
            p = s["table"].long()[a:b][:, j // page].clamp(min=0)
            k, v = (c.transpose(1, 2)[p, j % page].float() for c in (s["kc"], s["vc"]))
        else:
            at = (cu[a:b, None] + j).clamp(max=total - 1)
            k, v = s["k"][at].float(), s["v"][at].float()
        there = (j < kl)[:, :, None, None]
        k, v = torch.where(there, k, 0), torch.where(there, v, 0)
        q = q.unflatten(2, (hkv, hq // hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [n, hkv, g nq, d]
        x = (q @ k.permute(0, 2, 3, 1)).mul_(s["scale"]).unflatten(2, (hq // hkv, nq))
        seen = (j <= (kl - ql + i)[:, :, None])[:, None, None]
        x.masked_fill_(~seen, -math.inf)
        m = x.amax(-1, keepdim=True).clamp(min=-3e38)
        x = x.sub_(m).exp_()
        z = x.sum(-1)
        y = x.flatten(2, 3) @ v.transpose(1, 2)
        y = y.unflatten(2, (hq // hkv, nq)) / z[..., None].clamp(min=1e-37)
        rows = torch.where(i < ql, rows, total)
        o[rows] = y.permute(0, 3, 1, 2, 4).flatten(2, 3).to(o.dtype)
        lse[rows] = (m[..., 0] + z.log()).permute(0, 3, 1, 2).flatten(2, 3)
    return {"o": o[:total], "lse": lse[:total]}


# --------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _plan_one_by_one(s)
    if case["op"] == "append":
        out = {n: s[n].double() for n in ("kc", "vc")}
        page = s["kc"].shape[2]
        slots = s["slot"].tolist()
        kept = [t for t, x in enumerate(slots) if x >= 0]
        p = torch.tensor([slots[t] // page for t in kept], device=DEV, dtype=torch.int64)
        r = torch.tensor([slots[t] % page for t in kept], device=DEV, dtype=torch.int64)
        kept = torch.tensor(kept, device=DEV, dtype=torch.int64)
        out["kc"][p, :, r] = s["k"].double()[kept]
        out["vc"][p, :, r] = s["v"].double()[kept]
        return out
    total, hq, d = s["q"].shape
    o = torch.zeros((total, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((total, hq), dtype=torch.float64, device=DEV)
    for r, (nq, nk) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        if nq == 0:
            continue
        t0 = s["starts"][r]
        if "kc" in s:
            ids = s["table"][r, :_ceil(nk, case["page"])].long()
            k, v = (s[c][ids].permute(0, 2, 1, 3).flatten(0, 1)[:nk].double() for c in ("kc", "vc"))
        else:
            k, v = s["k"][t0:t0 + nk].double(), s["v"][t0:t0 + nk].double()
        step = max(1, (1 << 28) // (hq * nk))
        for a in range(0, nq, step):
            b = min(nq, a + step)
            last = nk - nq + b  # keys that any of these tokens sees
            for h in range(case["hkv"]):
                g = slice(h * (hq // case["hkv"]), (h + 1) * (hq // case["hkv"]))
                x = torch.einsum("tgd,jd->gtj", s["q"][t0 + a:t0 + b, g].double(), k[:last, h]) * s["scale"]
                hidden = torch.arange(last, device=DEV)[None, :] > (nk - nq + torch.arange(a, b, device=DEV))[:, None]
                x = x.masked_fill(hidden, -math.inf)
                l = torch.logsumexp(x, -1)
                o[t0 + a:t0 + b, g] = torch.einsum("gtj,jd->tgd", torch.exp(x - l[..., None]), v[:last, h])
                lse[t0 + a:t0 + b, g] = l.t()
    return {"o": o, "lse": lse}


def _plan_one_by_one(s):
    """The definition, one request after another."""
    old, new, table, ring = s["old"].tolist(), s["new"].tolist(), s["table"].tolist(), s["ring"].tolist()
    head, count = s["at"].tolist()
    page, pages = s["page"], len(ring)
    taken, given, cu, slot, kv = 0, 0, [0], [-1] * s["room"], []
    for r, (a, b) in enumerate(zip(old, new)):
        held, want = _ceil(a, page), _ceil(b, page)
        cu.append(cu[-1] + max(0, b - a))
        refused = want > len(table[r]) or (want > held and taken + want - held > count) or (b > a and cu[-1] > s["room"])
        kv.append(a if refused else b)
        if refused:
            continue
        for j in range(held, want):
            table[r][j] = ring[(head + taken) % pages]
            taken += 1
        for j in range(want, held):
            ring[(head + count + given) % pages] = table[r][j]
            given += 1
        for i in range(b - a):
            slot[cu[r] + i] = table[r][(a + i) // page] * page + (a + i) % page
    return {"kv_len": _ints(kv), "cu": _ints(cu), "slot": _ints(slot), "table": _ints(table), "ring": _ints(ring),
            "ring_at": _ints([(head + taken) % pages, count - taken + given])}
