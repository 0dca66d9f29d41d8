"""Measured cases of the latent-attention and rotated-append operators.

An attention layer of a hybrid stack may keep, instead of keys and values per
head, one latent vector a token from which every head's keys and values come
(and a short key part that all heads share and that carries the position). Its
operators, and the rotation by position for layers that keep plain keys:

  rope           queries and keys rotated by position, keys and values written
                 to the paged cache
  latent_append  a token's latent and its rotated key part written to the paged
                 latent cache, its queries' part rotated
  latent_prompt  causal attention over packed prompts, keys and values of each
                 head expanded from the latent (the key part shared by all heads)
  latent_paged   causal attention of new tokens over the paged latent cache, the
                 expansion absorbed into queries and outputs: every head's keys
                 are the cached rows, its values their first 512 channels

Each has a plain form below (elementary torch operations in 32 bits, angles in
64) and its call through the package. Layouts: q [T, H, d], caches [pages, heads,
page, d], latent caches [pages, page, 512 + rope].
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SCORES = 1 << 31  # largest score tensor of the plain form, in elements
LATENT, NOPE, HEAD_V = 512, 128, 128


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one token each of a decode batch, rotated on its way to the cache: latency counts
        {"name": "rope_decode_t256", "op": "rope", "tokens": 256, "run": 1, "far": 8192, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "pairs": "halves", "page": 64, "io": "bf16"},
        # eight prompts of 8192 tokens
        {"name": "rope_prompt_t65536", "op": "rope", "tokens": 65536, "run": 8192, "far": 8192, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "pairs": "halves", "page": 64, "io": "bf16"},
        # one token each of a decode batch to the latent cache, far along in long contexts: latency counts
        {"name": "latent_append_decode_t256", "op": "latent_append", "tokens": 256, "run": 1, "far": 1048576, "hq": 32, "rope": 64,
         "pairs": "neighbours", "page": 64, "into": "absorbed", "io": "bf16"},
        # eight prompts of 8192 tokens to the latent cache, whose own attention is over expanded heads
        {"name": "latent_append_prompt_t65536", "op": "latent_append", "tokens": 65536, "run": 8192, "far": 8192, "hq": 32, "rope": 64,
         "pairs": "neighbours", "page": 64, "into": "expanded", "io": "bf16"},
        # a handful of short prompts on a small model: latency counts
        {"name": "latent_prompt_short_h4", "op": "latent_prompt", "n": 5, "longest": 255, "hq": 4, "rope": 64, "io": "bf16", "lengths": 3},
        # the accuracy path, in 32 bits
        {"name": "latent_prompt_f32_h8", "op": "latent_prompt", "n": 3, "longest": 1021, "hq": 8, "rope": 64, "io": "f32", "lengths": 4},
        # a packed batch of prompts of very different lengths
        {"name": "latent_prompt_ragged_n24", "op": "latent_prompt", "n": 24, "longest": 4096, "hq": 32, "rope": 64, "io": "bf16", "lengths": 5},
        # a prefill batch of long prompts
        {"name": "latent_prompt_n4_t8192", "op": "latent_prompt", "n": 4, "longest": 8192, "hq": 32, "rope": 64, "io": "bf16", "lengths": 0},
        # single tokens of three short conversations on a small model: latency counts
        {"name": "latent_paged_n3_h8", "op": "latent_paged", "n": 3, "longest": 700, "chunk": 1, "chunks": 0, "hq": 8, "rope": 64, "page": 16,
         "io": "bf16", "lengths": 6},
        # a decode batch: 256 requests, one token each
        {"name": "latent_paged_decode_n256", "op": "latent_paged", "n": 256, "longest": 8192, "chunk": 1, "chunks": 0, "hq": 32, "rope": 64,
         "page": 64, "io": "bf16", "lengths": 7},
        # four draft tokens of two very long contexts, verified in one pass
        {"name": "latent_paged_draft_long", "op": "latent_paged", "n": 2, "longest": 262147, "chunk": 4, "chunks": 2, "hq": 32, "rope": 64,
         "page": 128, "io": "bf16", "lengths": 0},
        # a mixed step of a layer without positions, in 32 bits: two chunks of prompts among single tokens
        {"name": "latent_paged_mixed_f32", "op": "latent_paged", "n": 9, "longest": 2049, "chunk": 33, "chunks": 2, "hq": 8, "rope": 0, "page": 32,
         "io": "f32", "lengths": 8},
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "latent_append", "latent_prompt", "latent_prompt", "latent_paged", "latent_paged"])
    while True:
        page = rng.choice([16, 32, 64, 128])
        io = rng.choice(["bf16", "bf16", "bf16", "f32"])
        heads = rng.choice([1, 2, 3, 5, 8, 10, 32, 40, 64])
        rope = rng.choice([64, 64, 0])
        pairs = rng.choice(["halves", "neighbours"])
        seed = rng.randrange(1, 1 << 30)
        tokens = _log_int(rng, 1, 65536)
        run = rng.choice([1, min(tokens, 4), tokens])
        far = _log_int(rng, max(run, 64), 1 << 20)
        if op == "rope":
            hkv, d = rng.choice([1, 2, 3, 5, 8]), rng.choice([64, 128])
            c = {"op": op, "tokens": tokens, "run": run, "far": far, "hq": hkv * rng.choice([2, 3, 5, 7]), "hkv": hkv, "d": d,
                 "rot": rng.choice([d, d, d // 2, 16, 48]), "pairs": pairs, "page": page, "io": io}
        elif op == "latent_append":
            c = {"op": op, "tokens": tokens, "run": run, "far": far, "hq": heads, "rope": rope, "pairs": pairs, "page": page,
                 "into": rng.choice(["absorbed", "expanded"]), "io": io}
        elif op == "latent_prompt":
            c = {"op": op, "n": _log_int(rng, 1, 32), "longest": _log_int(rng, 1, 1021 if io == "f32" else 8192), "hq": heads,
                 "rope": rope, "io": io, "lengths": seed}
        else:
            n = _log_int(rng, 1, 256)
            c = {"op": op, "n": n, "longest": _log_int(rng, 1, 4099 if io == "f32" else 65536),
                 "chunk": _log_int(rng, 1, 33 if io == "f32" else 512), "chunks": rng.choice([0, 0, 1, min(n, 2), n]),
                 "hq": heads, "rope": rope, "page": page, "io": io, "lengths": seed}
        w = work(c)
        # no dearer than the largest listed cases, for either form
        if w["bytes"] <= 1.7e9 and w["flops"] <= (1.1e10 if io == "f32" else 2e12) and _padded(c) <= 1.5e12:
            return c


def _lengths(case):
    """(new tokens, keys) per request, or prompt lengths: by the case alone."""
    rng = random.Random(case["lengths"])
    n, longest = case["n"], case["longest"]
    if case["op"] == "latent_prompt":
        if case["lengths"] == 0:
            return [longest] * n
        return [longest if i == 0 else max(0, _log_int(rng, 1, longest) - rng.choice([0, 0, 0, 1])) for i in range(n)]
    kv = [longest - 5 * i if case["lengths"] == 0 else longest if i == 0 else rng.randint(1, longest) for i in range(n)]
    kv = [max(1, x) for x in kv]
    q = [1] * n
    for i in range(case["chunks"]):
        q[i] = case["chunk"] if i % 2 == 0 or case["lengths"] == 0 else rng.randint(1, case["chunk"])
    return [min(a, b) for a, b in zip(q, kv)], kv


def _ceil(a, b):
    return -(-a // b)


def _padded(case):
    """Score elements x channels that the plain form computes."""
    if case["op"] == "latent_prompt":
        return sum(x * x for x in _lengths(case)) * case["hq"] * (NOPE + case["rope"] + HEAD_V)
    if case["op"] == "latent_paged":
        q, kv = _lengths(case)
        d = 2 * LATENT + case["rope"]
        return max(q) * sum(kv) * case["hq"] * d if max(q) * max(kv) * case["n"] * case["hq"] <= SCORES else \
            sum(a * b for a, b in zip(q, kv)) * case["hq"] * d
    return 0


def work(case):
    es = 2 if case["io"] == "bf16" else 4
    if case["op"] == "rope":
        t, d = case["tokens"], case["d"]
        # a slot and a position; queries, keys and values read and written; the frequencies
        return {"bytes": t * (8 + 2 * (case["hq"] + 2 * case["hkv"]) * d * es) + 4 * case["rot"],
                "flops": 3 * t * (case["hq"] + case["hkv"]) * case["rot"]}
    if case["op"] == "latent_append":
        t, r = case["tokens"], case["rope"]
        copies = 2 if case["into"] == "absorbed" else 3  # the rotated key part once more, for the prompt's attention
        return {"bytes": t * (4 + 2 * LATENT * es + (4 + 2 * case["hq"] * r * es + copies * r * es if r else 0)) + 4 * r,
                "flops": 3 * t * (case["hq"] + 1) * r}
    h, r = case["hq"], case["rope"]
    if case["op"] == "latent_prompt":
        lens = _lengths(case)
        pairs = sum(x * (x + 1) // 2 for x in lens)
        return {"bytes": sum(lens) * (h * (2 * NOPE + r + 2 * HEAD_V) * es + r * es + 4 * h) + 4 * len(lens) + 4,
                "flops": 2 * pairs * h * (NOPE + r + HEAD_V)}
    q, kv = _lengths(case)
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, kv))
    return {"bytes": sum(q) * (h * (2 * LATENT + r) * es + 4 * h) + sum(kv) * (LATENT + r) * es
            + sum(4 * _ceil(x, case["page"]) for x in kv) + 8 * case["n"] + 4, "flops": 2 * pairs * h * (2 * LATENT + r)}


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


def _frequencies(rot):
    """Radians a token of each pair of channels."""
    return torch.tensor([10000.0 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64)


def _positions(case, gen):
    """Runs of consecutive positions, one a request, at random starts."""
    t, run = case["tokens"], case["run"]
    starts = torch.randint(0, case["far"] - run + 1, (_ceil(t, run),), generator=gen, device=DEV)
    i = torch.arange(t, device=DEV)
    return (starts[i // run] + i % run).to(torch.int32)


def _slots(t, page, gen):
    """Every token's slot: whole pages in any order; each 64th token has none."""
    pages = _ceil(t + t // 4, page) + 1
    order = torch.randperm(pages, generator=gen, device=DEV)
    i = torch.arange(t, device=DEV)
    slot = order[i // page] * page + i % page
    return pages, torch.where(i % 64 == 63, -1, slot).to(torch.int32), i[i % 64 != 63]


def _paged(s, q, kv, page, gen):
    """A block table of pages in any order, and which slots were never written."""
    held = [_ceil(x, page) for x in kv]
    pages = sum(held) + 3
    perm = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    first = [0]
    for h in held:
        first.append(first[-1] + h)
    col = torch.arange(max(held) + 1, device=DEV)
    at = _ints(first[:-1])[:, None] + col[None, :]
    s["table"] = torch.where(col[None, :] < _ints(held)[:, None], perm[at.clamp(max=pages - 1)], -1).to(torch.int32)
    used = torch.zeros(pages, dtype=torch.int64, device=DEV)
    used[perm[:sum(held)].long()] = torch.tensor([min(page, x - j * page) for x, h in zip(kv, held) for j in range(h)], device=DEV)
    s.update(q_lens=q, kv_lens=kv, kv_len=_ints(kv), most=max(q))
    return pages, (torch.arange(page, device=DEV)[None, :] >= used[:, None]).nonzero(as_tuple=True)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": case, "op": case["op"]}
    dt = DTYPES[case["io"]]
    if case["op"] in ("rope", "latent_append"):
        t, page = case["tokens"], case["page"]
        pages, slot, live = _slots(t, page, gen)
        rot = case["rot"] if case["op"] == "rope" else case["rope"]
        freq = _frequencies(rot)
        s.update(slot=slot, live=live, pos=_positions(case, gen), freq=freq.to(DEV), rot=rot, neighbours=case["pairs"] == "neighbours")
        if own and rot:
            from gated_delta_rule_57_gb300 import kda
            s["turns"] = kda.kda_rope_turns(freq, device=DEV)
        if case["op"] == "rope":
            hq, hkv, d = case["hq"], case["hkv"], case["d"]
            qkv = _randn(gen, (t, hq + 2 * hkv, d), dt)  # the fused projection
            s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], kc=_randn(gen, (pages, hkv, page, d), dt),
                     vc=_randn(gen, (pages, hkv, page, d), dt))
            return s
        h = case["hq"]
        down = _randn(gen, (t, LATENT + rot), dt)  # the projection to latent and shared key part
        s.update(c=down[:, :LATENT], kr=down[:, LATENT:] if rot else None, cache=_randn(gen, (pages, page, LATENT + rot), dt),
                 qr=None, q_out=None, k_out=None)
        if rot:
            s["qr"] = _randn(gen, (t, h, NOPE + rot), dt)[..., NOPE:]
            # where the rotated parts go: beside the absorbed queries, or beside the expanded ones and the expanded keys
            left = LATENT if case["into"] == "absorbed" else NOPE
            s["q_out"] = torch.zeros((t, h, left + rot), dtype=dt, device=DEV)[..., left:]
            if case["into"] == "expanded":
                s["k_out"] = torch.zeros((t, rot), dtype=dt, device=DEV)
        return s
    h, r = case["hq"], case["rope"]
    s["scale"] = (NOPE + r) ** -0.5
    if case["op"] == "latent_prompt":
        lens = _lengths(case)
        total = sum(lens)
        kv = _randn(gen, (total, h, NOPE + HEAD_V), dt)  # the latent expanded by one product
        s.update(q=_randn(gen, (total, h, NOPE + r), dt, 1.5), k=kv[..., :NOPE], v=kv[..., NOPE:], kr=_randn(gen, (total, r), dt) if r else None,
                 q_lens=lens, kv_lens=lens, most=max(lens))
    else:
        q, kv = _lengths(case)
        pages, stale = _paged(s, q, kv, case["page"], gen)
        s["cache"] = _randn(gen, (pages, case["page"], LATENT + r), dt)
        s["cache"][stale] = float("nan")  # what was never written holds anything at all
        s["q"] = _randn(gen, (sum(q), h, LATENT + r), dt)
    cu = [0]
    for x in s["q_lens"]:
        cu.append(cu[-1] + x)
    s.update(cu=_ints(cu), starts=cu)
    return s


# --------------------------------------------------------------------------- the operators
def run(s):
    if own:
        return _framework(s)
    return {"rope": _rope, "latent_append": _latent_append, "latent_prompt": _attend, "latent_paged": _attend}[s["op"]](s)


def _framework(s):
    from gated_delta_rule_57_gb300 import kda
    if s["op"] == "rope":
        q = kda.kda_kv_append_rope(s["q"], s["k"], s["v"], s["slot"], s["pos"], s["turns"], s["kc"], s["vc"], neighbours=s["neighbours"])
        return {"q": q, "kc": s["kc"], "vc": s["vc"]}
    if s["op"] == "latent_append":
        kda.kda_latent_append(s["c"], s["kr"], s["slot"], s["cache"], positions=s["pos"] if s["rot"] else None, turns=s.get("turns"),
                              q_r=s["qr"], q_out=s["q_out"], k_out=s["k_out"], neighbours=s["neighbours"])
        return {n: s[n] for n in ("cache", "q_out", "k_out") if s[n] is not None}
    if s["op"] == "latent_prompt":
        o, lse = kda.kda_attn_latent_prompt(s["q"], s["k"], s["kr"], s["v"], s["cu"], max_len=s["most"], scale=s["scale"])
    else:
        o, lse = kda.kda_attn_latent_paged(s["q"], s["cache"], s["table"], s["cu"], s["kv_len"], max_q=s["most"], scale=s["scale"])
    return {"o": o, "lse": lse}


def _rotate(s, x, angle=None):
    """x [T, H, d]: pairs of its first `rot` channels turned by their angles."""
    if angle is None:
        angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = (f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    y = x.float()
    rot, half = s["rot"], s["rot"] // 2
    a, b = (y[..., :rot:2], y[..., 1:rot:2]) if s["neighbours"] else (y[..., :half], y[..., half:rot])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if s["neighbours"] else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _rope(s):
    page, live = s["kc"].shape[2], s["live"]
    slot = s["slot"][live].long()
    s["kc"][slot // page, :, slot % page] = _rotate(s, s["k"])[live]
    s["vc"][slot // page, :, slot % page] = s["v"][live]
    return {"q": _rotate(s, s["q"]), "kc": s["kc"], "vc": s["vc"]}


def _latent_append(s):
    page, live = s["cache"].shape[1], s["live"]
    slot = s["slot"][live].long()
    row = s["c"]
    if s["rot"]:
        kr = _rotate(s, s["kr"][:, None])[:, 0]
        row = torch.cat([row, kr], -1)
        s["q_out"].copy_(_rotate(s, s["qr"]))
        if s["k_out"] is not None:
            s["k_out"].copy_(kr)
    s["cache"][slot // page, slot % page] = row[live]
    return {n: s[n] for n in ("cache", "q_out", "k_out") if s[n] is not None}


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
    total, hq, _ = s["q"].shape
    paged = "cache" in s
    d = LATENT if paged else HEAD_V
    o = torch.empty((total + 1, hq, d), dtype=s["q"].dtype, device=DEV)  # the last row takes what pads
    lse = torch.empty((total + 1, hq), dtype=torch.float32, device=DEV)
    cu = s["cu"].long()
    for a, b, nq, nk in _groups(s):
        i, j = torch.arange(nq, device=DEV), torch.arange(nk, device=DEV)
        ql = (cu[a + 1:b + 1] - cu[a:b])[:, None]
        kl = s["kv_len"].long()[a:b, None] if paged else ql
        rows = cu[a:b, None] + i
        q = s["q"][rows.clamp(max=total - 1)].float()  # [n, nq, hq, .]
        if paged:
            page = s["cache"].shape[1]
            p = s["table"].long()[a:b][:, j // page].clamp(min=0)
            k = torch.where((j < kl)[:, :, None], s["cache"][p, j % page].float(), 0)
            v = k[..., :LATENT]
            # all heads share the keys: [n, 1, hq nq, .] against [n, 1, nk, .]
            q, k, v = q.transpose(1, 2).flatten(1, 2)[:, None], k[:, None], v[:, None]
        else:
            at = (cu[a:b, None] + j).clamp(max=total - 1)
            k, v = s["k"][at].float(), s["v"][at].float()
            if s["kr"] is not None:
                k = torch.cat([k, s["kr"][at].float()[:, :, None].expand(-1, -1, hq, -1)], -1)
            there = (j < kl)[:, :, None, None]
            k, v = (torch.where(there, x, 0).transpose(1, 2) for x in (k, v))
            q = q.transpose(1, 2)
        x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(b - a, hq, nq, nk)
        x.masked_fill_(~(j <= (kl - ql + i)[:, :, None])[:, None], -math.inf)
        m = x.amax(-1, keepdim=True).clamp(min=-3e38)
        x = x.sub_(m).exp_()
        z = x.sum(-1)
        y = (x.flatten(1, 2)[:, None] if paged else x) @ v
        y = y.view(b - a, hq, nq, d) / z[..., None].clamp(min=1e-37)
        rows = torch.where(i < ql, rows, total)
        o[rows] = y.transpose(1, 2).to(o.dtype)
        lse[rows] = (m[..., 0] + z.log()).transpose(1, 2)
    return {"o": o[:total], "lse": lse[:total]}


# --------------------------------------------------------------------------- 64 bits
def _turned(s, x):
    """Pairs as complex numbers, multiplied by e^{i angle}."""
    rot = s["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), torch.outer(s["pos"].double(), s["freq"]))[:, None]
    y = x.double()
    pair = y[..., :rot].unflatten(-1, (-1, 2)) if s["neighbours"] else y[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
    y[..., :rot] = (z if s["neighbours"] else z.transpose(-1, -2)).flatten(-2)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "latent_append"):
        slots = s["slot"].tolist()
        kept = [t for t, x in enumerate(slots) if x >= 0]
        p, r = (torch.tensor([f(slots[t], case["page"]) for t in kept], device=DEV, dtype=torch.int64) for f in
                (lambda x, n: x // n, lambda x, n: x % n))
        kept = torch.tensor(kept, device=DEV, dtype=torch.int64)
        if case["op"] == "rope":
            out = {n: s[n].double() for n in ("kc", "vc")}
            out["kc"][p, :, r] = _turned(s, s["k"])[kept]
            out["vc"][p, :, r] = s["v"].double()[kept]
            return {"q": _turned(s, s["q"]), **out}
        out = {"cache": s["cache"].double()}
        out["cache"][p, r, :LATENT] = s["c"].double()[kept]
        if s["rot"]:
            kr = _turned(s, s["kr"][:, None])[:, 0]
            out["cache"][p, r, LATENT:] = kr[kept]
            out["q_out"] = _turned(s, s["qr"])
            if s["k_out"] is not None:
                out["k_out"] = kr
        return out
    total, hq, _ = s["q"].shape
    d = LATENT if "cache" in s else HEAD_V
    o = torch.zeros((total, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((total, hq), dtype=torch.float64, device=DEV)
    for n, (nq, nk) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        if nq == 0:
            continue
        t0 = s["starts"][n]
        for h in range(hq):
            if "cache" in s:
                if h == 0:
                    k = s["cache"][s["table"][n, :_ceil(nk, case["page"])].long()].flatten(0, 1)[:nk].double()
                    v = k[:, :LATENT]
            else:
                k, v = s["k"][t0:t0 + nk, h].double(), s["v"][t0:t0 + nk, h].double()
                if s["kr"] is not None:
                    k = torch.cat([k, s["kr"][t0:t0 + nk].double()], -1)
            step = max(1, (1 << 28) // nk)
            for a in range(0, nq, step):
                b = min(nq, a + step)
                last = nk - nq + b  # keys that any of these tokens sees
                x = torch.einsum("td,jd->tj", s["q"][t0 + a:t0 + b, h].double(), k[:last]) * s["scale"]
                hidden = torch.arange(last, device=DEV)[None, :] > (nk - nq + torch.arange(a, b, device=DEV))[:, None]
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                o[t0 + a:t0 + b, h] = torch.exp(x - z[:, None]) @ v[:last]
                lse[t0 + a:t0 + b, h] = z
    return {"o": o, "lse": lse}
