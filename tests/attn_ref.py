"""64-bit definitions of the paged-cache and attention operators, one request
and one head at a time, and the error they allow.

Tolerances. With u = 2^-8 (half a unit in the last place of bf16: its significand
has 8 bits, so rounding moves x by at most 2^-8 |x|), rounding the
probabilities p_j moves an output by at most u A, A = sum_j p_j |v_j|, and
rounding the output by at most u (|o| + u A). What is left is fp32: a score
x = scale q . k carries a relative error of a few sqrt(d) 2^-24 of
scale sum_c |q_c k_c| (below 40 for the inputs drawn here), i.e. at most about
3e-5, which is a relative error of the same size on p_j; sums over n keys add
sqrt(n) 2^-24. 1e-4 A covers both.
    bf16: |o - ref| <= 1.01 u (A + |ref|) + 1e-4 A
    fp32: |o - ref| <= 1e-4 A
    lse:  |lse - ref| <= 1e-4 (the same score error; |lse| < 50 adds 50 2^-24)
"""
import math

import torch

U = 2.0 ** -8


def attend(q, k, v, kv_len, scale):
    """One request: q [n, Hq, d], k, v [kv_len, Hkv, d]; o, lse and A in 64 bits."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    o = torch.zeros(n, hq, d, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    if n == 0 or kv_len == 0:
        return o, lse, a
    j = torch.arange(kv_len, device=q.device)
    sees = j[None, :] <= kv_len - n + torch.arange(n, device=q.device)[:, None]
    rows = sees.any(1)
    for h in range(hq):
        kh, vh = k[:, h // g].double(), v[:, h // g].double()
        x = (q[:, h].double() @ kh.t()) * scale
        x = torch.where(sees, x, -math.inf)
        lse[rows, h] = torch.logsumexp(x[rows], 1)
        p = torch.zeros_like(x)
        p[rows] = torch.exp(x[rows] - lse[rows, h][:, None])
        o[:, h] = p @ vh
        a[:, h] = p @ vh.abs()
    return o, lse, a


def prompt(q, k, v, lens, scale):
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    t = 0
    for n in lens:
        o[t:t + n], lse[t:t + n], a[t:t + n] = attend(q[t:t + n], k[t:t + n], v[t:t + n], n, scale)
        t += n
    return o, lse, a


def gather(cache, table_row, kv_len):
    """The first kv_len tokens of a request: [kv_len, Hkv, d]."""
    page = cache.shape[2]
    ids = table_row[:-(-kv_len // page)].long()
    return cache[ids].permute(0, 2, 1, 3).flatten(0, 1)[:kv_len]


def paged(q, kc, vc, table, q_lens, kv_lens, scale):
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    t = 0
    for r, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        o[t:t + n], lse[t:t + n], a[t:t + n] = attend(
            q[t:t + n], gather(kc, table[r], kv), gather(vc, table[r], kv), kv, scale)
        t += n
    return o, lse, a


def check(o, lse, ref):
    ro, rl, a = ref
    assert torch.isfinite(o).all()
    tol = 1e-4 * a + (1.01 * U * (a + ro.abs()) if o.dtype == torch.bfloat16 else 0)
    over = (o.double() - ro).abs() - tol
    assert (over <= 0).all(), f"o off by {float(over.max()):.3e} over its bound"
    if lse is not None:
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
        d = (lse.double() - rl)[~empty].abs()
        assert d.numel() == 0 or float(d.max()) <= 1e-4, f"lse off by {float(d.max()):.3e}"


def plan(old, new, table, ring, at, page, room):
    """The plan of a step, one request after another, on Python lists.
    Returns kv, cu, slot, table, ring, ring_at and whether one was refused."""
    table, ring = [list(r) for r in table], list(ring)
    (head, count), pages = at, len(ring)
    need = taken = given = 0
    cu, slot, kv, short = [0], [-1] * room, [], False
    for r, (a, b) in enumerate(zip(old, new)):
        held, want = -(-a // page), -(-b // page)
        cu.append(cu[-1] + max(0, b - a))
        if held < want <= len(table[r]):
            need += want - held
        if want > len(table[r]) or (want > held and need > count) or (b > a and cu[-1] > room):
            kv.append(a)
            short = True
            continue
        kv.append(b)
        for j in range(held, want):
            table[r][j] = ring[(head + taken) % pages]
            taken += 1
        for j in range(want, held):
            ring[(head + count + given) % pages] = table[r][j]
            given += 1
        for i in range(b - a):
            slot[cu[r] + i] = table[r][(a + i) // page] * page + (a + i) % page
    return kv, cu, slot, table, ring, [(head + taken) % pages, count - taken + given], short
