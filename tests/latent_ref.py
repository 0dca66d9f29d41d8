"""64-bit definitions of the rotated appends and of latent attention, and the error
they allow.

Attention: as attn_ref (same roundings, its check() is used), with the scores'
bound scale sum_c |q_c k_c| below 40 for the inputs drawn here too.

Rotation. An angle is off by 1.9e-7 rad at most (a fraction of a turn rounded to fp32,
pi 2^-24), the cos and sin by 2^-22 more (a few units in the last place of fp32), the
two products and their sum by 3 2^-24 of |a| + |b|; together below 6e-7 (|a| + |b|).
Then one rounding to the output's type, half a unit in its last place:
    bf16: |y - ref| <= 2^-8 |ref| + 7e-7 (|a| + |b|)
    fp32: |y - ref| <= 2^-24 |ref| + 7e-7 (|a| + |b|)
"""
import math

import torch

import attn_ref

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def frequencies(rot, base=10000.0):
    return [base ** (-2 * i / rot) for i in range(rot // 2)]


def rotate(x, pos, freq, neighbours):
    """x [T, H, d] rotated in 64 bits, and |a| + |b| of each channel's pair (0 where
    a channel is copied)."""
    rot = 2 * len(freq)
    t = torch.outer(pos.double(), torch.tensor(freq, dtype=torch.float64, device=x.device))[:, None]
    y, size = x.double(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)
    a, b = x[..., ia].double(), x[..., ib].double()
    y[..., ia] = a * t.cos() - b * t.sin()
    y[..., ib] = a * t.sin() + b * t.cos()
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def check_rotated(got, ref):
    y, size = ref
    tol = torch.where(size > 0, HALF[got.dtype] * y.abs() + 7e-7 * size, 0)
    over = (got.double() - y).abs() - tol
    assert (over <= 0).all(), f"off by {float(over.max()):.3e} over its bound"


def attend(q, k, v, kv_len, scale):
    """attn_ref.attend with keys and values of different widths, and of one head or all."""
    n, hq, _ = q.shape
    if n == 0 or kv_len == 0:
        return (torch.zeros(n, hq, v.shape[2], dtype=torch.float64, device=q.device),
                torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device),
                torch.zeros(n, hq, v.shape[2], dtype=torch.float64, device=q.device))
    j = torch.arange(kv_len, device=q.device)
    sees = j[None, :] <= kv_len - n + torch.arange(n, device=q.device)[:, None]
    rows = sees.any(1)
    o = torch.zeros(n, hq, v.shape[2], dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device=q.device)
    for h in range(hq):
        g = h if k.shape[1] == hq else 0
        kh, vh = k[:, g].double(), v[:, g].double()
        x = torch.where(sees, (q[:, h].double() @ kh.t()) * scale, -math.inf)
        lse[rows, h] = torch.logsumexp(x[rows], 1)
        p = torch.zeros_like(x)
        p[rows] = torch.exp(x[rows] - lse[rows, h][:, None])
        o[:, h] = p @ vh
        a[:, h] = p @ vh.abs()
    return o, lse, a


def _all(parts):
    return tuple(torch.cat(x) for x in zip(*parts))


def prompt(q, k, k_r, v, lens, scale):
    if k_r is not None:
        k = torch.cat([k, k_r[:, None].expand(-1, k.shape[1], -1)], -1)
    cut = [x.split(lens) for x in (q, k, v)]
    return _all([attend(a, b, c, len(a), scale) for a, b, c in zip(*cut)])


def paged(q, cache, table, q_lens, kv_lens, scale):
    parts, t = [], 0
    for r, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        rows = attn_ref.gather(cache[:, None], table[r], kv)
        parts.append(attend(q[t:t + n], rows, rows[..., :512], kv, scale))
        t += n
    return _all(parts)
