"""Binding of the calls for rotation by position and for layers that keep one latent
vector a token (``include/kda.h``): argument marshalling only, as in ``kda.py``, whose
conventions (streams, what a call makes, errors) hold here too. The calls are attributes of
`kda` as well, as all others are.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import kda as _k
from .kda import KDA_ERR_INVALID_ARG, KDA_F32, KDA_LATENT_SHORT_KEYS, KdaError, lib

__all__ = ["kda_rope_turns", "kda_kv_append_rope", "kda_latent_append", "kda_attn_latent_workspace_size",
           "kda_attn_latent_paged", "kda_attn_latent_prompt"]

_PI = (314159265358979323846264338327950288419716939937510582097494459 << 200) // 10 ** 62  # pi 2^200


def kda_rope_turns(inv_freq, device="cuda"):
    """Frequencies of the rotation's pairs, in radians per token (a sequence or
    tensor of rot / 2 numbers, taken as they are in 64 bits, e.g. base ** (-2 i / rot)),
    as the int64 tensor of 64-bit fractions of a turn that the appends take. Made
    once, on the host."""
    if isinstance(inv_freq, torch.Tensor):
        inv_freq = inv_freq.detach().double().reshape(-1).tolist()
    turns = []
    for f in inv_freq:
        n, d = float(f).as_integer_ratio()
        x = (n << 264) // (d * _PI) + 1 >> 1  # 2^63 f / pi, rounded
        turns.append((x + 2 ** 63) % 2 ** 64 - 2 ** 63)
    return torch.tensor(turns, dtype=torch.int64, device=device)


def _device(t: torch.Tensor) -> int:
    """Number of a call's device: its first tensor's, which is to be the current one, where
    the call's kernels run."""
    device = t.get_device()
    if device < 0 or device != torch._C._cuda_getDevice():
        raise ValueError("KDA tensors must live on the current CUDA device")
    return device


def _ptr(dev: int, t: Optional[torch.Tensor]):
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError("KDA tensors must live on one CUDA device")
    if not t.is_contiguous():
        raise ValueError("KDA tensors must be contiguous")
    return t.data_ptr()


def _ints(dev: int, name: str, t: torch.Tensor, *shape):
    """Address of an int32 tensor of the given shape."""
    if t.shape != shape or t.dtype is not torch.int32:
        raise ValueError(f"{name} must be an int32 tensor of shape {shape}")
    return _ptr(dev, t)


def _heads(dev: int, name: str, t: torch.Tensor, T, H, d, dtype):
    """Address, token and head stride of a [T, H, d] tensor whose channels are contiguous."""
    if t.shape != (T, H, d) or t.dtype is not dtype:
        raise ValueError(f"{name} must be [{T}, {H}, {d}] of {dtype}")
    st, sh, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    if H <= 1:
        sh = d
    if t.get_device() != dev:
        raise ValueError("KDA tensors must live on one CUDA device")
    return t.data_ptr(), st if T > 1 else d, sh  # (one token's stride says nothing: the least that is taken)


def _packed(dev: int, name: str, t: torch.Tensor, T, H, d, dtype):
    """Address and token stride of a [T, H, d] tensor whose heads are contiguous."""
    if t.shape != (T, H, d) or t.dtype is not dtype:
        raise ValueError(f"{name} must be [{T}, {H}, {d}] of {dtype}")
    st, sh, sd = t.stride()
    if sd != 1 and d > 1 or sh != d and H > 1:
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if t.get_device() != dev:
        raise ValueError("KDA tensors must live on one CUDA device")
    return t.data_ptr(), st if T > 1 else H * d


def _flat(dev: int, name: str, t: torch.Tensor, T, d, dtype):
    """Address and token stride of a [T, d] tensor whose channels are contiguous."""
    if t.shape != (T, d) or t.dtype is not dtype:
        raise ValueError(f"{name} must be [{T}, {d}] of {dtype}")
    st, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the channels of a token must be contiguous")
    if t.get_device() != dev:
        raise ValueError("KDA tensors must live on one CUDA device")
    return t.data_ptr(), st if T > 1 else d


def _per_token(dev: int, name: str, t: torch.Tensor, T):
    """Address of an int32 tensor with an entry for each of T tokens, or more."""
    shape = t.shape
    if len(shape) != 1 or shape[0] < T or t.dtype is not torch.int32:
        raise ValueError(f"{name} must be an int32 tensor with an entry per token")
    return _ptr(dev, t)


def _turns(dev: int, t: torch.Tensor):
    """Address of a rotation's frequencies, and the channels that it turns."""
    shape = t.shape
    if len(shape) != 1 or t.dtype is not torch.int64:
        raise ValueError("turns must be an int64 tensor [rot / 2], as kda_rope_turns makes it")
    return _ptr(dev, t), 2 * shape[0]


def kda_kv_append_rope(q, k, v, slot_map, positions, turns, k_cache, v_cache, *,
                       neighbours: bool = False, q_out=None, k_out=None,
                       status: Optional[torch.Tensor] = None, stream=None):
    """kda_kv_append with rotation by position: q [T, Hq, d] is rotated into q_out (made
    here when not given; q itself: in place), k rotated and v copied to their slots; the
    rotated keys go to k_out [T, Hkv, d] too where one is given (k itself: in place).
    positions: [T] int32; turns: see kda_rope_turns (its length is rot / 2; channels from
    rot on are copied); neighbours: pairs are channels 2 i, 2 i + 1 instead of i,
    i + rot / 2. q may be None. Returns q_out."""
    pages, Hkv, page, d = k_cache.shape
    dt = k.dtype
    io = _k._DTYPE.get(dt)
    if io is None:
        raise TypeError(f"unsupported k dtype {dt}")
    T = k.shape[0]
    dev = _device(k)
    if v_cache.shape != (pages, Hkv, page, d) or k_cache.dtype is not dt or v_cache.dtype is not dt:
        raise ValueError("the caches must be [num_pages, Hkv, page_size, d] of k's dtype")
    qp = op = kop = None
    Hq = qs = os_ = kos = 0
    if k_out is not None:
        kop, kos = _packed(dev, "k_out", k_out, T, Hkv, d, dt)
    if q is None:
        if q_out is not None:
            raise ValueError("without q there is no q_out")
    else:
        Hq = q.shape[1]
        qp, qs = _packed(dev, "q", q, T, Hq, d, dt)
        if q_out is None:
            q_out = _k._empty((T, Hq, d), dt, q, stream)
            op, os_ = q_out.data_ptr(), Hq * d
        else:
            op, os_ = _packed(dev, "q_out", q_out, T, Hq, d, dt)
    kp, ks = _packed(dev, "k", k, T, Hkv, d, dt)
    vp, vs = _packed(dev, "v", v, T, Hkv, d, dt)
    tp, rot = _turns(dev, turns)
    code = (_k._lib or lib()).kda_kv_append_rope(
        qp, kp, vp, _per_token(dev, "slot_map", slot_map, T), _per_token(dev, "positions", positions, T), tp,
        _ptr(dev, k_cache), _ptr(dev, v_cache), op, kop, T, Hq, Hkv, d, rot, neighbours, qs, ks, vs, os_,
        kos, pages, page, io, _ptr(dev, status), _k._stream(stream))
    if code:
        _k._check(code)
    return q_out


def kda_latent_append(c, k_r, slot_map, cache, *, positions=None, turns=None, q_r=None, q_out=None,
                      k_out=None, neighbours: bool = False, status: Optional[torch.Tensor] = None,
                      stream=None):
    """Write the latents c [T, 512] and the rotated key parts k_r [T, 64] (None: a
    layer without) of T tokens to the slots slot_map [T] of cache [num_pages,
    page_size, 512 or 576], in place; rotate the queries' part q_r [T, Hq, 64] (a view
    of any strides) into q_out (made here when not given; q_r itself: in place) and write
    the rotated key part to k_out [T, 64] too where one is given. positions, turns and
    neighbours as for kda_kv_append_rope. Returns q_out (None without q_r)."""
    pages, page, dc = cache.shape
    T, dl = c.shape
    dt = c.dtype
    io = _k._DTYPE.get(dt)
    if io is None:
        raise TypeError(f"unsupported c dtype {dt}")
    dev = _device(c)
    dr = 0 if k_r is None else k_r.shape[1]
    if dc != dl + dr or cache.dtype != dt:
        raise ValueError("cache must be [num_pages, page_size, dl + dr] of c's dtype")
    cp, cs = _flat(dev, "c", c, T, dl, dt)
    kp = qp = op = kop = tp = pp = None
    ks = qs = qh = os_ = oh = kos = Hq = 0
    if k_r is None:
        if q_r is not None or q_out is not None or k_out is not None:
            raise ValueError("without k_r there are no q_r, q_out and k_out")
    else:
        if turns is None or positions is None:
            raise ValueError("k_r needs positions and turns")
        kp, ks = _flat(dev, "k_r", k_r, T, dr, dt)
        (tp, rot), pp = _turns(dev, turns), _per_token(dev, "positions", positions, T)
        if rot != dr:
            raise ValueError("turns must have an entry per pair of k_r's channels")
        if k_out is not None:
            kop, kos = _flat(dev, "k_out", k_out, T, dr, dt)
        if q_r is None:
            if q_out is not None:
                raise ValueError("without q_r there is no q_out")
        else:
            Hq = q_r.shape[1]
            qp, qs, qh = _heads(dev, "q_r", q_r, T, Hq, dr, dt)
            if q_out is None:
                q_out = _k._empty((T, Hq, dr), dt, c, stream)
            op, os_, oh = _heads(dev, "q_out", q_out, T, Hq, dr, dt)
    code = (_k._lib or lib()).kda_latent_append(
        cp, kp, qp, _per_token(dev, "slot_map", slot_map, T), pp, tp, _ptr(dev, cache), op, kop, T, Hq, dl, dr, neighbours,
        cs, ks, qs, qh, os_, oh, kos, pages, page, io, _ptr(dev, status), _k._stream(stream))
    if code:
        _k._check(code)
    return q_out if q_r is not None else None


def kda_attn_latent_workspace_size(N: int, total_q: int, max_q: int, Hq: int, dl: int = 512, dr: int = 64,
                                   io: torch.dtype = torch.bfloat16) -> int:
    n = lib().kda_attn_latent_workspace_size(N, total_q, max_q, Hq, dl, dr, _k._DTYPE[io])
    if n == ctypes.c_size_t(-1).value:
        raise KdaError(KDA_ERR_INVALID_ARG, "unsupported problem size")
    return int(n)


def kda_attn_latent_paged(q, cache, block_table, cu_q, kv_len, *, scale: float, max_q: Optional[int] = None,
                          o=None, lse=None, want_lse: bool = True, workspace=None,
                          status: Optional[torch.Tensor] = None, stream=None):
    """Causal attention of each request's last tokens over its paged latent cache, in
    the absorbed form: every head's keys are the cached rows, its values their first
    512 channels. q: [T, Hq, 512 + dr] (a view of any token and head strides); cache:
    [num_pages, page_size, 512 + dr]; block_table, cu_q, kv_len and max_q as for
    kda_attn_paged; scale: that of the expanded heads, e.g. (128 + dr) ** -0.5.
    Returns (o [T, Hq, 512], lse [T, Hq] or None)."""
    T, Hq, d = q.shape
    pages, page, dc = cache.shape
    N, max_pages = block_table.shape
    io = _k._DTYPE.get(q.dtype)
    if io is None:
        raise TypeError(f"unsupported q dtype {q.dtype}")
    if dc != d or cache.dtype != q.dtype or d < 512:
        raise ValueError("the cache must be [num_pages, page_size, 512 + dr] of q's channels and dtype")
    most = T if max_q is None else max_q
    dev = _device(q)
    o, lse = _k._attn_outputs(q, 512, o, lse, want_lse, stream)
    if workspace is None and max_pages * page > KDA_LATENT_SHORT_KEYS // (4 if io == KDA_F32 else 1):
        need = (_k._lib or lib()).kda_attn_latent_workspace_size(N, T, most, Hq, 512, d - 512, io)
        if need != ctypes.c_size_t(-1).value and need:  # the call itself reports bad arguments
            workspace = _k._empty(need, torch.uint8, q, stream, scratch=True)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    qp, qs, qh = _heads(dev, "q", q, T, Hq, d, q.dtype)
    _k._check((_k._lib or lib()).kda_attn_latent_paged(
        qp, _ptr(dev, cache), _ints(dev, "block_table", block_table, N, max_pages), _ints(dev, "cu_q", cu_q, N + 1),
        _ints(dev, "kv_len", kv_len, N), _ptr(dev, o), _ptr(dev, lse), N, T, most, Hq, 512, d - 512, qs, qh, pages, page,
        max_pages, scale, io, _ptr(dev, workspace), ws_bytes, _ptr(dev, status), _k._stream(stream)))
    return o, lse


def kda_attn_latent_prompt(q, k, k_r, v, cu_seqlens, *, max_len: Optional[int] = None,
                           scale: Optional[float] = None, o=None, lse=None, want_lse: bool = True,
                           workspace=None, status: Optional[torch.Tensor] = None, stream=None):
    """Causal attention over packed prompts whose heads' keys and values were expanded
    from the latents. q: [T, H, 128 + dr]; k, v: [T, H, 128]; k_r: [T, dr], the rotated
    key channels that all heads share (None: dr = 0); views of any token and head
    strides; cu_seqlens and max_len as for kda_attn_prompt; scale: None for
    1 / sqrt(128 + dr). Returns (o [T, H, 128], lse [T, H] or None)."""
    T, H, dq = q.shape
    d = k.shape[-1]
    N = cu_seqlens.numel() - 1
    dr = 0 if k_r is None else k_r.shape[1]
    if k.shape != (T, H, d) or v.shape != k.shape or dq != d + dr:
        raise ValueError("q must be [T, H, d + dr], k and v [T, H, d]")
    most = T if max_len is None else max_len
    dev = _device(q) if q.dtype in _k._DTYPE else -1
    io, o, lse, workspace, ws_bytes = _k._attn_buffers(q, N, most, most, H, o, lse, want_lse, workspace, stream, d)
    dt = q.dtype
    qp, qs, qh = _heads(dev, "q", q, T, H, dq, dt)
    kp, ks, kh = _heads(dev, "k", k, T, H, d, dt)
    vp, vs, vh = _heads(dev, "v", v, T, H, d, dt)
    rp, rs = _flat(dev, "k_r", k_r, T, dr, dt) if dr else (None, 0)
    _k._check((_k._lib or lib()).kda_attn_latent_prompt(
        qp, kp, rp, vp, _ints(dev, "cu_seqlens", cu_seqlens, N + 1), _ptr(dev, o), _ptr(dev, lse), N, T, most, H, d, dr, qs, qh,
        ks, kh, rs, vs, vh, dq ** -0.5 if scale is None else scale, io, _ptr(dev, workspace), ws_bytes,
        _ptr(dev, status), _k._stream(stream)))
    return o, lse
