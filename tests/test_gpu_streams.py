"""Calls given `stream=` beside work that still uses memory the current stream's
allocator thinks free. Reading the host side: tests/test_binding_streams.py."""
import pytest
import torch

import attn_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_attn import BF, DEV, F32, cached, cumulative, ints, packed

pytestmark = pytest.mark.gpu


def long_fill(numbers):
    """Work of a millisecond or more on the current stream, ending in NaN in blocks that
    are free again for the allocator."""
    a = torch.ones(4096, 4096, device=DEV)
    for _ in range(8):
        a = a @ a.mul(1e-4)
    for n in numbers:
        torch.empty(n, dtype=torch.uint8, device=DEV).view(torch.int8).fill_(-1)  # NaN in either type


@pytest.mark.parametrize("io", [BF, F32])
def test_outputs_and_workspace_meet_no_other_work(io):
    q_lens, kv_lens = [1, 3], [4000, 2500]
    q, kc, vc, table = cached(q_lens, kv_lens, 8, 2, 128, 64, io)
    cu, kv = cumulative(q_lens), ints(kv_lens)
    ref = attn_ref.paged(q, kc, vc, table, q_lens, kv_lens, 128 ** -0.5)
    need = kda.kda_attn_workspace_size(2, 4, 3, 8, 2, 128, io)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        long_fill([need, q.numel() * q.element_size(), 4 * 8 * 4])
        o, lse = kda.kda_attn_paged(q, kc, vc, table, cu, kv, max_q=3, stream=s)
        torch.cuda.synchronize()
        attn_ref.check(o, lse, ref)


def test_dropped_outputs_are_not_reused_too_early():
    """An lse that the caller drops belongs to `stream` until the kernel is done."""
    lens = [3000, 1000]
    q, k, v = packed(lens, 8, 2, 128, BF)
    cu = cumulative(lens)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        o, _ = kda.kda_attn_prompt(q, k, v, cu, max_len=3000, stream=s)
        taken = [torch.full((4000, 8), 7.0, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        assert all((t == 7).all() for t in taken)


def test_plan_on_a_stream_of_its_own():
    n, page = 300, 16
    old, new = [5] * n, [6 + i % 40 for i in range(n)]
    table = [[i] + [-1] * 3 for i in range(n)]
    ring = list(range(n, 3 * n)) + [-1] * n
    room = sum(b - a for a, b in zip(old, new)) + 3
    want = attn_ref.plan(old, new, table, ring, [0, 2 * n], page, room)
    s = torch.cuda.Stream()
    for _ in range(5):
        a, b, t, r, at = ints(old), ints(new), ints(table), ints(ring), ints([0, 2 * n])
        torch.cuda.synchronize()
        long_fill([4 * n, 4 * n + 4, 4 * room, 8])
        kv, cu, slot, out = kda.kda_kv_plan(a, b, t, r, at, page_size=page, max_tokens=room, stream=s)
        torch.cuda.synchronize()
        assert [x.tolist() for x in (kv, cu, slot, t, r, out)] == list(want[:6])
