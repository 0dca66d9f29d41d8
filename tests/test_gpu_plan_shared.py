"""Plans whose prefix sums just fill the shared memory that a kernel has unasked."""
import pytest

import attn_ref
from test_gpu_cache import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [4000, 4009, 4010, 4088, 4089, 4090, 4093, 4094, 4095, 4096])
def test_plan_around_48_kb(n):
    old, new = [i % 5 for i in range(n)], [(i * 3) % 7 for i in range(n)]
    table, ring = [[-1, -1] for _ in range(n)], list(range(2 * n)) + [-1] * n
    for r, x in enumerate(old):
        if x:
            table[r][0] = 2 * n + r
    room = sum(max(0, b - a) for a, b in zip(old, new))
    got, status = run(old, new, table, ring, [0, 2 * n], 4, room)
    assert got == list(attn_ref.plan(old, new, table, ring, [0, 2 * n], 4, room)[:6]) and status == 0
