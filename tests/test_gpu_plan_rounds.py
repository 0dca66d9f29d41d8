"""Plans of more requests than a block holds in one round, against the serial definition."""
import random

import pytest

import attn_ref
from gated_delta_rule_57_gb300 import kda
from test_gpu_cache import run, state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2048, 2049, 4095, 4096, 4097, 8192, 8200, 12289, 16384])
@pytest.mark.parametrize("short", ["", "pages", "row", "tokens"])
def test_plan_of_several_rounds(n, short):
    rng = random.Random(n + len(short))
    page, longest = 16, 90
    old = [rng.choice([0, rng.randint(0, longest)]) for _ in range(n)]
    new = [rng.choice([x, x + 1, min(longest, x + rng.randint(0, 3 * page)), max(0, x - rng.randint(0, page)), 0]) for x in old]
    max_pages = -(-max(old + new) // page)
    table, ring, at = state(rng, old, page, max_pages, spare=4 * n)
    room = sum(max(0, b - a) for a, b in zip(old, new)) + 5
    if short == "pages":  # run out late, in another round than the first
        at[1] = int(0.8 * sum(max(0, -(-b // page) + a // -page) for a, b in zip(old, new)))
    elif short == "row":
        new[n // 2] = max_pages * page + 1
        room += new[n // 2]
    elif short == "tokens":
        room = int(room * 0.7)
    got, status = run(old, new, table, ring, at, page, room)
    want = attn_ref.plan(old, new, table, ring, at, page, room)
    assert got == list(want[:6])
    assert status == (kda.KDA_DEV_PAGES if want[6] else 0)
    assert want[6] == bool(short)
