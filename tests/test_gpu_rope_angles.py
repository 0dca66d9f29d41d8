"""The rotation of a pair (1, 0) in fp32 is the angle's cos and sin as they are: near their
zeros too, at any position.

An angle is position x turns modulo 2^64, exactly, less its nearest quarter turn: at most an
eighth of a turn, cut at 2^-34 of a turn (3.7e-10 rad) and rounded to fp32 once, which moves its
sin by 2^-24 of itself and its cos by less. The functions are good to a unit in the last place,
2^-23 at most. So |y - ref| <= 3.1 x 2^-24 |ref| + 3.7e-10; at quarter turns exactly 0 and 1."""
import math
import random

import pytest
import torch

from gated_delta_rule_57_gb300 import kda

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cos_sin(turn):
    """Of a fraction turn / 2^64 of a turn: reduced in whole numbers, then in 64 bits."""
    quarter = (turn + (1 << 61) >> 62) % 4
    rest = (turn - (quarter << 62) + (1 << 63)) % (1 << 64) - (1 << 63)
    t = math.ldexp(rest, -63) * math.pi
    c, s = math.cos(t), math.sin(t)
    return [(c, s), (-s, c), (-c, -s), (s, -c)][quarter]


def signed(x):
    return (x + (1 << 63)) % (1 << 64) - (1 << 63)


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("kind", ["any", "near quarters", "quarters"])
def test_cos_and_sin(kind, neighbours):
    rng = random.Random(kind)
    n, rot = 500, 64
    if kind == "any":
        turns = [rng.getrandbits(64) for _ in range(rot // 2)]
        pos = [rng.randrange(-(1 << 31), 1 << 31) for _ in range(n)]
    elif kind == "near quarters":
        turns = [(rng.randrange(4) << 62) + rng.choice([-1, 1]) * rng.getrandbits(rng.randint(1, 55)) for _ in range(rot // 2)]
        pos = [rng.randint(-100, 100) for _ in range(n)]
    else:
        turns = [i << 62 for i in range(rot // 2)]
        pos = list(range(-n // 2, n // 2))
    x = torch.zeros(n, 1, rot, device=DEV)
    x[..., slice(0, rot, 2) if neighbours else slice(0, rot // 2)] = 1
    kv = torch.zeros(n, 0, rot, device=DEV)
    cache = torch.zeros(1, 0, 16, rot, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    y = kda.kda_kv_append_rope(x, kv, kv, torch.full((n,), -1, **i32), torch.tensor(pos, **i32),
                               torch.tensor([signed(t) for t in turns], dtype=torch.int64, device=DEV), cache, cache, neighbours=neighbours)
    y = y[:, 0].double().cpu()
    a, b = (y[:, ::2], y[:, 1::2]) if neighbours else (y[:, :rot // 2], y[:, rot // 2:])
    ref = torch.tensor([[cos_sin(p * t % (1 << 64)) for t in turns] for p in pos], dtype=torch.float64)
    for got, want in ((a, ref[..., 0]), (b, ref[..., 1])):
        over = (got - want).abs() - 3.1 * 2.0 ** -24 * want.abs() - (3.7e-10 if kind != "quarters" else 0)
        assert (over <= 0).all(), f"off by {float(over.max()):.3e} over its bound"
