"""The binding of the rotated appends and of latent attention without a GPU: whose memory
a call on a stream of its own makes, and what is refused before the library is called."""
import inspect

import pytest
import torch

import gated_delta_rule_57_gb300 as pkg
from gated_delta_rule_57_gb300 import kda, latent
from test_binding_streams import CURRENT, OTHER, Recorded, bf, i32, made  # noqa: F401

T, H = 4, 2
TURNS = torch.zeros(32, dtype=torch.int64)
QKV = bf(T, 3 * H, 64).split(H, 1)
CALLS = {
    "kda_kv_append_rope": lambda s: pkg.kda_kv_append_rope(*QKV, i32(T), i32(T), TURNS, bf(9, H, 16, 64), bf(9, H, 16, 64), stream=s),
    "kda_latent_append": lambda s: pkg.kda_latent_append(bf(T, 512), bf(T, 64), i32(T), bf(9, 16, 576), positions=i32(T), turns=TURNS,
                                                         q_r=bf(T, H, 64), stream=s),
    "kda_attn_latent_prompt": lambda s: pkg.kda_attn_latent_prompt(bf(T, H, 192), bf(T, H, 128), bf(T, 64), bf(T, H, 128), i32(2),
                                                                   max_len=1 << 20, stream=s),
    "kda_attn_latent_paged": lambda s: pkg.kda_attn_latent_paged(bf(T, H, 576), bf(200, 16, 576), i32(1, 150), i32(2), i32(1), scale=0.1,
                                                                 stream=s),
}


@pytest.fixture
def fakes(made, monkeypatch):  # noqa: F811
    monkeypatch.setattr(latent, "_device", lambda t: t.get_device())  # (all tensors here are the host's)
    return made


def test_every_call_with_a_stream_is_here():
    assert {n for n, f in vars(latent).items() if n.startswith("kda_") and inspect.isfunction(f)
            and "stream" in inspect.signature(f).parameters} == set(CALLS)


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_is_the_streams_own(fakes, name):
    out = CALLS[name](OTHER)
    assert fakes and all(stream is OTHER for stream, _ in fakes)
    for x in out if isinstance(out, tuple) else (out,):  # outputs wait for the caller's stream too
        assert not isinstance(x, Recorded) or CURRENT in x.__dict__.get("told", [])


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("stream", [None, CURRENT])
def test_on_the_current_stream_nothing_is_told(fakes, name, stream):
    CALLS[name](stream)
    assert all(s is CURRENT and not t.__dict__.get("told") for s, t in fakes)


@pytest.mark.parametrize("error,call", [
    (ValueError, lambda: CALLS["kda_kv_append_rope"](None)),  # not on a GPU
    (ValueError, lambda: CALLS["kda_latent_append"](None)),
    (ValueError, lambda: CALLS["kda_attn_latent_prompt"](None)),
    (ValueError, lambda: CALLS["kda_attn_latent_paged"](None)),
    (TypeError, lambda: pkg.kda_attn_latent_prompt(bf(T, H, 192).half(), bf(T, H, 128), bf(T, 64), bf(T, H, 128), i32(2))),
    (ValueError, lambda: pkg.kda_attn_latent_prompt(bf(T, H, 128), bf(T, H, 128), bf(T, 64), bf(T, H, 128), i32(2))),
    (ValueError, lambda: pkg.kda_attn_latent_prompt(bf(T, H, 192), bf(T, H, 128), bf(T, 64), bf(T, 1, 128), i32(2))),
    (TypeError, lambda: pkg.kda_attn_latent_paged(bf(T, H, 576).half(), bf(9, 16, 576), i32(1, 9), i32(2), i32(1), scale=1.0)),
    (ValueError, lambda: pkg.kda_attn_latent_paged(bf(T, H, 576), bf(9, 16, 512), i32(1, 9), i32(2), i32(1), scale=1.0)),
    (ValueError, lambda: pkg.kda_attn_latent_paged(bf(T, H, 576), bf(9, 16, 576).float(), i32(1, 9), i32(2), i32(1), scale=1.0)),
    (ValueError, lambda: pkg.kda_attn_latent_paged(bf(T, H, 128), bf(9, 16, 128), i32(1, 9), i32(2), i32(1), scale=1.0)),
    (ValueError, lambda: pkg.kda_attn_latent_paged(bf(T, H, 576), bf(9, 16, 576), i32(1, 9), i32(2), i32(1), scale=1.0, o=bf(T, H, 128))),
    (TypeError, lambda: pkg.kda_latent_append(bf(T, 512).half(), None, i32(T), bf(9, 16, 512))),
    (ValueError, lambda: pkg.kda_latent_append(bf(T, 512), None, i32(T), bf(9, 16, 576))),
    (ValueError, lambda: pkg.kda_latent_append(bf(T, 512), None, i32(T), bf(9, 16, 512), q_r=bf(T, H, 64))),
    (ValueError, lambda: pkg.kda_latent_append(bf(T, 512), bf(T, 64), i32(T), bf(9, 16, 576))),  # no positions
    (ValueError, lambda: pkg.kda_kv_append_rope(*QKV, i32(T), i32(T), TURNS, bf(9, 3, 16, 64), bf(9, 3, 16, 64))),
    (ValueError, lambda: pkg.kda_kv_append_rope(QKV[0][:2], *QKV[1:], i32(T), i32(T), TURNS, bf(9, H, 16, 64), bf(9, H, 16, 64))),
    (TypeError, lambda: pkg.kda_kv_append_rope(*(x.half() for x in QKV), i32(T), i32(T), TURNS, bf(9, H, 16, 64), bf(9, H, 16, 64))),
])
def test_refuses(error, call):
    with pytest.raises(error):
        call()


@pytest.mark.parametrize("call", [  # with addresses taken as they are
    lambda: pkg.kda_kv_append_rope(*QKV, i32(T - 1), i32(T), TURNS, bf(9, H, 16, 64), bf(9, H, 16, 64)),
    lambda: pkg.kda_kv_append_rope(*QKV, i32(T), i32(T - 1), TURNS, bf(9, H, 16, 64), bf(9, H, 16, 64)),
    lambda: pkg.kda_kv_append_rope(*QKV, i32(T).long(), i32(T), TURNS, bf(9, H, 16, 64), bf(9, H, 16, 64)),
    lambda: pkg.kda_kv_append_rope(*QKV, i32(T), i32(T), TURNS.double(), bf(9, H, 16, 64), bf(9, H, 16, 64)),
    lambda: pkg.kda_kv_append_rope(*QKV, i32(T), i32(T), TURNS, bf(9, H, 16, 64), bf(9, H, 16, 64), q_out=bf(T, H, 128)),
    lambda: pkg.kda_kv_append_rope(None, *QKV[1:], i32(T), i32(T), TURNS, bf(9, H, 16, 64), bf(9, H, 16, 64), q_out=bf(T, H, 64)),
    lambda: pkg.kda_latent_append(bf(T, 512), None, i32(T), bf(9, 16, 512), q_out=bf(T, H, 64)),
    lambda: pkg.kda_latent_append(bf(T, 512), bf(T, 64), i32(T), bf(9, 16, 576), positions=i32(T), turns=TURNS, q_out=bf(T, H, 64)),
    lambda: pkg.kda_latent_append(bf(512, T).t(), bf(T, 64), i32(T), bf(9, 16, 576), positions=i32(T), turns=TURNS),
    lambda: pkg.kda_latent_append(bf(T, 512), bf(T, 64), i32(T), bf(9, 16, 576), positions=i32(T), turns=TURNS[:16]),
    lambda: pkg.kda_latent_append(bf(T, 512), bf(T, 64), i32(T), bf(9, 16, 576), positions=i32(T), turns=TURNS, q_r=bf(T, H, 32)),
    lambda: pkg.kda_latent_append(bf(T, 512), bf(T, 64), i32(T), bf(9, 16, 576), positions=i32(T), turns=TURNS, k_out=bf(T, 32)),
    lambda: pkg.kda_attn_latent_paged(bf(T, 576, H).transpose(1, 2), bf(9, 16, 576), i32(1, 9), i32(2), i32(1), scale=1.0),
    lambda: pkg.kda_attn_latent_paged(bf(T, H, 576), bf(9, 16, 576), i32(1, 9), i32(3), i32(1), scale=1.0),
])
def test_refuses_shapes(fakes, call):
    with pytest.raises(ValueError):
        call()


def test_turns():
    """Exact fractions of a turn, whatever the size and sign of a frequency."""
    import math
    f = [1.0, 10000.0 ** -0.5, 1e-9, 0.0, -1.0, 2 * math.pi, 100.0]
    got = pkg.kda_rope_turns(f, device="cpu")
    assert got.dtype == torch.int64 and got.shape == (7,)
    for x, t in zip(f, got.tolist()):
        turn = math.remainder(x / (2 * math.pi), 1.0)
        assert abs(math.remainder(t / 2 ** 64 - turn, 1.0)) <= 2.0 ** -49 * max(1, abs(x))
    assert torch.equal(got, pkg.kda_rope_turns(torch.tensor(f, dtype=torch.float64), device="cpu"))


def test_short_keys_matches_header():
    import re
    from gated_delta_rule_57_gb300 import build
    text = open(build.INCLUDE + "/kda.h").read()
    assert kda.KDA_LATENT_SHORT_KEYS == int(re.search(r"#define KDA_LATENT_SHORT_KEYS (\d+)", text).group(1))
