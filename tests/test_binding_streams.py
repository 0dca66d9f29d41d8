"""What a call given `stream=` makes for itself comes from that stream's memory.

With fakes for the library, the streams and the tensors' device, so that no GPU is
needed; tests/test_gpu_streams.py runs the calls."""
import contextlib
import inspect
from types import SimpleNamespace

import pytest
import torch

from gated_delta_rule_57_gb300 import kda

CURRENT, OTHER = SimpleNamespace(cuda_stream=1), SimpleNamespace(cuda_stream=2)


class Recorded(torch.Tensor):
    """A tensor that notes the streams told to the allocator."""

    def record_stream(self, stream):
        self.__dict__.setdefault("told", []).append(stream)


@pytest.fixture
def made(monkeypatch):
    """[(stream whose memory it is, tensor)] of every tensor the binding makes."""
    log, now = [], [CURRENT]

    @contextlib.contextmanager
    def use(stream):
        now.append(stream)
        yield
        now.pop()

    empty = torch.empty

    def recording_empty(*a, **kw):
        t = empty(*a, **kw).as_subclass(Recorded)
        log.append((now[-1], t))
        return t

    def call(name):
        return lambda *a: 4096 if name.endswith("workspace_size") else 2 if name.endswith("hint") else 0

    class Lib:
        def __getattr__(self, name):
            return call(name)

    monkeypatch.setattr(kda, "_lib", Lib())
    monkeypatch.setattr(kda, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(kda, "_rows", lambda name, t, dtype=None: (t.data_ptr(), t.stride(0)))
    monkeypatch.setattr(kda, "_stream", lambda s: CURRENT.cuda_stream if s is None else s.cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch, "empty", recording_empty)
    return log


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


B, T, H, D = 1, 4, 2, 64
SEQ = (bf(B, T, H, D), bf(B, T, H, D), bf(B, T, H, D), torch.zeros(B, T, H, D), torch.zeros(B, T, H))
TOK = tuple(x[0, :1] for x in SEQ)
CACHE = (bf(200, H, 16, D), bf(200, H, 16, D))
CALLS = {
    "kda_chunk_fwd": lambda s: kda.kda_chunk_fwd(*SEQ, stream=s),
    "kda_chunk_fwd_decay_probe": lambda s: kda.kda_chunk_fwd_decay_probe(SEQ[3], stream=s),
    "kda_chunk_fwd_segmented": lambda s: kda.kda_chunk_fwd_segmented(*SEQ, nseg=2, stream=s),
    "kda_chunk_fwd_segmented_noalloc": lambda s: kda.kda_chunk_fwd_segmented_noalloc(*SEQ, nseg=2, stream=s),
    "kda_chunk_fwd_slice_transition": lambda s: kda.kda_chunk_fwd_slice_transition(*(SEQ[i] for i in (0, 1, 3, 4)), stream=s),
    "kda_chunk_fwd_slice_correct": lambda s: kda.kda_chunk_fwd_slice_correct(
        *(SEQ[i] for i in (0, 1, 3, 4)), torch.zeros(B, H, D, D), SEQ[2], stream=s),
    "kda_state_scan": lambda s: kda.kda_state_scan(torch.zeros(2, B, H, D, D), torch.zeros(1, B, H, D, D), stream=s),
    "kda_selftest_wait_timeout": lambda s: kda.kda_selftest_wait_timeout(i32(1), stream=s),
    "kda_chunk_fwd_ckpt": lambda s: kda.kda_chunk_fwd_ckpt(*SEQ, ckpt_every=2, stream=s),
    "kda_decode_step": lambda s: kda.kda_decode_step(*TOK, torch.zeros(1, H, D, D), stream=s),
    "kda_decode_multi": lambda s: kda.kda_decode_multi(*SEQ, torch.zeros(1, H, D, D), stream=s),
    "kda_kv_plan": lambda s: kda.kda_kv_plan(i32(2), i32(2), i32(2, 3), i32(9), i32(2), page_size=16, max_tokens=5, stream=s),
    "kda_kv_append": lambda s: kda.kda_kv_append(SEQ[1][0], SEQ[2][0], i32(T), *CACHE, stream=s),
    "kda_attn_prompt": lambda s: kda.kda_attn_prompt(*(x[0] for x in SEQ[:3]), i32(2), max_len=1 << 20, stream=s),
    "kda_attn_paged": lambda s: kda.kda_attn_paged(SEQ[0][0], *CACHE, i32(1, 150), i32(2), i32(1), stream=s),
}
MAKES_NOTHING = {"kda_chunk_fwd_slice_correct", "kda_selftest_wait_timeout", "kda_kv_append"}


def test_every_call_with_a_stream_is_here():
    have = {n for n, f in vars(kda).items() if n.startswith("kda_") and inspect.isfunction(f)
            and "stream" in inspect.signature(f).parameters}
    assert have == set(CALLS)


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_is_the_streams_own(made, name):
    out = CALLS[name](OTHER)
    assert bool(made) == (name not in MAKES_NOTHING)
    assert all(stream is OTHER for stream, _ in made)
    # outputs given back wait for the caller's stream too
    for x in out if isinstance(out, tuple) else (out,):
        if isinstance(x, Recorded):
            assert CURRENT in x.__dict__.get("told", [])


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("stream", [None, CURRENT])
def test_on_the_current_stream_nothing_is_told(made, name, stream):
    CALLS[name](stream)
    assert all(s is CURRENT and not t.__dict__.get("told") for s, t in made)
