"""Which stream the binding's own allocations belong to, on the host: a call
that is given a stream and no workspace must take its scratch from that stream's
memory.  Taken from the current stream's, the caching allocator could hand it
out again while the call's kernels still read and write it."""
import contextlib
import inspect
import re

import pytest
import torch

import test_prompt_binding as tp
from eagle_speculative_decoding_gb300 import binding as eb


class FakeLib:
    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("workspace_size") else 0


class FakeStream:
    cuda_stream = 77


@pytest.fixture
def allocations(monkeypatch):
    """(stream the allocation is made under, dtype) of every torch.empty."""
    seen, under = [], [None]
    real = torch.empty

    @contextlib.contextmanager
    def stream(s):
        under.append(s)
        yield
        under.pop()

    def empty(*shape, dtype=None, device=None):
        seen.append((under[-1], dtype))
        return real(*shape, dtype=dtype)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(eb, "_lib", FakeLib())
    monkeypatch.setattr(eb, "_raw_stream", lambda s, device: 0)
    monkeypatch.setattr(eb, "_lengths", lambda *a: (tp.B, tp.W))
    return seen


@pytest.mark.parametrize("name", ["attn", "attn4", "draft", "draft4"])
@pytest.mark.parametrize("given", [False, True])
def test_scratch_is_the_streams(allocations, name, given):
    call, base = tp.CALLS[name]
    s = FakeStream() if given else None
    call(**base(), stream=s)
    assert allocations == [(s, torch.uint8)]


def test_a_given_workspace_is_taken(allocations):
    call, base = tp.CALLS["attn"]
    call(**base(), stream=FakeStream(), ws=torch.zeros(16, dtype=torch.uint8))
    assert allocations == []


@pytest.mark.parametrize("given", [False, True])
def test_rope_table_is_the_streams(allocations, given):
    s = FakeStream() if given else None
    assert eb.eagle_rope_table(8, 128, 1e4, stream=s).shape == (8, 2, 64)
    assert allocations == [(s, torch.float32)]


def test_older_calls_too(allocations):
    x, s = torch.zeros(2, 64, dtype=torch.bfloat16), FakeStream()
    eb.eagle_linear(x, x, x, stream=s)
    eb.eagle_fuse_proj(x, x, x, x, x, stream=s)
    eb.eagle_draft_input(x, x, x, x, x, stream=s)
    eb.eagle_lmhead_topk(x, x, 1, x, x, stream=s)
    assert allocations == [(s, torch.uint8)] * 4


def test_every_call_that_allocates_names_its_stream():
    calls = [f for n, f in vars(eb).items() if n.startswith("eagle_") and "ws is None" in inspect.getsource(f)]
    assert len(calls) == 12
    for f in calls:
        assert re.search(r"ws = workspace\([^=]*, stream\)\n", inspect.getsource(f)), f.__name__
