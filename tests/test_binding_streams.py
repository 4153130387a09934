"""What the binding allocates for a call on another stream (no GPU): a block of PyTorch's caching allocator belongs
to the stream that is current when it is handed out, and may still be written by that stream's queued work, so
it has to come from the stream that the call runs on.  Outputs are recorded on the caller's stream, too, which
reads them."""

import contextlib

import pytest

torch = pytest.importorskip("torch")

import post_weight_quantization_03_amd as g  # noqa: E402
from post_weight_quantization_03_amd import attn  # noqa: E402


class Block:
    """A tensor's stand-in that knows which stream was current when it was made."""

    def __init__(self, of):
        self.of, self.recorded = of, []

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def streams(monkeypatch):
    now = ["callers"]

    @contextlib.contextmanager
    def current(stream):
        before, now[0] = now[0], stream
        try:
            yield
        finally:
            now[0] = before

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[0])
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Block(now[0]))
    monkeypatch.setattr(torch, "empty_like", lambda *a, **k: Block(now[0]))
    return now


class Like:
    device, shape = "cuda:0", (4, 2, 64)

    def new_empty(self, *a, **k):
        return Block(torch.cuda.current_stream())


MAKERS = {"workspace": lambda s: g._workspace(1 << 20, Like(), s),
          "output": lambda s: attn._empty((4, 2), Like(), s, None),
          "output like an input": lambda s: attn._empty_as(Like(), s)}


@pytest.mark.parametrize("what", MAKERS)
def test_memory_for_a_call_on_another_stream_is_of_that_stream(streams, what):
    block = MAKERS[what]("side")
    assert block.of == "side" and streams == ["callers"]
    assert block.recorded == ([] if what == "workspace" else ["callers"])


@pytest.mark.parametrize("what", MAKERS)
def test_memory_for_a_call_on_the_current_stream_is_of_it(streams, what):
    block = MAKERS[what](None)
    assert block.of == "callers" and block.recorded == []
