"""Calls on a given stream: whose memory their outputs are.  A block that the
caching allocator takes from the current stream's pool may still be in use by
that stream's pending work, which the given stream does not wait for; so what a
call allocates has to come from the given stream's pool, and to be marked as
used by the current one.  Stand-ins for streams and for the native calls: no
GPU call."""
import contextlib
import types

import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from linear_recurrence_chunked_gated_amd import _lib

DEV = torch.device("cuda", 0)


class Stream:
    device, cuda_stream = DEV, 64


class Made:
    """An output that a native call allocated."""

    def __init__(self):
        self.marked = []

    def numel(self):
        return 8

    def record_stream(self, stream):
        self.marked.append(stream)


@pytest.fixture
def streams(monkeypatch):
    """(current stream, calls): calls collects, for each native call, the
    stream that was current at it."""
    state = types.SimpleNamespace(current=Stream(), calls=[])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state.current)

    @contextlib.contextmanager
    def switch(s):
        before, state.current = state.current, s
        try:
            yield
        finally:
            state.current = before

    monkeypatch.setattr(torch.cuda, "stream", switch)

    def native(count):
        def call(*args):
            state.calls.append(state.current)
            return Made() if count is None else tuple(Made() for _ in range(count))
        return call

    monkeypatch.setattr(_lib, "_calls", types.SimpleNamespace(
        recurrent_step=native(None), shortconv_step=native(None), gated_norm_fwd=native(None),
        gated_norm_bwd=native(4), residual_norm_fwd=native(2), residual_norm_bwd=native(5)))
    return state


X = types.SimpleNamespace(is_cuda=True, device=DEV)
CALLS = {
    "recurrent_step": lambda s: gdn.recurrent_step(X, X, X, X, X, X, stream=s),
    "shortconv_step": lambda s: gdn.shortconv_step(X, X, X, stream=s),
    "gated_norm_fwd": lambda s: gdn.gated_norm_fwd(X, X, X, stream=s),
    "gated_norm_bwd": lambda s: gdn.gated_norm_bwd(X, X, X, X, stream=s),
    "residual_norm_fwd": lambda s: gdn.residual_norm_fwd(X, X, X, X, stream=s),
    "residual_norm_bwd": lambda s: gdn.residual_norm_bwd(X, X, X, X, X, X, stream=s),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_outputs_belong_to_the_given_stream(streams, name):
    here, side = streams.current, Stream()
    got = CALLS[name](side)
    assert streams.calls == [side] and streams.current is here
    for t in got if isinstance(got, tuple) else (got,):
        assert t.marked == [here]


@pytest.mark.parametrize("name", list(CALLS))
def test_the_current_stream_given_by_name(streams, name):
    here = streams.current
    got = CALLS[name](here)
    assert streams.calls == [here]
    for t in got if isinstance(got, tuple) else (got,):
        assert t.marked == []


def test_outputs_of_the_caller_are_not_marked(streams):
    mine = [Made() for _ in range(4)]
    _lib._calls.recurrent_step = lambda *a: mine[0]
    _lib._calls.residual_norm_fwd = lambda *a: (mine[1], mine[2])
    gdn.recurrent_step(X, X, X, X, X, X, o=mine[0], stream=Stream())
    gdn.residual_norm_fwd(X, X, h=mine[2], y=mine[1], stream=Stream())
    _lib._calls.gated_norm_bwd = lambda *a: tuple(mine)
    gdn.gated_norm_bwd(X, X, X, X, grads=tuple(mine[:3]), workspace=mine[3], stream=Stream())
    # without r the norm's h is x, the caller's own
    _lib._calls.residual_norm_fwd = lambda *a: (made, mine[3])
    made, here = Made(), streams.current
    gdn.residual_norm_fwd(X, stream=Stream())
    assert made.marked == [here] and all(t.marked == [] for t in mine)


@pytest.mark.parametrize("given", ["none", "current", "side"])
def test_new_buffers_belong_to_the_given_stream(streams, given):
    """The chunk, convolution and chain calls make their buffers by new_on."""
    here = streams.current
    stream = {"none": None, "current": here, "side": Stream()}[given]

    def make(n, dtype=None):
        streams.calls.append(streams.current)
        assert n == 3 and dtype == "x"
        return Made()

    t = _lib.new_on(stream, make, 3, dtype="x")
    assert streams.calls == [stream if given == "side" else here] and streams.current is here
    assert t.marked == ([here] if given == "side" else [])
    assert _lib.new_on(stream, lambda: None) is None  # an empty workspace
