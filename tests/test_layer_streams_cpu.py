"""Where a layer's calls on another stream than the current one allocate:
blocks of the current stream's pool may have work still to come there, and a
workspace freed to it would be written again while the call still runs."""
import contextlib
import types

import numpy as np
import pytest
import torch

from input_adaptive_rank_amd import dyra as D

CURRENT = object()


class OtherStream:
    def __init__(self):
        self.waits = []

    def wait_stream(self, stream):
        self.waits.append(stream)


@pytest.fixture
def blocks(monkeypatch):
    at, made = [CURRENT], []

    class Block:
        def __init__(self, shape, dtype=None, device=None):
            self.shape, self.stream, self.recorded = shape, at[-1], []
            made.append(self)

        def record_stream(self, stream):
            self.recorded.append(stream)

        def numel(self):
            return self.shape if isinstance(self.shape, int) else int(np.prod(self.shape))

    @contextlib.contextmanager
    def on(stream):
        at.append(at[-1] if stream is None else stream)
        yield
        at.pop()

    monkeypatch.setattr(torch, "empty", Block)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: CURRENT)
    return made


def layer():
    t = D.DyraLayer.__new__(D.DyraLayer)
    t.spec = D.make_spec(D.KIND_LOWRANK, 64, 96, 8, k=16)
    t.dtype, t.device, t.half_steps, t.eps, t.solver = D.DT_BF16, "cuda:0", 2, 1e-6, 0
    t.plan = t.bias = t._ws = t._ws_key = None
    return t


ROWS = types.SimpleNamespace(dtype=torch.bfloat16, device="cuda:0")


@pytest.mark.parametrize("other", [False, True])
def test_ragged_call(blocks, monkeypatch, other):
    stream = OtherStream() if other else None
    monkeypatch.setattr(D, "forward_varlen", lambda *a, **k: None)
    Y, status = layer().forward_varlen(ROWS, [0, 30, 100], stream=stream)
    assert [b.stream for b in blocks] == [stream if other else CURRENT] * 3   # Y, workspace, status
    for b in (Y, status):
        assert b.recorded == ([CURRENT] if other else [])


@pytest.mark.parametrize("other", [False, True])
def test_uniform_call(blocks, monkeypatch, other):
    stream = OtherStream() if other else None
    monkeypatch.setattr(D, "forward", lambda *a, **k: None)
    t = layer()
    Y = t.forward(ROWS, 2, 50, stream=stream)
    assert Y.stream is (stream if other else CURRENT) and Y.recorded == ([CURRENT] if other else [])
    # the workspace is the layer's own: the stream waits for what its block's pool may still have to do
    assert t._ws.stream is CURRENT and t._ws.recorded == ([stream] if other else [])
    assert not other or stream.waits == [CURRENT]
    t.forward(ROWS, 2, 50, stream=stream)
    assert not other or (stream.waits == [CURRENT] and t._ws.recorded == [stream, stream])
