"""Whose memory a workspace is that a call allocates itself (no GPU needed): the caller cannot order
it, so it has to come from the stream that uses it, or that stream has to be known to the allocator."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import combine_quant_amd as cq
from combine_quant_amd import binding

CFG = cq.make_config(2, 8, 3, 1024, 2)
X = torch.zeros((2, 3, 1024), dtype=torch.bfloat16)
IDS, W = torch.zeros((2, 3, 2), dtype=torch.int32), torch.zeros((2, 3, 2))


class _Scratch:
    """Stands for a workspace: where it was allocated and which streams were recorded on it."""

    def __init__(self, stream):
        self.stream, self.recorded = stream, []

    def record_stream(self, stream):
        self.recorded.append(stream)


class _Streams:
    """The current stream, and the workspaces allocated meanwhile."""

    def __init__(self, monkeypatch):
        self.now, self.made, self.launched = SimpleNamespace(cuda_stream=1), [], []
        empty = torch.empty

        def fake_empty(*args, **kw):
            if kw.get("dtype") is not torch.uint8:
                return empty(*args, **kw)
            self.made.append(_Scratch(self.now))
            return self.made[-1]

        @contextlib.contextmanager
        def use(stream):
            before, self.now = self.now, self.now if stream is None else stream
            yield
            self.now = before

        def marshalled(*args):
            return (lambda s: self.launched.append(s.value) or 0), (), torch.device("cuda", 0)
        monkeypatch.setattr(torch, "empty", fake_empty)
        monkeypatch.setattr(torch.cuda, "stream", use)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.now)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: self.now.cuda_stream, raising=False)
        monkeypatch.setattr(binding, "_experts_layer_call", marshalled)
        monkeypatch.setattr(binding, "_combine_scatter_call", marshalled)


def _layer(prepare, **kw):
    call = cq.prepare_experts_layer if prepare else cq.experts_layer
    return call(CFG, cq.make_experts(144), X, IDS, W, X, X, **kw)


def _scatter(prepare, **kw):
    call = cq.prepare_combine_scatter if prepare else cq.combine_scatter
    return call(CFG, X, IDS, IDS, IDS, W, **kw)


@pytest.mark.parametrize("call", [_layer, _scatter])
def test_a_call_on_another_stream_allocates_there(monkeypatch, call):
    streams, other = _Streams(monkeypatch), SimpleNamespace(cuda_stream=2)
    call(False, stream=other)
    assert streams.launched == [2] and len(streams.made) == 1
    assert streams.made[0].stream is other
    call(False)
    assert streams.launched == [2, 1] and streams.made[1].stream is streams.now


@pytest.mark.parametrize("call", [_layer, _scatter])
def test_a_plan_makes_other_streams_known(monkeypatch, call):
    streams, other = _Streams(monkeypatch), SimpleNamespace(cuda_stream=2)
    launch, _ = call(True)
    launch()
    assert streams.made[0].recorded == []
    launch(other)
    assert streams.made[0].recorded == [other]
    streams.now = SimpleNamespace(cuda_stream=3)
    launch()
    assert streams.made[0].recorded == [other, streams.now] and streams.launched == [1, 2, 3]


@pytest.mark.parametrize("call", [_layer, _scatter])
def test_the_callers_workspace_is_the_callers(monkeypatch, call):
    streams, other, mine = _Streams(monkeypatch), SimpleNamespace(cuda_stream=2), _Scratch(None)
    launch, _ = call(True, workspace=mine)
    launch(other)
    call(False, workspace=mine, stream=other)
    assert streams.made == [] and mine.recorded == [] and streams.launched == [2, 2]
