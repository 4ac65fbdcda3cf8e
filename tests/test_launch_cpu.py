"""Which stream a plan enqueues on (no GPU needed)."""
from types import SimpleNamespace

import pytest
import torch

from combine_quant_amd import binding


@pytest.mark.parametrize("raw", [True, False])
def test_current_stream_with_and_without_the_handles_function(monkeypatch, raw):
    asked, launched = [], []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda i: asked.append(i) or SimpleNamespace(cuda_stream=7))
    if raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: asked.append(i) or 7, raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    launch = binding.Launch(lambda s: launched.append(s.value) or 0, (), torch.device("cuda", 1), None)
    launch()
    launch(SimpleNamespace(cuda_stream=9))
    assert launched == [7, 9] and asked == [1]
