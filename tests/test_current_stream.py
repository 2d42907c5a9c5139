"""A call without a stream runs on torch's current one, whether or not torch hands out its handle directly (CPU)."""
from types import SimpleNamespace

import pytest
import torch

import chunk_wise_hierarchical_hils_b200 as hils


@pytest.mark.parametrize("direct", [True, False])
def test_the_current_stream(direct, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(cuda_stream=4000))
    if direct:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 * (device + 1), raising=False)
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    assert hils._stream(None) == 4000
    assert hils._stream(17) == 17 and hils._stream(SimpleNamespace(cuda_stream=18)) == 18
