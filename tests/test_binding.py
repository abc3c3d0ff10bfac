"""The Python binding's own steps, without a GPU."""
import torch

import fp4_sparse_attention_csa_gb300 as csa


def test_current_stream_with_and_without_the_raw_handle(monkeypatch):
    """The handle comes from torch's raw lookup where there is one, else from the
    public stream object."""
    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 1000 + dev, raising=False)
    assert csa._stream(None) == 1003
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    assert csa._stream(None) == 77
    assert csa._stream(5) == 5 and csa._stream(Stream) == 77
