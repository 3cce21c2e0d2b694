"""The binding's handle of the current stream, with and without the functions of
torch's that it comes from."""
import pytest


@pytest.mark.parametrize("gone", [(), ("_cuda_getCurrentRawStream",), ("_cuda_getDevice",)])
def test_source(monkeypatch, gone):
    import torch
    from hierarchical_sparse_attention_hisa_b200 import _lib
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0x1000 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("S", (), {"cuda_stream": 0x2000})())
    for n in gone:
        monkeypatch.delattr(torch._C, n)
    assert _lib._stream_source()() == (0x2000 if gone else 0x1003)


@pytest.mark.gpu
def test_is_the_current_stream():
    import torch
    from hierarchical_sparse_attention_hisa_b200 import _lib
    side = torch.cuda.Stream()
    assert _lib._s(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert _lib._s(None) == side.cuda_stream
