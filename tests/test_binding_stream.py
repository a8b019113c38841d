"""The binding's handle of the current stream, with and without torch's private accessors (no GPU needed)."""

import types

import pytest

from decode_qwen3_decoder_gb300 import qw as binding


def test_current_stream_without_the_private_accessors(monkeypatch):
    import torch
    public = types.SimpleNamespace(cuda_stream=77)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: public)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
        monkeypatch.setattr(binding, "_current_stream", None)
        assert binding._stream(None) == 1003
        monkeypatch.delattr(torch._C, name)
        monkeypatch.setattr(binding, "_current_stream", None)
        assert binding._stream(None) == 77
        public.cuda_stream = 78
        assert binding._stream(None) == 78  # asked for at every call
        public.cuda_stream = 77
    assert binding._stream(5) == 5 and binding._stream(public) == 77


@pytest.mark.gpu
def test_current_stream_is_torchs(qw):
    import torch
    for st in (torch.cuda.default_stream(), torch.cuda.Stream(), torch.cuda.Stream(priority=-1)):
        with torch.cuda.stream(st):
            assert qw.qw._stream(None) == torch.cuda.current_stream().cuda_stream == st.cuda_stream
