"""CPU checks of the streams that the layer products and dropout take, and of
what their documentation says of streams and autograd."""
import pytest


def test_the_per_thread_stream_is_refused(monkeypatch):
    """hipStreamPerThread is another stream in every host thread, but one stream to the
    allocator that a call takes its memory from: refused as a handle, as an object and as
    the current stream, as the norm refuses it."""
    import torch

    import optimizer_muon_step_amd as mu
    x, w, y = torch.zeros(4, 8).bfloat16(), torch.zeros(8, 16).bfloat16(), torch.zeros(4, 16).bfloat16()
    calls = [lambda **s: mu.muon_linear(x, w, **s), lambda **s: mu.muon_linear_dx(y, w, **s),
             lambda **s: mu.muon_linear_dw(x, y, torch.zeros(8, 16), **s), lambda **s: mu.muon_dropout(x, 0.1, (1, 2), **s)]
    for call in calls:
        with pytest.raises(ValueError, match="hipStreamPerThread"):
            call(stream=2)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 2)
    for call in calls:
        with pytest.raises(ValueError, match="hipStreamPerThread"):
            call()
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    for call in calls:  # another stream: what is wrong is that the tensors are on the CPU
        with pytest.raises(ValueError, match="on the GPU"):
            call()


def test_the_documentation_names_streams_and_autograd():
    import optimizer_muon_step_amd as mu
    for call in (mu.muon_linear, mu.muon_linear_dx, mu.muon_linear_dw, mu.muon_dropout):
        text = " ".join(call.__doc__.split())
        assert "No autograd graph is recorded" in text and "`stream`" in text, call.__name__
