"""The package's own workspaces, for calls that are given none (no GPU)."""
import pytest
import torch

DEV = torch.device("cuda:0")


@pytest.fixture
def w8(monkeypatch):
    import bit_quantized_gemm_token_amd as mod
    monkeypatch.setattr(mod, "_workspaces", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return mod


def test_each_stream_has_its_own(w8):
    """Calls that share counters and partials must not overlap, and calls on
    two streams may."""
    a, b = (w8._default_workspace(DEV, stream) for stream in (0x1000, 0x2000))
    assert a is not b
    assert w8._default_workspace(DEV, 0x1000) is a and w8._default_workspace(DEV, 0x2000) is b
    assert w8._default_workspace(torch.device("cuda:1"), 0x1000) is not a


def test_a_capture_takes_one_that_is_there(w8, monkeypatch):
    """Where the stream's own is missing or too small: the largest on the
    device, none of another device's; and where there is none that is large
    enough the Workspace refuses to grow."""
    for stream, nbytes in ((0x1000, 256), (0x2000, 4096), (0x3000, 1024)):
        w8._default_workspace(DEV, stream).buf = torch.zeros(nbytes, dtype=torch.uint8)
    w8._default_workspace(torch.device("cuda:1"), 0x2000).buf = torch.zeros(8192, dtype=torch.uint8)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    new, small = w8._default_workspace(DEV, 0x9000), w8._default_workspace(DEV, 0x3000)
    assert new.reserve(512).numel() == 4096 and small.reserve(2048).numel() == 4096
    assert small.reserve(1024).numel() == 1024  # its own
    for w in (new, small, w8._default_workspace(torch.device("cuda:2"), 0x9000)):
        with pytest.raises(RuntimeError, match="capture"):
            w.reserve(8192)
    assert new.buf is None and small.buf.numel() == 1024  # (what was lent is not kept)
