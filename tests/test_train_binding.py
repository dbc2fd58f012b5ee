"""The binding of libmxfp4_train without a GPU: what train.py hands to the library, seen by a library that only records it."""
import contextlib

import pytest
import torch


class Recorder:
    """Stands in for the library: every call succeeds and is kept."""

    def __init__(self, need):
        self.need, self.calls = need, []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *sizes: self.need
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def recorded(monkeypatch):
    import mxfp4_block_scaled_h16_amd.train as train
    lib = Recorder(4096)
    monkeypatch.setattr(train, "train_lib", lambda: lib)
    monkeypatch.setattr(train, "_same_device", lambda **tensors: torch.device("cpu"))
    monkeypatch.setattr(train, "_on", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(train, "_current", lambda: 0)
    train._need.cache_clear()
    yield train, lib
    train._need.cache_clear()


def _calls(train, workspace):
    u8, bf = torch.uint8, torch.bfloat16
    q, s = torch.zeros(4, 128, dtype=u8), torch.zeros(4, 16, dtype=u8)
    x, w, target = torch.zeros(4, 64, dtype=bf), torch.zeros(8, 64, dtype=bf), torch.zeros(4, dtype=torch.int64)
    rows = torch.zeros(4)
    return [lambda: train.fp8_gemm(q, s, q, s, workspace=workspace),
            lambda: train.fp8_linear_fprop(x, w, workspace=workspace),
            lambda: train.fp8_linear_wgrad(x, x, workspace=workspace),
            lambda: train.linear_xent_forward(x, w, target, workspace=workspace),
            lambda: train.linear_xent_backward(rows, x, w, target, rows, workspace=workspace),
            lambda: train.orthogonalize(x, workspace=workspace)]


def test_a_workspace_counts_the_bytes_it_has(recorded):
    """A workspace that repeats or skips its bytes (expanded, strided) is refused: its number of elements says nothing
    about what lies behind its pointer."""
    train, lib = recorded
    whole = torch.zeros(8192, dtype=torch.uint8)
    for call in _calls(train, whole):
        call()
    assert len(lib.calls) == 6
    for name, args in lib.calls:
        at = args.index(whole.data_ptr())
        assert args[at + 1] == 8192, name
    lib.calls.clear()
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(8192), torch.zeros(16384, dtype=torch.uint8)[::2],
                torch.zeros(64, 1, dtype=torch.uint8).expand(64, 128)):
        for call in _calls(train, bad):
            with pytest.raises(ValueError, match="workspace must be contiguous"):
                call()
    assert not lib.calls
