"""Streams and workspaces of another device than the tensors' are refused before anything is launched (no GPU
needed: the check comes before the device is asked for)."""
import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd import binding as B  # noqa: E402


class _Stream:
    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_stream_of_another_device():
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        B._on_device(torch.device("cuda", 0), _Stream(1))


def test_host_tensors():
    with pytest.raises(ValueError, match="device tensor"):
        B._on_device(torch.device("cpu"), None)
