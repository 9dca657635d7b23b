"""Rows' flush beside the calls that lead to it: a load of cached states switches to its tensors' device, and so does the
flush that forms the loaded rows' sketches (no GPU needed: only which device is current at the call is looked at)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd import binding as B  # noqa: E402


class _Tensor:
    """What the binding looks at of a device tensor."""
    is_cuda = True

    def __init__(self, index):
        self.device = torch.device("cuda", index)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


class _Stream:
    cuda_stream = 77

    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.fixture
def calls(monkeypatch):
    current, log = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        yield
        current[0] = before

    class Lib:
        @staticmethod
        def sketchssm_flush_seq(*args):
            log.append((current[0], args[-1]))
            return 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(B, "lib", lambda: Lib)
    return log


def _flush(index, stream=None):
    class Plan:
        handle = 1
    t = _Tensor(index)
    B.sketchssm_flush_seq(Plan, t, None, None, t, t, t, None, t, t, 2, stream)


def test_the_tensors_device_is_current(calls):
    for index in (0, 1):
        _flush(index)
    assert calls == [(0, 100), (1, 101)]


def test_given_streams(calls):
    _flush(1, _Stream(1))
    _flush(1, 5)
    assert calls == [(1, 77), (1, 5)]
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        _flush(1, _Stream(0))
    assert len(calls) == 2


def test_addresses(calls):
    class Plan:
        handle = 1
    B.sketchssm_flush_seq(Plan, *[1 << 20] * 9, 2, None)
    assert calls == [(0, 100)]
