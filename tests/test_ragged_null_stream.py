"""The null stream's handle is 0, which torch.cuda.ExternalStream takes for "no handle given": it hands out a stream of
its pool then.  What a call on handle 0 allocates has to belong to the default stream all the same, else memory that
queued work still uses could go to others.  (No GPU needed: only which stream is asked for is looked at.)"""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd import binding as B  # noqa: E402

DEV = torch.device("cuda", 0)


@pytest.fixture
def asked(monkeypatch):
    log = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))

    @contextlib.contextmanager
    def current(stream):
        log.append(stream)
        yield
    monkeypatch.setattr(torch.cuda, "stream", current)
    return log


def test_null_stream_is_the_default_stream(asked):
    with B.owned_by(0, DEV):
        pass
    assert asked == [("default", DEV)]


def test_other_handles(asked):
    with B.owned_by(4096, DEV), B.owned_by("a stream object", DEV), B.owned_by(None, DEV):
        pass
    assert asked == [("external", 4096, DEV), "a stream object"]


@pytest.mark.gpu
def test_memory_of_a_call_on_the_null_stream():
    """The same as seen by torch, and a prompt call with handle 0 of a side stream's thread of work."""
    import ragged_reference as ref
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side), B.owned_by(0, DEV):
        assert torch.cuda.current_stream().cuda_stream == 0
    import numpy as np
    from rank_state_read_amd.layer import SketchLayer
    lens, H, V = [70, 33], 4, 64
    d = ref.draw("gdn", "bf16", lens, H, H, V, seed=70)
    L = SketchLayer(B=2, H=H, K=128, V=V, W=16, G=1, basis_rows=79, rank_cap=49, kind="gdn", qkv="bf16",
                    rank=np.zeros(H, np.int32), group=np.zeros(H, np.int32), basis=np.zeros((1, 79, 128), np.float32))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y = L.prefill(d["offsets"], 70, d["q"], d["k"], d["v"], d["a"], d["beta"], stream=0)
        torch.empty(1 << 22, device="cuda").fill_(float("nan"))
    torch.cuda.synchronize()
    yr, Sr = ref.run("gdn", d, lens, torch.zeros(2, H, 128, V, device="cuda"))
    assert ref.slab_err(y, yr) <= 1e-4 and ref.slab_err(L.S, Sr) <= 1e-4
