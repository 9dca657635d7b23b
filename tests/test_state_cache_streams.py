"""A cache of states is made for calls on a stream: its memory belongs to that stream, and its zeros are written before
any store, on whatever stream that is."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd import layer as L  # noqa: E402
from rank_state_read_amd.model import SketchModel  # noqa: E402


def test_memory_belongs_to_the_stream(monkeypatch):
    """Both arrays are taken, and zeroed, inside the context of the stream that the calls will be on."""
    inside, seen = [], []

    @contextlib.contextmanager
    def owned_by(stream, device):
        inside.append((stream, device))
        yield
        inside.pop()

    zeros = torch.zeros

    def recorded(*a, **kw):
        seen.append(inside[-1] if inside else None)
        return zeros(*a, **kw)

    monkeypatch.setattr(L._b, "owned_by", owned_by)
    monkeypatch.setattr(torch, "zeros", recorded)
    c = L.StateCache(3, 2, 128, 64, "i8", device="cpu", stream="s")
    assert seen == [("s", torch.device("cpu"))] * 2 and not c.codes.any() and not c.scales.any()


def test_a_layer_and_a_model_pass_the_stream_on():
    class Layer:
        W = 16

        def new_cache(self, n, fmt, stream=None):
            return n, fmt, stream

    assert SketchModel([Layer(), Layer()]).new_cache(4, "i8", stream=7) == [(4, "i8", 7)] * 2


@pytest.mark.gpu
@pytest.mark.timeout(300)
@pytest.mark.parametrize("given", [False, True])
def test_a_store_outlives_the_zeros(given):
    """The stream that the cache is made on is behind with its work; the store runs on another one."""
    import numpy as np
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lay = L.SketchLayer(B=4, H=32, K=128, V=128, W=16, G=1, basis_rows=79, rank_cap=49, kind="gdn", qkv="bf16",
                        rank=np.zeros(32, np.int32), group=np.zeros(32, np.int32),
                        basis=np.zeros((1, 79, 128), np.float32))
    lay.S.copy_(torch.randn(lay.S.shape, generator=torch.Generator().manual_seed(1)))
    want = lay.new_cache(4)
    lay.cache_store(want)
    big, s = torch.zeros(8192, 8192, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        big = big @ big
    cache = lay.new_cache(4, stream=s) if given else lay.new_cache(4)
    lay.cache_store(cache, stream=s)
    torch.cuda.synchronize()
    assert cache.codes.any() and torch.equal(cache.codes, want.codes) and torch.equal(cache.scales, want.scales)
