"""A layer made on "cuda" stays on the device that was current then, for what its calls allocate later too."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_layer_keeps_its_device():
    import numpy as np
    from rank_state_read_amd.layer import SketchLayer
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L = SketchLayer(B=1, H=2, K=128, V=64, W=16, G=1, basis_rows=79, rank_cap=49, kind="gdn", qkv="bf16",
                    rank=np.zeros(2, np.int32), group=np.zeros(2, np.int32), basis=np.zeros((1, 79, 128), np.float32))
    assert L.device == L.S.device == torch.device("cuda", torch.cuda.current_device())
