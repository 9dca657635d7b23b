"""A layer's tree_read takes another plan only if that reads the state: the layer's sketch is its own plan's (no GPU needed:
the call is looked at, not made)."""
import pytest

torch = pytest.importorskip("torch")

import numpy as np  # noqa: E402

from rank_state_read_amd import layer as L  # noqa: E402


def test_plans_of_a_call(monkeypatch):
    lay = L.SketchLayer(B=2, H=4, K=128, V=64, W=16, G=1, basis_rows=79, rank_cap=49, kind="gdn", qkv="bf16",
                        rank=[0, 6, 7, 0], group=[0] * 4, basis=np.zeros((1, 79, 128), np.float32),
                        fmap=lambda g, r: np.zeros((r, 128), np.float32), device="cpu")
    seen = []
    monkeypatch.setattr(L._b, "sketchssm_tree_read", lambda plan, S, Z, frames, *a: seen.append((plan, S, Z, frames)))
    x = torch.zeros(3, 4, 64)
    args = (None, 3, None, x, x, x, x, x)
    lay.tree_read(*args, y=x)
    dense = L._b.Plan(lay.shape, [0] * 4, [0] * 4)
    lay.tree_read(*args, y=x, plan=dense)
    assert [s[0] for s in seen] == [lay.plan, dense]
    assert seen[0][2] is lay.Z and seen[0][3] is lay.frames and seen[1][2:] == (None, None)
    ranked = L._b.Plan(lay.shape, [0, 6, 8, 0], [0] * 4)
    with pytest.raises(ValueError, match="ranks"):
        lay.tree_read(*args, y=x, plan=ranked)
    assert len(seen) == 2
