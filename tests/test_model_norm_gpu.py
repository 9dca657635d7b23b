"""A model's layer whose norm has no gate: normed outputs of prompts and of decode steps, against the formula in 64
bits (tolerance: y's 1e-4 of a slab's largest value, twice through the norm, and the rounding to bf16)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ragged_reference as ref  # noqa: E402


@pytest.mark.timeout(300)
@pytest.mark.parametrize("skip", [False, True])
def test_norm_without_gate(skip):
    import numpy as np
    from rank_state_read_amd.layer import SketchLayer
    from rank_state_read_amd.model import SketchModel
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    n, steps, H, V = 33, 3, 8, 64
    L = SketchLayer(B=1, H=H, K=128, V=V, W=16, G=1, basis_rows=79, rank_cap=49, kind="gdn", qkv="bf16",
                    rank=np.zeros(H, np.int32), group=np.zeros(H, np.int32), basis=np.zeros((1, 79, 128), np.float32))
    d = ref.draw("gdn", "bf16", [n + steps], H, H, V, seed=60)
    g = torch.Generator().manual_seed(61)
    w, D = 1 + 0.2 * torch.randn(V, generator=g).cuda(), torch.randn(H, generator=g).cuda() if skip else None
    L.set_norm(w, 1, "none", D=D)
    y = ref.run("gdn", d, [n + steps], torch.zeros(1, H, 128, V, device="cuda"))[0]
    want = ref.norm(y, d["v"] if skip else None, D, None, w, 1, "none", 1e-5)
    take = lambda a, b: {key: d[key][a:b].contiguous() for key in ("q", "k", "v", "a", "beta")}  # noqa: E731
    model = SketchModel([L])
    offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    got = [model.prefill([take(0, n)], offsets, n)[0]]
    got += [model.decode_step([take(t, t + 1)])[0] for t in range(n, n + steps)]
    got = torch.cat(got)
    assert got.dtype == torch.bfloat16 and ref.slab_err(got, want) <= 2e-4 + 2.0 ** -8
