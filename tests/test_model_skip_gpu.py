"""SketchModel on a Mamba-2 layer with step sizes: h <- exp(dt A) h + B (dt x)^T, y = C^T h + D x, keys and queries
shared by several heads, so that dt can only sit in the layer's v = dt x while the skip takes x.

Tolerance: y's 1e-4 of a slab's largest value, twice through a norm that keeps relative sizes, and the rounding to
bf16."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ragged_reference as ref  # noqa: E402


@pytest.mark.timeout(300)
def test_step_sizes_and_skip():
    import numpy as np
    from rank_state_read_amd.layer import SketchLayer
    from rank_state_read_amd.model import SketchModel
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lens, steps, B, H, Hk, V = [40, 75], 20, 2, 16, 4, 80
    L = SketchLayer(B=B, H=H, K=128, V=V, W=16, G=1, basis_rows=79, rank_cap=49, kind="mamba2", qkv="bf16",
                    rank=np.zeros(H, np.int32), group=np.zeros(H, np.int32), basis=np.zeros((1, 79, 128), np.float32),
                    kq_heads=Hk)
    full = [n + steps for n in lens]
    d = ref.draw("mamba2", "bf16", full, H, Hk, V, seed=50)
    g = torch.Generator().manual_seed(51)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    T = sum(full)
    dt, A, D = torch.nn.functional.softplus(rn(T, H) - 2), -torch.exp(rn(H)), rn(H)
    x, z = rn(T, H, V).to(torch.bfloat16), rn(T, H, V).to(torch.bfloat16)
    d.update(a=torch.exp(dt * A), v=(dt[:, :, None] * x.float()).to(torch.bfloat16), x=x, z=z)
    w = 1 + 0.2 * rn(H, V)
    L.set_norm(w, 4, "silu_first", D=D)
    model = SketchModel([L])
    y = ref.run("mamba2", d, full, torch.zeros(B, H, 128, V, device="cuda"))[0]
    want = ref.norm(y, x, D, z, w, 4, "silu_first", 1e-5)
    off = d["offsets"].tolist()

    def take(idx):
        return {key: None if d[key] is None else d[key][idx].contiguous() for key in ("q", "k", "v", "a", "beta", "x", "z")}

    prompt = torch.cat([torch.arange(off[b], off[b] + n) for b, n in enumerate(lens)]).cuda()
    offsets = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
    bar = 2e-4 + 2.0 ** -8
    got = model.prefill([take(prompt)], offsets, max(lens))[0]
    assert ref.slab_err(got, want[prompt]) <= bar
    for t in range(steps):
        idx = torch.tensor([off[b] + n + t for b, n in enumerate(lens)]).cuda()
        got = model.decode_step([take(idx)])[0]
        assert ref.slab_err(got, want[idx]) <= bar, t
