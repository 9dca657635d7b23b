"""A row that held tokens back starts again from a cached state: its position is the caller's, 0 after the load, and
nothing of the row's window before reaches it then."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import tree_reference as ref  # noqa: E402

K, W = ref.K, ref.W


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", ["mamba2", "gdn", "kda"])
def test_a_row_that_held_tokens(kind):
    """Row 2 holds 11 tokens when row 0's state is loaded to it.  Read from position 0 it has the bits of a row whose
    window is empty; read at its old position it has not, so the position does matter."""
    import numpy as np
    from rank_state_read_amd.layer import SketchLayer
    from rank_state_read_amd.model import SketchModel
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B, H, V, ranks = 4, 4, 80, [0, 6, 17, 0]
    g = np.random.default_rng(1)
    basis = np.stack([np.linalg.qr(g.standard_normal((K, 79)))[0].T for _ in range(2)]).astype(np.float32)
    lay = SketchLayer(B=B, H=H, K=K, V=V, W=W, G=2, basis_rows=79, rank_cap=64, kind=kind, qkv="bf16", rank=ranks,
                      group=[0, 0, 1, 1], basis=basis, fmap=lambda gr, r: basis[gr, :r], kq_heads=2)
    m = SketchModel([lay])
    held = [0, 0, 11, 0]
    d = ref.draw(kind, "bf16", [9, 9], B, H, 2, V, ranks, held, 3)
    for key in ("S", "kbuf", "vbuf", "abuf", "bbuf"):
        if d[key] is not None:
            getattr(lay, key).copy_(d[key])
    for key in ("q", "k", "v", "a", "beta"):  # both rows read the same tree
        if d[key] is not None:
            d[key][9:] = d[key][:9]
    d["parents"][9:] = d["parents"][:9]
    m.start()
    pos, rows = _i32(held), _i32([2, 3])
    cache = m.new_cache(1)
    m.cache_store(cache, _i32([0]), _i32([0]))
    m.cache_load(cache, _i32([0, 0]), rows)

    def read():
        y = m.tree_read([d], d["parents"], d["offsets"], 9, pos=pos, rows=rows)[0]
        torch.cuda.synchronize()
        return y[:9], y[9:]

    a, b = read()
    assert not torch.equal(a, b)
    pos[rows.long()] = 0
    a, b = read()
    assert torch.equal(a, b) and bool(a.isfinite().all())
