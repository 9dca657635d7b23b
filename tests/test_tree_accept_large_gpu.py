"""Accepted paths in trees of more nodes than are read at once: an accepted node far behind the first 256, with parents on
both sides of it, and a parent there that is none."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import tree_reference as ref  # noqa: E402
from test_tree_accept_gpu import WINDOW, _bits, _expect, _i32, accept  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rank_state_read_amd import binding
    binding.lib()


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", ["mamba2", "gdn", "kda"])
@pytest.mark.parametrize("bad", [None, 280, 256, 255])
def test_behind_256_nodes(bad, kind):
    sizes, B, H, Hk, V, held = [300, 3, 257], 4, 9, 3, 80, [2, 0, 5, 1]
    d = ref.draw(kind, "bf16", sizes, B, H, Hk, V, [0] * H, held, 4, "tree", 2, 1)
    for child, parent in zip([299, 280, 256, 255, 100, 7, 0], [280, 256, 255, 100, 7, 0, -1]):
        d["par"][0][child] = parent
    d["parents"][2:302] = _i32(d["par"][0])
    taken = [299, 2, 256]
    rows = [3, 0, 2]
    if bad is not None:  # that node's parent is none: nothing of the first tree is accepted
        d["parents"][2 + bad] = bad
    win, pos = _expect(d, rows, [taken[0] if bad is None else -1] + taken[1:], held)
    assert pos[3] == (8 if bad is None else 1)
    new = accept(d, B, H, V, "bf16", Hk, _i32(rows), _i32(taken), _i32(held))
    torch.cuda.synchronize()
    assert new.tolist() == pos
    for b, _ in WINDOW:
        if d[b] is not None:
            assert torch.equal(_bits(d[b]), _bits(win[b])), b
