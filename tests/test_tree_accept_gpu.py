"""Accepted paths of drafted trees in the window: bit for bit the tokens, in order, behind the held-back ones, nothing
else touched, and positions of every row."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import tree_reference as ref  # noqa: E402

W = 16
WINDOW = [("kbuf", "k"), ("vbuf", "v"), ("abuf", "a"), ("bbuf", "beta")]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rank_state_read_amd import binding
    binding.lib()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _bits(x):
    return x.view({2: torch.int16, 4: torch.int32}[x.element_size()])


def accept(d, B, H, V, qkv, Hk, rows, accepted, pos, **kw):
    from rank_state_read_amd import sketchssm_tree_accept
    new = torch.full((B,), -99, dtype=torch.int32, device="cuda")
    sketchssm_tree_accept(ref.shape_of(B, H, V, d["kind"], qkv, Hk), d["kbuf"], d["vbuf"], d["abuf"], d["bbuf"], pos, new,
                          rows, d["offsets"], d["parents"], accepted, d["k"], d["v"], d["a"], d["beta"], **kw)
    return new


def _expect(d, rows, taken, pos):
    """(window, positions) after the call, by the definition."""
    win = {b: d[b].clone() for b, _ in WINDOW if d[b] is not None}
    pos, off = list(pos), d["offsets"].tolist()
    for i, row in enumerate(rows):
        if not 0 <= taken[i] < len(d["par"][i]) or not 0 <= row < len(pos):
            continue
        p = ref.path(d["par"][i], taken[i])
        if not 0 <= pos[row] <= W or pos[row] + len(p) > W:
            continue
        for m in p:
            for b, t in WINDOW:
                if d[b] is not None:
                    win[b][pos[row], :, row] = d[t][off[i] + m]
            pos[row] += 1
    return win, pos


def check(kind, qkv, sizes, H, Hk, V, how="tree", seed=0, held=None, taken=None, rows="shuffled"):
    n = len(sizes)
    B = n + 3
    order = [(5 * i + 1) % B if B % 5 else (7 * i + 1) % B for i in range(n)]
    held = [(3 * b + 5) % 13 for b in range(B)] if held is None else held
    d = ref.draw(kind, qkv, sizes, B, H, Hk, V, [0] * H, held, seed, how, 3, 5)
    if rows is None:
        order = list(range(n))
    taken = [(7 * i + 3) % s if s else -1 for i, s in enumerate(sizes)] if taken is None else taken
    win, pos = _expect(d, order, taken, held)
    print(f"  {kind} {qkv} {H}/{Hk} V={V} {how} {sizes} held={held} taken={taken}", flush=True)
    new = accept(d, B, H, V, qkv, Hk, None if rows is None else _i32(order), _i32(taken), _i32(held))
    torch.cuda.synchronize()
    assert new.tolist() == pos
    for b, x in win.items():
        assert torch.equal(_bits(d[b]), _bits(x)), b


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", ["mamba2", "gdn", "kda"])
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("V", [64, 80, 112, 128])
def test_widths_and_types(V, qkv, kind):
    check(kind, qkv, [13, 1, 0, 64, 7], 6, 3, V)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("H,Hk", [(1, 1), (8, 1), (9, 9), (40, 5), (128, 8)])
@pytest.mark.parametrize("how", ["chain", "star", "comb"])
def test_heads_and_trees(how, H, Hk):
    check("gdn", "bf16", [3, 16, 5, 11], H, Hk, 80, how)


def test_rows_in_order():
    check("kda", "bf16", [4, 9], 4, 2, 96, rows=None)


def test_what_is_not_accepted():
    """None, a node that is not there, a path that does not fit, a full window, bad positions, rows and parents."""
    check("gdn", "bf16", [5, 5, 5, 5, 5, 5, 5], 4, 4, 64, "chain", held=[0, 14, 16, 12, 17, -1, 3, 11, 11, 2],
          taken=[-1, 5, 2, 4, 0, 3, 4])


def test_bad_lists():
    sizes, B, H = [4, 4, 4, 4], 6, 4
    d = ref.draw("mamba2", "bf16", sizes, B, H, 2, 80, [0] * H, [2] * B, 1, "chain")
    d["parents"][5], d["parents"][10], d["parents"][14] = 1, -2, 99  # of its own index, below -1, past the end
    before = {b: d[b].clone() for b, _ in WINDOW if d[b] is not None}
    new = accept(d, B, H, 80, "bf16", 2, _i32([0, 1, 2, 3]), _i32([3, 3, 3, 3]), _i32([2] * B))
    assert new.tolist() == [6, 2, 2, 2, 2, 2]
    for b in before:
        before[b][2:6, :, 0] = d[dict(WINDOW)[b]][:4]
        assert torch.equal(_bits(d[b]), _bits(before[b])), b
    new = accept(d, B, H, 80, "bf16", 2, _i32([-1, 6, 1 << 30, -(1 << 31)]), _i32([0, 0, 0, 0]), _i32([2] * B))
    assert new.tolist() == [2] * B
    for off in ([0, 17, 4, -3, 16], [-4, 0, 0, 0, 0], [16, 20, 1 << 30, 4, 4]):
        d["offsets"] = _i32(off)
        assert accept(d, B, H, 80, "bf16", 2, None, _i32([0] * 4), _i32([2] * B)).tolist()[1:] == [2] * (B - 1)
    for b in before:
        assert torch.equal(_bits(d[b][:, :, 1:]), _bits(before[b][:, :, 1:])), b


def test_no_sequences():
    d = ref.draw("gdn", "bf16", [], 3, 2, 2, 64, [0, 0], [1, 2, 3])
    assert accept(d, 3, 2, 64, "bf16", 2, _i32([]), _i32([]), _i32([1, 2, 3])).tolist() == [1, 2, 3]
