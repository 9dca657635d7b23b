"""Trees of drafted tokens over sketches, states and windows against the definition in 64 bits: every node's state is
its parent's with one token applied.

Tolerance 1e-4 of a slab's largest value, a slab being one node's y of one head (the bar of every read of this
library): an fp32 sum over K = 128 channels is off by at most (K + 2) 2^-24 = 7.7e-6 of the sum of its terms'
magnitudes, which for independent terms is about sqrt(K) times the result: 8.8e-5."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ragged_reference as rr  # noqa: E402
import tree_reference as ref  # noqa: E402

TOL = 1e-4
KINDS = ["mamba2", "gdn", "kda"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rank_state_read_amd import binding
    binding.lib()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _plan(d, B, H, V, qkv, Hk):
    from rank_state_read_amd import Plan
    return Plan(ref.shape_of(B, H, V, d["kind"], qkv, Hk), d["ranks"], d["groups"])


def _read(plan, d, rows, y, max_nodes=None, **kw):
    from rank_state_read_amd import sketchssm_tree_read
    sketchssm_tree_read(plan, d["S"], d["Z"], d["frames"], d["kbuf"], d["vbuf"], d["abuf"], d["bbuf"], d["pos"],
                        None if rows is None else _i32(rows), d["offsets"],
                        max(d["sizes"]) if max_nodes is None else max_nodes, d["parents"], d["q"], d["k"], d["v"], d["a"],
                        d["beta"], y, **kw)


RANKS = {"dense": [0], "sketch": [6], "mixed": [0, 6, 17, 1, 49, 0, 33, 64]}


def _check(kind, qkv, sizes, H=4, Hk=2, V=128, ranks="mixed", held=None, seed=0, how="tree", edit=None):
    n = len(sizes)
    B = n + 3
    rows = [(5 * i + 1) % B if B % 5 else (7 * i + 1) % B for i in range(n)]
    held = [(3 * b + 5) % 17 for b in range(B)] if held is None else [held] * B
    rk = (RANKS[ranks] * H)[:H]
    lead, tail = 3, 5
    d = ref.draw(kind, qkv, sizes, B, H, Hk, V, rk, held, seed, how, lead, tail)
    if edit:
        edit(d)
    y = torch.full(d["v"].shape, 9.0, device="cuda")
    print(f"  {kind} {qkv} V={V} H={H}/{Hk} {ranks} {how} sizes={sizes} held={held}", flush=True)
    _read(_plan(d, B, H, V, qkv, Hk), d, rows, y)
    torch.cuda.synchronize()
    e = rr.slab_err(y[lead:lead + sum(sizes)], ref.read(d, rows)[lead:lead + sum(sizes)])
    print(f"    {e:.2e}", flush=True)
    assert e <= TOL
    assert (y[:lead] == 9).all() and (y[lead + sum(sizes):] == 9).all(), "y of nodes outside the sequences"
    return d, rows, y


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ranks", ["dense", "sketch", "mixed"])
@pytest.mark.parametrize("sizes", [[1], [0, 1, 2, 0], [3, 4, 5], [7, 8, 9], [15, 16, 17], [31, 32, 33, 1], [63, 64, 1]],
                         ids=str)
def test_sizes(sizes, ranks, kind):
    _check(kind, "bf16", sizes, ranks=ranks)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [64, 80, 96, 112, 128])
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("big", [13, 20, 47])
def test_widths_and_types(big, qkv, V, kind):
    _check(kind, qkv, [big, 2], V=V, H=5, Hk=5, seed=V)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,Hk", [(1, 1), (8, 1), (12, 4), (16, 2)])
@pytest.mark.parametrize("ranks", ["dense", "mixed"])
def test_head_groups(ranks, H, Hk, kind):
    _check(kind, "bf16", [11, 6], H=H, Hk=Hk, V=80, ranks=ranks)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("held", [0, 1, 15, 16])
@pytest.mark.parametrize("how", ["chain", "star", "comb"])
def test_windows_and_shapes_of_trees(how, held, kind):
    _check(kind, "bf16", [1, 16, 30], V=96, held=held, how=how)


# -- values that must not reach a node, degenerate tokens ---------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ranks", ["dense", "sketch"])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("key", ["q", "k", "v", "a"])
def test_other_branches_do_not_reach_a_node(key, what, ranks, kind):
    """A value of one node reaches that node and those below it alone; nodes on other paths keep their bits."""
    sizes, B, H, Hk, V = [17, 40], 4, 4, 2, 80
    d = ref.draw(kind, "bf16", sizes, B, H, Hk, V, (RANKS[ranks] * H)[:H], [3, 0, 16, 9], 5)
    plan = _plan(d, B, H, V, "bf16", Hk)
    y = torch.zeros(d["v"].shape, device="cuda")
    _read(plan, d, [3, 1], y)
    for node in (0, 5, 16):
        e = dict(d, **{key: d[key].clone()})
        e[key][node] = what
        z = torch.zeros_like(y)
        _read(plan, e, [3, 1], z)
        torch.cuda.synchronize()
        hit = [n for n in range(17) if node in ref.path(d["par"][0], n)] if key != "q" else [node]
        keep = [n for n in range(57) if n not in hit]
        assert torch.equal(z[keep], y[keep])
        if key != "a":  # (a decay of a first token is never used where nothing stands before it)
            assert not z[hit].isfinite().all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("a", [0.0, 1.0, -0.5, 1e-30])
def test_decays(a, kind):
    def edit(d):
        d["a"][3:9] = a
        d["abuf"][1] = a
    _check(kind, "bf16", [14, 7], held=5, how="chain", edit=edit)


@pytest.mark.parametrize("kind", KINDS)
def test_zero_tokens(kind):
    def edit(d):
        d["q"][4], d["k"][5], d["v"][6] = 0, 0, 0
        if d["beta"] is not None:
            d["beta"][7] = 0
    d, rows, y = _check(kind, "bf16", [14, 7], how="chain", edit=edit)
    assert (y[4] == 0).all()


# -- lists ----------------------------------------------------------------------------------------------------
def test_rows_in_order_and_without_windows():
    sizes, H, V = [5, 0, 20], 4, 128
    for kind in KINDS:
        d = ref.draw(kind, "bf16", sizes, 4, H, 2, V, RANKS["mixed"][:H], [0] * 4, 3)
        e = dict(d, kbuf=None, vbuf=None, abuf=None, bbuf=None, pos=None)
        y, z = (torch.zeros(d["v"].shape, device="cuda") for _ in range(2))
        plan = _plan(d, 4, H, V, "bf16", 2)
        _read(plan, d, None, y)
        _read(plan, e, None, z)
        assert rr.slab_err(y, ref.read(d, [0, 1, 2])) <= TOL and torch.equal(y, z)


def test_several_trees_of_one_row_and_a_loose_bound():
    sizes = [9, 12, 3]
    d = ref.draw("gdn", "bf16", sizes, 2, 4, 4, 96, RANKS["mixed"][:4], [7, 12], 8)
    y, z = (torch.zeros(d["v"].shape, device="cuda") for _ in range(2))
    plan = _plan(d, 2, 4, 96, "bf16", 4)
    _read(plan, d, [1, 1, 0], y)
    _read(plan, d, [1, 1, 0], z, max_nodes=64)
    r = ref.read(d, [1, 1, 0])
    assert rr.slab_err(y, r) <= TOL and rr.slab_err(z, r) <= TOL


def test_sequences_out_of_order_of_their_nodes():
    """The second sequence's nodes stand before the first's, an idle entry between them."""
    d = ref.draw("kda", "bf16", [6, 9], 3, 4, 2, 64, RANKS["mixed"][:4], [4, 8, 16], 2)
    y = torch.zeros(d["v"].shape, device="cuda")
    plan = _plan(d, 3, 4, 64, "bf16", 2)
    e = dict(d, offsets=_i32([6, 15, 0, 6]))
    _read(plan, e, [2, 1, 0], y, max_nodes=9)
    assert rr.slab_err(y, ref.read(d, [0, 2])) <= TOL


def test_bad_lists_idle_what_they_name():
    sizes, B, H, V = [4, 4, 4, 4], 4, 4, 80
    d = ref.draw("gdn", "bf16", sizes, B, H, 2, V, RANKS["mixed"][:H], [2, 3, 4, 5], 1, "chain")
    plan = _plan(d, B, H, V, "bf16", 2)
    good = torch.full(d["v"].shape, 9.0, device="cuda")
    _read(plan, d, [0, 1, 2, 3], good)

    def check(idle, rows=(0, 1, 2, 3), max_nodes=4, **edit):
        y = torch.full(d["v"].shape, 9.0, device="cuda")
        _read(plan, dict(d, **edit), list(rows), y, max_nodes=max_nodes)
        torch.cuda.synchronize()
        keep = [n for n in range(16) if n not in idle]
        assert torch.equal(y[keep], good[keep]) and (y[list(idle)] == 9).all()

    check(())
    check(range(4, 8), rows=(0, 4, 2, 3))
    check(range(8, 12), rows=(0, 1, -1, 3))
    check(range(0, 4), rows=(-(1 << 31), 1, 2, 3))
    check(range(4, 8), pos=_i32([2, 17, 4, 5]))
    check(range(4, 8), pos=_i32([2, -1, 4, 5]))
    check(range(4, 8), pos=_i32([2, 1 << 30, 4, 5]))
    check(range(16), max_nodes=3)
    check(range(12, 16), offsets=_i32([0, 4, 8, 12, 17]))
    check(range(0, 4), offsets=_i32([-4, 4, 8, 12, 16]))
    for bad in (1, 2, 63, 64, 1 << 30, -2, -(1 << 31)):  # the parent of node 1 of the second sequence: it, and those below
        par = d["parents"].clone()
        par[5] = bad
        check(range(5, 8), parents=par)
    par = d["parents"].clone()
    par[4] = 0  # a node that is its own parent
    check(range(4, 8), parents=par)


def test_nothing_to_do():
    d = ref.draw("gdn", "bf16", [0, 0], 2, 2, 2, 64, [0, 3], [1, 2])
    y = torch.zeros(d["v"].shape, device="cuda")
    _read(_plan(d, 2, 2, 64, "bf16", 2), d, [0, 1], y)


# -- beside the decode reads ------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
def test_a_single_node_is_a_decode_read(kind):
    from rank_state_read_amd import sketchssm_decode_read_seq
    B, H, Hk, V = 5, 6, 3, 80
    d = ref.draw(kind, "bf16", [1] * B, B, H, Hk, V, RANKS["mixed"][:H], [0, 3, 15, 8, 11], 4)
    plan = _plan(d, B, H, V, "bf16", Hk)
    y, z = (torch.zeros(d["v"].shape, device="cuda") for _ in range(2))
    _read(plan, d, None, y)
    sketchssm_decode_read_seq(plan, d["S"], d["Z"], d["frames"], d["q"], d["k"], d["v"], d["a"], d["beta"], d["kbuf"],
                              d["vbuf"], d["abuf"], d["bbuf"], d["pos"], z)
    assert rr.slab_err(y, z) <= 2 * TOL  # both within TOL of the definition


@pytest.mark.parametrize("kind", KINDS)
def test_same_bits_again_and_beside_others(kind):
    """A tree's outputs do not depend on the other sequences of the call."""
    sizes = [12, 33, 5]
    d = ref.draw(kind, "bf16", sizes, 3, 4, 2, 128, RANKS["mixed"][:4], [9, 2, 16], 6)
    plan = _plan(d, 3, 4, 128, "bf16", 2)
    y, z = (torch.zeros(d["v"].shape, device="cuda") for _ in range(2))
    _read(plan, d, [0, 1, 2], y, max_nodes=33)
    _read(plan, d, [0, 1, 2], z, max_nodes=33)
    assert torch.equal(y, z)
    alone = dict(d, offsets=_i32([12, 45]))
    z.zero_()
    _read(plan, alone, [1], z, max_nodes=33)
    assert torch.equal(y[12:45], z[12:45]) and (z[:12] == 0).all() and (z[45:] == 0).all()
