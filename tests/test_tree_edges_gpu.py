"""Trees, accepted paths and cached states where addresses, lists and values are at their ends: rows and nodes behind
2^31 bytes, parents that are none in trees of several tiles, infinities in the state, the largest call in a graph."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ragged_reference as rr  # noqa: E402
import tree_reference as ref  # noqa: E402

K, W = ref.K, ref.W
KINDS = ["mamba2", "gdn", "kda"]
TOL = 1e-4  # per node and head, relative to its largest value, as for the decode reads


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


def _read(plan, d, rows, y, max_nodes=None):
    from rank_state_read_amd import sketchssm_tree_read
    sketchssm_tree_read(plan, d["S"], d["Z"], d["frames"], d["kbuf"], d["vbuf"], d["abuf"], d["bbuf"], d["pos"], rows,
                        d["offsets"], max(d["sizes"]) if max_nodes is None else max_nodes, d["parents"], d["q"], d["k"],
                        d["v"], d["a"], d["beta"], y)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("size", [13, 30, 61])
def test_parents_that_are_none(size, qkv, kind):
    """A node whose parent is not below it, and the nodes below that one, keep their y; the others have theirs."""
    sizes, H, V = [size, 5], 4, 96
    d = ref.draw(kind, qkv, sizes, 2, H, 2, V, [0, 6, 17, 0], [5, 16], size)
    plan = _plan(d, 2, H, V, qkv, 2)
    good = torch.full(d["v"].shape, 9.0, device="cuda")
    _read(plan, d, None, good)
    for node in (0, 1, size // 2, size - 1):
        below = {node}
        for n in range(size):
            if d["par"][0][n] in below:
                below.add(n)
        keep = [n for n in range(size + 5) if n not in below]
        for bad in (node, size, 64, 1 << 30, -2, -(1 << 31)):
            par = d["parents"].clone()
            par[node] = bad
            y = torch.full_like(good, 9.0)
            _read(plan, dict(d, parents=par), None, y)
            torch.cuda.synchronize()
            assert torch.equal(y[keep], good[keep]) and (y[sorted(below)] == 9).all(), (node, bad)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind,qkv,rank", [("mamba2", "bf16", 6), ("mamba2", "f32", 0), ("gdn", "bf16", 0), ("gdn", "f32", 9),
                                           ("kda", "f32", 0), ("kda", "bf16", 6)])
def test_rows_behind_two_gigabytes(kind, qkv, rank):
    """One head with the most rows that its arrays take: the last rows' states lie 8 GB, KDA's decays and float32 keys
    2 GB behind their arrays' starts.  Read, accepted into, stored and loaded they have a small call's bits."""
    from rank_state_read_amd import sketchssm_cache_load, sketchssm_cache_store, sketchssm_tree_accept
    sizes, V, B = [7, 33], 64, (1 << 18) - 1
    small = ref.draw(kind, qkv, sizes, 3, 1, 1, V, [rank], [4, 0, 9], 1)
    at = _i32([B - 1, B - 2, 5])  # where the small call's rows are
    big = dict(small, S=torch.zeros(B, 1, K, V, device="cuda"))
    big["S"][at.long()] = small["S"]
    if rank:
        big["Z"] = torch.zeros(B, rank, V, device="cuda")
        big["Z"][at.long()] = small["Z"].view(3, rank, V)
    for key in ("kbuf", "vbuf", "abuf", "bbuf"):
        if small[key] is not None:
            x = small[key]
            big[key] = torch.zeros((W, x.shape[1], B) + tuple(x.shape[3:]), dtype=x.dtype, device="cuda")
            big[key][:, :, at.long()] = x
    big["pos"] = torch.full((B,), 16, dtype=torch.int32, device="cuda")
    big["pos"][at.long()] = small["pos"]
    rows = _i32([0, 2])
    y, z = (torch.zeros(small["v"].shape, device="cuda") for _ in range(2))
    _read(_plan(small, 3, 1, V, qkv, 1), small, rows, y)
    _read(_plan(small, B, 1, V, qkv, 1), big, at[rows.long()].contiguous(), z)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and rr.slab_err(z, ref.read(small, [0, 2])) <= TOL
    # the accepted paths
    new, far = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    for dd, B_, r, n in ((small, 3, rows, new), (big, B, at[rows.long()].contiguous(), far)):
        sketchssm_tree_accept(ref.shape_of(B_, 1, V, kind, qkv, 1), dd["kbuf"], dd["vbuf"], dd["abuf"], dd["bbuf"], dd["pos"],
                              n, r, dd["offsets"], dd["parents"], _i32([3, 20]), dd["k"], dd["v"], dd["a"], dd["beta"])
    torch.cuda.synchronize()
    assert torch.equal(far[at.long()], new) and (new > small["pos"]).any()
    assert int((far != big["pos"]).sum()) == int((new != small["pos"]).sum())
    for key in ("kbuf", "vbuf", "abuf", "bbuf"):
        if small[key] is not None:
            assert torch.equal(big[key][:, :, at.long()].nan_to_num(7.0), small[key].nan_to_num(7.0)), key
            assert not bool(big[key][:, :, 6:B - 2].any()), key
    # states, to a slot more than 2^32 bytes behind the cache's start
    n_slots = (1 << 19) + 2
    codes = torch.zeros(n_slots, 1, K, V, dtype=torch.int8, device="cuda")
    scales = torch.zeros(n_slots, 1, K, dtype=torch.bfloat16, device="cuda")
    shape = ref.shape_of(B, 1, V, kind, qkv, 1)
    sketchssm_cache_store(shape, big["S"], at[:2].contiguous(), codes, scales, _i32([n_slots - 1, 0]), "i8")
    sketchssm_cache_load(shape, codes, scales, _i32([n_slots - 1]), big["S"], _i32([B - 3]), "i8")
    torch.cuda.synchronize()
    for slot, row in ((n_slots - 1, 0), (0, 1)):
        assert torch.equal(codes[slot].double() * scales[slot].double()[..., None], ref.quantised(small["S"][row], "i8")[1])
    assert torch.equal(big["S"][B - 3].double(), ref.quantised(small["S"][0], "i8")[1])
    assert not bool(codes[1:n_slots - 1].any()) and not bool(big["S"][6:B - 3].any())


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_nodes_behind_four_gigabytes(kind):
    """The last of very many nodes, alone in its sequence or in a tree."""
    H, Hk, V, sizes = 128, 1, 128, [1, 30]
    d = ref.draw(kind, "bf16", sizes, 2, H, Hk, V, ([0, 6, 17] * H)[:H], [3, 16], 2)
    T, n = 70000, 31
    plan = _plan(d, 2, H, V, "bf16", Hk)
    far = dict(d)
    for key in ("q", "k", "v", "a", "beta", "parents"):
        if d[key] is not None:
            far[key] = torch.zeros((T,) + tuple(d[key].shape[1:]), dtype=d[key].dtype, device="cuda")
            far[key][T - n:] = d[key]
    far["offsets"] = d["offsets"] + (T - n)
    y, z = torch.zeros(d["v"].shape, device="cuda"), torch.zeros(T, H, V, device="cuda")
    _read(plan, d, None, y)
    _read(plan, far, None, z)
    torch.cuda.synchronize()
    assert torch.equal(z[T - n:], y) and not bool(z[:T - n].any()) and rr.slab_err(y, ref.read(d, [0, 1])) <= TOL


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("what", [float("inf"), float("nan")])
def test_a_state_that_overflowed(what, qkv, kind):
    """One value of a state that is no number reaches its own column of its own head's y only."""
    sizes, H, V = [11, 40], 3, 112
    d = ref.draw(kind, qkv, sizes, 2, H, H, V, [0, 6, 0], [5, 16], 3)
    plan = _plan(d, 2, H, V, qkv, H)
    y, z = (torch.zeros(d["v"].shape, device="cuda") for _ in range(2))
    _read(plan, d, None, y)
    d["S"][1, 2, 77, 50] = what
    _read(plan, d, None, z)
    torch.cuda.synchronize()
    assert not bool(z[11:, 2, 50].isfinite().any())
    y[11:, 2, 50] = z[11:, 2, 50] = 0
    assert torch.equal(y, z)


@pytest.mark.timeout(300)
def test_the_largest_trees_in_a_graph():
    """Float32 KDA with 64 nodes takes the most memory of a compute unit; captured before any eager call of it."""
    sizes, H, V = [64, 1, 50], 3, 80
    d = ref.draw("kda", "f32", sizes, 3, H, 1, V, [0, 6, 33], [5, 16, 0], 5)
    plan = _plan(d, 3, H, V, "f32", 1)
    y, z = (torch.zeros(d["v"].shape, device="cuda") for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _read(plan, d, None, y)
    for seed in range(3):
        e = ref.draw("kda", "f32", sizes, 3, H, 1, V, [0, 6, 33], [5, 16, 0], 6 + seed)
        for key in d:
            if isinstance(d[key], torch.Tensor):
                d[key].copy_(e[key])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _read(plan, e, None, z)
        torch.cuda.synchronize()
        assert torch.equal(y, z) and rr.slab_err(z, ref.read(e, [0, 1, 2])) <= TOL
