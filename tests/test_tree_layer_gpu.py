"""Drafted trees as a model uses them: prompts, trees read over every layer, accepted paths kept, windows emptied,
states cached and forked; replayed graphs; other streams; a caller's plan.  The reference is the token-by-token
recurrence in 64 bits.  Tolerance 1e-4 per slab, as of every read; a sequence that starts from an 8-bit state is
compared with the recurrence from the state that the cache holds, so the same tolerance applies."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ragged_reference as rr  # noqa: E402
import tree_reference as ref  # noqa: E402

TOL = 1e-4
K, W = 128, 16


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rank_state_read_amd import binding
    binding.lib()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _layer(kind, B, H, V, Hk, ranks, seed):
    """A layer whose sketch heads' basis rows are orthonormal, so F_r is its first r rows."""
    import numpy as np
    from rank_state_read_amd.layer import SketchLayer
    g = np.random.default_rng(seed)
    basis = np.stack([np.linalg.qr(g.standard_normal((K, 79)))[0].T for _ in range(2)]).astype(np.float32)
    groups = [h * 2 // H for h in range(H)]
    return SketchLayer(B=B, H=H, K=K, V=V, W=W, G=2, basis_rows=79, rank_cap=64, kind=kind, qkv="bf16", rank=ranks,
                       group=groups, basis=basis, fmap=lambda gr, r: basis[gr, :r], kq_heads=Hk), basis, groups


class _Oracle:
    """One layer's rows in 64 bits: the state at the last flush and the held-back tokens."""

    def __init__(self, lay, kind, ranks, basis, groups):
        self.kind, self.share = kind, lay.H // lay.Hk
        self.S = torch.zeros_like(lay.S, dtype=torch.float64)
        self.held = [[] for _ in range(lay.B)]
        self.proj = [None if r == 0 else torch.from_numpy(basis[g, :r]).double().cuda() for r, g in zip(ranks, groups)]

    def seen(self, row):
        """What a query sees of the row's last flush: the state, through the sketch of a sketch head."""
        S = self.S[row].clone()
        for h, P in enumerate(self.proj):
            if P is not None:
                S[h] = P.t().contiguous() @ (P @ S[h])
        return S

    def run(self, S, tokens):
        for t in tokens:
            S = ref.step(self.kind, S, t["k"], t["v"], t["a"], t["beta"], self.share)
        return S

    def flush(self, row):
        self.S[row] = self.run(self.S[row], self.held[row])
        self.held[row] = []

    def read(self, row, tokens):
        """y of the last token behind the window's and the others."""
        S = self.run(self.seen(row), self.held[row] + tokens)
        return (tokens[-1]["q"].double().repeat_interleave(self.share, 0)[:, :, None] * S).sum(1)


def _token(d, t):
    return {key: None if d[key] is None else d[key][t] for key in ("q", "k", "v", "a", "beta")}


@pytest.mark.timeout(300)
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_a_served_batch(fmt):
    from rank_state_read_amd.model import SketchModel
    B, shapes = 4, [("gdn", 6, 96, 3, [0, 6, 17, 1, 0, 33]), ("mamba2", 8, 80, 2, [5, 0, 9, 16, 2, 3, 40, 6]),
                    ("kda", 4, 128, 4, [0, 0, 7, 12])]
    layers, orcs = [], []
    for i, (kind, H, V, Hk, ranks) in enumerate(shapes):
        lay, basis, groups = _layer(kind, B, H, V, Hk, ranks, i)
        layers.append(lay)
        orcs.append(_Oracle(lay, kind, ranks, basis, groups))
    m = SketchModel(layers)

    def draw(sizes, seed, how="tree"):
        return [ref.draw(kind, "bf16", sizes, B, H, Hk, V, ranks, [0] * B, seed * 10 + i, how)
                for i, (kind, H, V, Hk, ranks) in enumerate(shapes)]

    # prompts
    prompts = [40, 3, 70, 21]
    d = draw(prompts, 1, "chain")
    m.prefill(d, d[0]["offsets"], max(prompts))
    for lay, orc, x in zip(layers, orcs, d):
        off = x["offsets"].tolist()
        for b in range(B):
            orc.S[b] = orc.run(orc.S[b], [_token(x, t) for t in range(off[b], off[b + 1])])
        assert rr.slab_err(lay.S, orc.S) <= TOL
    pos, held = _i32([0] * B), [0] * B

    def verify(rows, sizes, taken, seed, how="tree"):
        nonlocal pos
        d = draw(sizes, seed, how)
        par, off = d[0]["par"], d[0]["offsets"].tolist()
        for x in d[1:]:  # the same trees in every layer
            x["parents"] = d[0]["parents"]
        ys = m.tree_read(d, d[0]["parents"], d[0]["offsets"], max(sizes), pos=pos, rows=_i32(rows))
        for y, orc, x in zip(ys, orcs, d):
            exp = torch.stack([orc.read(row, [_token(x, off[i] + a) for a in ref.path(par[i], n)])
                               for i, row in enumerate(rows) for n in range(sizes[i])])
            e = rr.slab_err(y, exp)
            print(f"  {orc.kind} rows={rows} held={held} {e:.2e}", flush=True)
            assert e <= TOL
        pos = m.tree_accept(d, d[0]["parents"], d[0]["offsets"], _i32(taken), pos, rows=_i32(rows))
        for i, row in enumerate(rows):
            p = ref.path(par[i], taken[i])
            held[row] += len(p)
            for orc, x in zip(orcs, d):
                orc.held[row] += [_token(x, off[i] + a) for a in p]
        assert pos.tolist() == held

    def flush(rows):
        nonlocal pos
        m.flush_seq(_i32(rows), pos[rows].contiguous())
        pos = pos.clone()
        pos[rows] = 0
        for row in rows:
            held[row] = 0
            for lay, orc in zip(layers, orcs):
                orc.flush(row)
                assert rr.slab_err(lay.S[row][None], orc.S[row][None]) <= TOL

    verify([2, 0, 3], [7, 12, 1], [4, 9, 0], 2)
    verify([0, 1, 2, 3], [5, 5, 5, 5], [4, -1, 2, 3], 3, "chain")
    verify([3, 1], [17, 9], [16, 8], 4)
    flush([0, 3])
    verify([0, 1, 2, 3], [16, 3, 20, 2], [6, 2, 11, 1], 5)
    flush([0, 1, 2, 3])
    # rows 2 and 0 to the cache; rows 1 and 3 go on from row 2's state, row 0 from none
    caches = m.new_cache(5, fmt)
    m.cache_store(caches, _i32([2, 0]), _i32([4, 1]))
    m.cache_load(caches, _i32([4, -1, 4]), _i32([1, 0, 3]))
    for lay, orc, c in zip(layers, orcs, caches):
        back = ref.quantised(lay.S[2], fmt)[1]
        assert torch.equal(lay.S[1].double(), back) and torch.equal(lay.S[3].double(), back)
        assert (lay.S[0] == 0).all()
        # what 8 bits lose of a key row: half a step of 1/127 (rounded up to 8 bits, 2^-7) of its largest value at
        # most, or 2^-4 of each value and 2^-10 of the scale, itself under 2 / 448 of the largest
        worst = (back - lay.S[2].double()).abs().amax(-1) / lay.S[2].double().abs().amax(-1).clamp(min=1e-30)
        assert worst.max() <= (0.5 / 127 * (1 + 2 ** -7) if fmt == "i8" else 2 ** -4)
        orc.S[1], orc.S[3], orc.S[0] = back, back, 0
    verify([0, 1, 2, 3], [4, 9, 14, 3], [3, 5, 6, 0], 6)
    flush([1])
    verify([1], [33], [2], 7)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", ["mamba2", "gdn", "kda"])
def test_replayed_graph(kind):
    """A step of read, accept and copies in a graph, replayed on new tokens with eager work in between; every replay
    has the eager call's bits."""
    from rank_state_read_amd import Plan, sketchssm_cache_load, sketchssm_cache_store, sketchssm_tree_accept, \
        sketchssm_tree_read
    sizes, B, H, Hk, V, ranks = [12, 20, 3], 4, 6, 3, 96, [0, 6, 17, 1, 0, 33]
    rows, taken = _i32([2, 0, 3]), _i32([5, 2, 1])
    sh = ref.shape_of(B, H, V, kind, "bf16", Hk)
    d = ref.draw(kind, "bf16", sizes, B, H, Hk, V, ranks, [1, 2, 3, 4], 0)
    plan = Plan(sh, ranks, d["groups"])
    y, S2 = torch.zeros(d["v"].shape, device="cuda"), torch.zeros_like(d["S"])
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    codes = torch.zeros(2, H, K, V, dtype=torch.int8, device="cuda")
    scales = torch.zeros(2, H, K, dtype=torch.bfloat16, device="cuda")
    slots = _i32([1])

    def once(d, y, S2, new):
        sketchssm_tree_read(plan, d["S"], d["Z"], d["frames"], d["kbuf"], d["vbuf"], d["abuf"], d["bbuf"], d["pos"], rows,
                            d["offsets"], 20, d["parents"], d["q"], d["k"], d["v"], d["a"], d["beta"], y)
        sketchssm_tree_accept(sh, d["kbuf"], d["vbuf"], d["abuf"], d["bbuf"], d["pos"], new, rows, d["offsets"],
                              d["parents"], taken, d["k"], d["v"], d["a"], d["beta"])
        sketchssm_cache_store(sh, d["S"], rows[:1], codes, scales, slots, "i8")
        sketchssm_cache_load(sh, codes, scales, slots, S2, rows[:1], "i8")

    once(d, y, S2, new)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(d, y, S2, new)
    for seed in range(1, 5):
        e = ref.draw(kind, "bf16", sizes, B, H, Hk, V, ranks, [seed, 2, 0, 4], seed)
        for key in d:
            if isinstance(d[key], torch.Tensor):
                d[key].copy_(e[key])
        y.fill_(5), S2.fill_(5), new.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        y2, S3, new2 = torch.full_like(y, 5.0), torch.full_like(S2, 5.0), torch.full_like(new, 5)
        once(e, y2, S3, new2)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(S2, S3) and torch.equal(new, new2)
        for key in ("kbuf", "vbuf", "abuf", "bbuf"):
            if d[key] is not None:
                assert torch.equal(d[key].nan_to_num(7.0), e[key].nan_to_num(7.0))


@pytest.mark.timeout(300)
def test_other_streams():
    """Two calls at once on streams of their own, outputs taken by the layer."""
    lay, _, groups = _layer("gdn", 3, 4, 128, 2, [0, 5, 20, 0], 3)
    s = [torch.cuda.Stream() for _ in range(2)]
    d = [ref.draw("gdn", "bf16", [16, 9, 30], 3, 4, 2, 128, [0, 5, 20, 0], [0] * 3, i) for i in range(2)]
    lay.S.copy_(d[0]["S"])
    lay.flush(0)
    torch.cuda.synchronize()
    ys = []
    for x, st in zip(d, s):
        ys.append(lay.tree_read(x["offsets"], 30, x["parents"], x["q"], x["k"], x["v"], x["a"], x["beta"], stream=st))
    torch.cuda.synchronize()
    for x, y in zip(d, ys):
        z = lay.tree_read(x["offsets"], 30, x["parents"], x["q"], x["k"], x["v"], x["a"], x["beta"])
        torch.cuda.synchronize()
        assert torch.equal(y, z)
    cache = lay.new_cache(3, "e4m3")
    with torch.cuda.stream(s[0]):
        lay.cache_store(cache)
    lay.cache_load(cache, _i32([2, 1, 0]), stream=s[0])
    s[0].synchronize()
    assert torch.equal(lay.S[0].double(), ref.quantised(d[0]["S"][2], "e4m3")[1])


def test_verified_on_the_full_state():
    """An all-dense plan on a layer of sketch heads."""
    from rank_state_read_amd import Plan
    lay, _, groups = _layer("kda", 2, 4, 64, 4, [6, 6, 6, 6], 4)
    d = ref.draw("kda", "bf16", [9, 4], 2, 4, 4, 64, [0] * 4, [0, 0], 2)
    lay.S.copy_(d["S"])
    dense = Plan(lay.shape, [0] * 4, groups)
    y = lay.tree_read(d["offsets"], 9, d["parents"], d["q"], d["k"], d["v"], d["a"], d["beta"], pos=_i32([0, 0]),
                      plan=dense)
    assert rr.slab_err(y, ref.read(d, [0, 1])) <= TOL
