"""Prefill and the recurrent form over ragged batches against the token-by-token recurrence in 64 bits, and the
gated norm against its formula.

Tolerance of y and S: 1e-4 of a slab's largest value, a slab being one token's y or one state of one head (the
bar of every read of this library).  An fp32 sum over K = 128 channels is off by at most (K + 2) 2^-24 = 7.7e-6 of
the sum of its terms' magnitudes, which for independent terms is about sqrt(K) times the result: 8.8e-5.
Tolerance of the norm: see its test."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ragged_reference as ref  # noqa: E402

TOL = 1e-4
KINDS = ["mamba2", "gdn", "kda"]
CALLS = ["rmw_seq", "prefill"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rank_state_read_amd import binding
    binding.lib()


def _shape(B, H, V, kind, qkv, Hk):
    from rank_state_read_amd import make_shape
    return make_shape(B, H, 128, V, 16, 1, 79, 49, kind, qkv, Hk)


def _call(call, shape, d, S0, rows0, S, rows, max_len, y, stream=None):
    import rank_state_read_amd as lib
    fn = lib.sketchssm_rmw_seq if call == "rmw_seq" else lib.sketchssm_prefill
    fn(shape, S0, rows0, S, rows, d["offsets"], max_len, d["q"], d["k"], d["v"], d["a"], d["beta"], y, stream=stream)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _check(call, kind, qkv, lens, H=4, Hk=2, V=128, seed=0, edit=None, lead=3, tail=5, tol=TOL, zero=()):
    """Rows shuffled over a larger cache; sequences in `zero` start from zero, the others from other rows of S0."""
    n = len(lens)
    d = ref.draw(kind, qkv, lens, H, Hk, V, seed, lead, tail, state_rows=n + 2)
    if edit:
        edit(d)
    B = n + 3
    rows = [(5 * i + 1) % B if B % 5 else (7 * i + 1) % B for i in range(n)]
    assert len(set(rows)) == n
    rows0 = [-1 if i in zero else (i + 1) % (n + 2) for i in range(n)]
    S = torch.full((B, H, 128, V), 7.0, device="cuda")
    y = torch.full(d["v"].shape, 9.0, device="cuda")
    print(f"  {call} {kind} {qkv} V={V} H={H}/{Hk} lens={lens}", flush=True)
    _call(call, _shape(B, H, V, kind, qkv, Hk), d, d["S0"], _i32(rows0), S, _i32(rows), max(lens), y)
    torch.cuda.synchronize()
    first = torch.stack([torch.zeros_like(d["S0"][0]) if r < 0 else d["S0"][r] for r in rows0])
    yr, Sr = ref.run(kind, d, lens, first)
    eS, ey = ref.slab_err(S[rows], Sr), ref.slab_err(y[lead:lead + sum(lens)], yr[lead:lead + sum(lens)])
    print(f"    y {ey:.2e}  S {eS:.2e}", flush=True)
    assert eS <= tol and ey <= tol
    others = [r for r in range(B) if r not in rows]
    assert (S[others] == 7).all(), "a row that no sequence names was written"
    assert (y[:lead] == 9).all() and (y[lead + sum(lens):] == 9).all(), "y of tokens outside the sequences"
    for i, length in enumerate(lens):
        if length == 0:
            assert torch.equal(S[rows[i]], first[i])
    return d, S, y


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("lens", [[1], [0, 1, 2, 0], [7, 8, 9], [15, 16, 17], [31, 32, 33], [63, 64, 65, 1],
                                  [127, 0, 128, 129], [5, 211, 40]], ids=str)
def test_lengths(call, kind, lens):
    _check(call, kind, "bf16", lens, zero=(1,))


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [64, 80, 96, 112, 128])
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("call", CALLS)
def test_widths_and_types(call, qkv, V, kind):
    _check(call, kind, qkv, [70, 3, 45], V=V, H=6, Hk=3, zero=(0, 2))


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,Hk", [(1, 1), (5, 5), (8, 1), (12, 4)])
@pytest.mark.parametrize("call", CALLS)
def test_head_groups(call, H, Hk, kind):
    _check(call, kind, "bf16", [37, 66], H=H, Hk=Hk, V=80)


def _zero_decay(d):
    d["a"][40:44] = 0


def _decay_one(d):
    d["a"].fill_(1)


def _small_decay(d):
    d["a"][3:203] = 1e-3


def _tiny_decay(d):
    d["a"][10:90] = 1e-30


def _negative_decay(d):
    d["a"][20:120] *= -1


def _beta_zero(d):
    if d["beta"] is not None:
        d["beta"][10:60] = 0


def _zero_keys(d):
    d["k"][30:50] = 0


def _zero_queries(d):
    d["q"][30:50] = 0


def _zero_values(d):
    d["v"][3:120] = 0


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("edit", [_zero_decay, _decay_one, _small_decay, _tiny_decay, _negative_decay, _beta_zero,
                                  _zero_keys, _zero_queries, _zero_values], ids=lambda f: f.__name__[1:])
@pytest.mark.parametrize("call", CALLS)
def test_degenerate_tokens(call, edit, kind):
    d, S, y = _check(call, kind, "bf16", [150, 50], edit=edit)
    if edit is _zero_queries:
        assert (y[30:50] == 0).all()


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", ["gdn", "kda"])
@pytest.mark.parametrize("call", CALLS)
def test_one_key_written_again_and_again(call, kind):
    """The same unit key with beta = 1: every token replaces what the one before wrote, the state holds the last
    value (to the rounding of k to bf16, whose square then is not exactly 1)."""
    def edit(d):
        g = torch.Generator().manual_seed(3)
        k = torch.zeros(1, d["k"].shape[1], 128)
        k[..., torch.randperm(128, generator=g)[:4]] = 0.5
        d["k"][3:-5] = k.to(d["k"])
        d["beta"].fill_(1)
        d["a"].fill_(1)
    d, S, y = _check(call, kind, "bf16", [97], edit=edit)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_long_sequence(kind):
    """2500 tokens beside a short sequence: the error does not grow along the sequence."""
    d, S, y = _check("prefill", kind, "bf16", [2500, 130], H=2, Hk=1, V=128 if kind != "mamba2" else 80, zero=(0,))


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("call", CALLS)
def test_in_place_from_own_rows_and_zero(call, kind):
    """S0 is S: sequences go on from their own rows, one from zero, one forks a row that nothing writes."""
    lens, H, V, B = [20, 45, 33], 4, 80, 5
    d = ref.draw(kind, "bf16", lens, H, H, V, seed=5)
    g = torch.Generator().manual_seed(8)
    S = (0.05 * torch.randn(B, H, 128, V, generator=g)).cuda()
    before = S.clone()
    rows, rows0 = [2, 0, 4], [2, -1, 3]
    y = torch.empty(d["v"].shape, device="cuda")
    _call(call, _shape(B, H, V, kind, "bf16", 0), d, S, _i32(rows0), S, _i32(rows), 45, y)
    torch.cuda.synchronize()
    yr, Sr = ref.run(kind, d, lens, torch.stack([before[2], torch.zeros_like(before[0]), before[3]]))
    assert ref.slab_err(S[rows], Sr) <= TOL and ref.slab_err(y, yr) <= TOL
    assert torch.equal(S[[1, 3]], before[[1, 3]])


@pytest.mark.timeout(300)
@pytest.mark.parametrize("call", CALLS)
def test_default_rows(call):
    """rows NULL: sequence i is row i; S0 NULL: every sequence starts from zero."""
    lens = [18, 40]
    d = ref.draw("gdn", "bf16", lens, 2, 2, 64, seed=6)
    S = torch.full((3, 2, 128, 64), 7.0, device="cuda")
    y = torch.empty(d["v"].shape, device="cuda")
    _call(call, _shape(3, 2, 64, "gdn", "bf16", 0), d, None, None, S, None, 40, y)
    torch.cuda.synchronize()
    yr, Sr = ref.run("gdn", d, lens, torch.zeros(2, 2, 128, 64, device="cuda"))
    assert ref.slab_err(S[:2], Sr) <= TOL and ref.slab_err(y, yr) <= TOL and (S[2] == 7).all()


@pytest.mark.timeout(300)
@pytest.mark.parametrize("call", CALLS)
def test_bad_list_entries_idle_their_sequence(call):
    """Rows, first rows, offsets and lengths out of range leave their sequence alone and the others right."""
    lens, H, V = [20, 20, 20, 20, 50, 20], 2, 64
    d = ref.draw("gdn", "bf16", lens, H, H, V, seed=7)
    T = sum(lens)
    S = torch.full((6, H, 128, V), 7.0, device="cuda")
    y = torch.full(d["v"].shape, 9.0, device="cuda")
    rows, rows0 = [0, 6, -1, 3, 4, 5], [0, 1, 2, 6, 4, 5]
    sh = _shape(6, H, V, "gdn", "bf16", 0)
    _call(call, sh, d, d["S0"], _i32(rows0), S, _i32(rows), 20, y)  # rows 6 and -1, first row 6, 50 tokens
    torch.cuda.synchronize()
    yr, Sr = ref.run("gdn", d, lens, d["S0"])
    off = d["offsets"].tolist()
    for i in range(6):
        part = slice(off[i], off[i + 1])
        if i in (0, 5):
            assert ref.slab_err(S[[i]], Sr[[i]]) <= TOL and ref.slab_err(y[part], yr[part]) <= TOL
        else:
            assert (y[part] == 9).all()
    assert (S[1:5] == 7).all()
    S.fill_(7)
    y.fill_(9)
    bad = dict(d, offsets=_i32([-4, 20, 10, 30, 60, T + 1, T + 20]))  # only 10..30 and 30..60 are in range
    _call(call, sh, bad, d["S0"], None, S, None, T, y)
    torch.cuda.synchronize()
    assert (S[[0, 1, 4, 5]] == 7).all() and (S[2:4] != 7).any(-1).any(-1).all()
    assert (y[:10] == 9).all() and (y[60:] == 9).all()


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_pieces_of_a_prompt(kind):
    """A prompt in three calls, the pieces ending inside a chunk, gives what one call gives; the last piece goes
    through the recurrent form."""
    H, V, cuts = 4, 80, [0, 101, 170, 177]
    d = ref.draw(kind, "bf16", [177], H, 2, V, seed=9)
    sh = _shape(1, H, V, kind, "bf16", 2)
    S, y = torch.zeros(1, H, 128, V, device="cuda"), torch.empty(d["v"].shape, device="cuda")
    for i in range(3):
        piece = dict(d, offsets=_i32([cuts[i], cuts[i + 1]]))
        _call("rmw_seq" if i == 2 else "prefill", sh, piece, S, None, S, None, 177, y)
    torch.cuda.synchronize()
    yr, Sr = ref.run(kind, d, [177], torch.zeros(1, H, 128, V, device="cuda"))
    assert ref.slab_err(S, Sr) <= TOL and ref.slab_err(y, yr) <= TOL


@pytest.mark.timeout(300)
@pytest.mark.parametrize("call", CALLS)
def test_offsets_past_32_bits(call):
    """Tokens whose elements lie past 2^31 in v and y."""
    H, V, T, lens = 128, 128, 132000, [40, 21]
    sh = _shape(2, H, V, "mamba2", "bf16", 1)
    d = ref.draw("mamba2", "bf16", lens, H, 1, V, seed=10)
    big = {"offsets": _i32([T - 61, T - 21, T]), "beta": None}
    for key in ("q", "k", "v", "a"):
        big[key] = torch.zeros((T,) + tuple(d[key].shape[1:]), dtype=d[key].dtype, device="cuda")
        big[key][T - 61:] = d[key]
    assert big["v"].numel() > 2 ** 31
    S, y = torch.empty(2, H, 128, V, device="cuda"), torch.zeros(T, H, V, device="cuda")
    _call(call, sh, big, None, None, S, None, 40, y)
    torch.cuda.synchronize()
    yr, Sr = ref.run("mamba2", d, lens, torch.zeros_like(S))
    assert ref.slab_err(S, Sr) <= TOL and ref.slab_err(y[T - 61:], yr) <= TOL
    assert (y[:T - 61].abs().amax() == 0)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("call", CALLS)
def test_replays_and_streams(call, kind):
    """A captured call replayed between eager work, two calls at once on two streams, and a call on a stream other
    than the current one: bit for bit the eager result each time."""
    lens, H, V = [70, 33, 9], 8, 128
    sh = _shape(3, H, V, kind, "bf16", 4)
    ds = [ref.draw(kind, "bf16", lens, H, 4, V, seed=20 + i) for i in range(2)]
    Ss = [torch.zeros(3, H, 128, V, device="cuda") for _ in ds]
    ys = [torch.zeros(d["v"].shape, device="cuda") for d in ds]

    def go(i, stream=None):
        _call(call, sh, ds[i], ds[i]["S0"], None, Ss[i], None, 70, ys[i], stream=stream)

    def clear():
        for x in Ss + ys:
            x.fill_(float("nan"))
        torch.cuda.synchronize()

    for i in range(2):
        go(i)
    torch.cuda.synchronize()
    eager = [x.clone() for x in Ss + ys]
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            go(i)
    for rep in range(3):
        clear()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, e) for x, e in zip(Ss + ys, eager)), f"replay {rep}"
        go(rep % 2)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(3):
        clear()
        for i in range(2):
            go(i, streams[i] if rep != 1 else streams[i].cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, e) for x, e in zip(Ss + ys, eager)), f"two streams, {rep}"


# ---------------------------------------------------------------------------
# the gated norm
# ---------------------------------------------------------------------------
def _norm_case(qkv, H, V, n, heads, gate, skip, shared_w, seed=0, scale=1.0):
    import rank_state_read_amd as lib
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    dt = torch.bfloat16 if qkv == "bf16" else torch.float32
    y, z, x = scale * rn(n, H, V), (3 * rn(n, H, V)).to(dt), rn(n, H, V).to(dt)
    D, w = rn(H), 1 + 0.3 * (rn(V) if shared_w else rn(H, V))
    out = torch.full((n, H, V), 5.0, dtype=dt, device="cuda")
    z, x, D = (None if gate == "none" else z), (x if skip else None), (D if skip else None)
    lib.sketchssm_gated_norm(_shape(1, H, V, "mamba2", qkv, 0), y, x, D, z, w, heads, gate, 1e-5, out)
    torch.cuda.synchronize()
    want = ref.norm(y, x, D, z, w, heads, gate, 1e-5)
    # relative to each value: the sum of W squares is off by at most W steps of 2^-24 (all terms positive) and its
    # root by half of that; exp, the two divisions, the root and the products add less than 24 more; one rounding at
    # the store
    W = heads * V
    tol = (W / 2 + 24) * 2.0 ** -24 + (2.0 ** -8 if qkv == "bf16" else 0)
    err = ((out.double() - want).abs() / want.abs().clamp(min=1e-30)).max().item() if n else 0.0
    print(f"  norm {qkv} H={H} V={V} n={n} heads={heads} {gate}: {err:.2e} of {tol:.2e}", flush=True)
    assert err <= tol


@pytest.mark.timeout(300)
@pytest.mark.parametrize("gate", ["none", "silu_first", "silu", "sigmoid"])
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("skip,shared_w", [(False, True), (True, False)])
def test_norm_forms(gate, qkv, skip, shared_w):
    _norm_case(qkv, 12, 80, 37, 4, gate, skip, shared_w)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("H,V,heads", [(1, 64, 1), (3, 96, 1), (5, 112, 5), (32, 128, 1), (8, 64, 8), (40, 80, 8),
                                       (128, 80, 16), (16, 128, 16), (128, 64, 128), (64, 128, 64), (130, 64, 130),
                                       (256, 128, 256)])
def test_norm_widths(qkv, H, V, heads):
    for n in (1, 3, 18):
        _norm_case(qkv, H, V, n, heads, "silu_first", False, False, seed=n)


@pytest.mark.timeout(120)
def test_norm_extremes():
    """Large and tiny values, gates far out on both sides, no tokens."""
    for scale in (1e-12, 1e12):
        _norm_case("f32", 8, 80, 9, 2, "silu", False, True, scale=scale)
    _norm_case("bf16", 8, 80, 0, 2, "silu", False, True)
    import rank_state_read_amd as lib
    y = torch.ones(2, 1, 64, device="cuda")
    z = torch.full((2, 1, 64), -200.0, device="cuda")
    z[1] = 200.0
    out = torch.empty_like(y)
    for gate, low, high in (("sigmoid", 0.0, 1.0), ("silu", 0.0, 200.0)):
        lib.sketchssm_gated_norm(_shape(1, 1, 64, "gdn", "f32", 0), y, None, None, z, torch.ones(64, device="cuda"), 1,
                                 gate, 0.0, out)
        torch.cuda.synchronize()
        assert (out[0].abs() <= 1e-30).all() and (out[1] == high).all() and low == 0.0


# ---------------------------------------------------------------------------
# together: prompts, first sketches, decode, gated outputs
# ---------------------------------------------------------------------------
@pytest.mark.timeout(300)
@pytest.mark.parametrize("name,heads,gate", [("c1", 16, "silu_first"), ("c3", 1, "silu"), ("c4", 1, "sigmoid")])
def test_prompts_then_decode(name, heads, gate):
    """SketchModel: prompts of different lengths, then two windows of decode steps, with every layer's gated norm;
    the dense reads' outputs are the exact recurrence's, so every y follows from the prompts in 64 bits."""
    import numpy as np
    from rank_state_read_amd.layer import SketchLayer
    from rank_state_read_amd.model import SketchModel
    from workloads import CONFIGS
    c, lens, B, H = CONFIGS[name], [40, 1, 75], 3, 16
    share = 4
    mk = lambda: SketchLayer(B=B, H=H, K=128, V=c.V, W=16, G=1, basis_rows=79, rank_cap=49, kind=c.kind,  # noqa: E731
                             qkv="bf16", rank=np.zeros(H, np.int32), group=np.zeros(H, np.int32),
                             basis=np.zeros((1, 79, 128), np.float32), kq_heads=H // share)
    layers = [mk(), mk()]
    g = torch.Generator().manual_seed(2)
    D = torch.randn(H, generator=g).cuda() if c.kind == "mamba2" else None
    w = (1 + 0.2 * torch.randn(H, c.V, generator=g)).cuda()
    for L in layers:
        L.set_norm(w, heads, gate, D=D)
    model = SketchModel(layers)
    steps = 35
    ds = [ref.draw(c.kind, "bf16", [length + steps for length in lens], H, H // share, c.V, seed=30 + i)
          for i in range(2)]
    for d in ds:
        d["z"] = torch.randn(d["v"].shape, generator=g).cuda().to(torch.bfloat16)
    full = [ref.run(c.kind, d, [n + steps for n in lens], torch.zeros(B, H, 128, c.V, device="cuda"))[0] for d in ds]
    off = ds[0]["offsets"].tolist()
    keys = ("q", "k", "v", "a", "beta", "z")

    def take(d, idx):
        return {key: None if d[key] is None else d[key][idx].contiguous() for key in keys}

    def check(got, d, y, idx, what):
        want = ref.norm(y[idx], d["v"][idx] if D is not None else None, D, d["z"][idx], w, heads, gate, 1e-5)
        # y's own 1e-4 of a slab, through a norm that keeps relative sizes, and the rounding to bf16
        err = ref.slab_err(got, want)
        assert err <= 2 * TOL + 2.0 ** -8, f"{what}: {err:.2e}"

    prompt = torch.cat([torch.arange(off[b], off[b] + n) for b, n in enumerate(lens)]).cuda()
    offsets = _i32([0, lens[0], lens[0] + lens[1], sum(lens)])
    outs = model.prefill([take(d, prompt) for d in ds], offsets, max(lens))
    for d, y, o in zip(ds, full, outs):
        check(o, d, y, prompt, "prefill")
    for t in range(steps):
        idx = torch.tensor([off[b] + n + t for b, n in enumerate(lens)]).cuda()
        outs = model.decode_step([take(d, idx) for d in ds])
        for d, y, o in zip(ds, full, outs):
            check(o, d, y, idx, f"step {t}")
