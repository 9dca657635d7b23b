"""Prefill of few long sequences, which are cut into segments, against the token-by-token recurrence in 64 bits.

Tolerance: that of the uncut form, 1e-4 of a slab's largest value.  A segment's first state is N + M S, one more
sum over K = 128 channels with |M| <= 1 (keys of length 1, decays and beta up to 1): the same bound."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ragged_reference as ref  # noqa: E402

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


def _slow(d):
    """Decays near 1: a segment's end still depends on its start."""
    d["a"] = d["a"] ** 0.02


def _go(kind, qkv, d, H, Hk, V, S0, rows0, S, rows, y, max_len, stream=None, workspace=None, cut=True):
    import rank_state_read_amd as lib
    sh = lib.make_shape(S.shape[0], H, 128, V, 16, 1, 79, 49, kind, qkv, Hk)
    n = len(d["offsets"]) - 1
    need = lib.sketchssm_prefill_workspace(sh, n, d["v"].shape[0], max_len)
    assert not cut or need > lib.sketchssm_prefill_workspace(sh, n, d["v"].shape[0], 64), "not cut into segments"
    if workspace is None:
        workspace = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    lib.sketchssm_prefill(sh, S0, rows0, S, rows, d["offsets"], max_len, d["q"], d["k"], d["v"], d["a"], d["beta"], y,
                          workspace=workspace, stream=stream)


def _check(kind, qkv, lens, H, Hk, V, seed=0, edit=_slow, zero=(), max_len=None, cut=True):
    n = len(lens)
    d = ref.draw(kind, qkv, lens, H, Hk, V, seed, 3, 5)
    if edit:
        edit(d)
    rows, rows0 = [(i + 1) % n for i in range(n)], [-1 if i in zero else i for i in range(n)]
    S, y = torch.full((n + 1, H, 128, V), 7.0, device="cuda"), torch.full(d["v"].shape, 9.0, device="cuda")
    print(f"  {kind} {qkv} V={V} H={H}/{Hk} lens={lens}", flush=True)
    _go(kind, qkv, d, H, Hk, V, d["S0"], _i32(rows0), S, _i32(rows), y, max_len or max(lens), cut=cut)
    torch.cuda.synchronize()
    first = torch.stack([torch.zeros_like(d["S0"][0]) if r < 0 else d["S0"][r] for r in rows0])
    yr, Sr = ref.run(kind, d, lens, first)
    eS, ey = ref.slab_err(S[rows], Sr), ref.slab_err(y[3:-5], yr[3:-5])
    print(f"    y {ey:.2e}  S {eS:.2e}", flush=True)
    assert eS <= TOL and ey <= TOL
    assert (S[n] == 7).all() and (y[:3] == 9).all() and (y[-5:] == 9).all()


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [64, 80, 96, 112, 128])
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
def test_widths_and_types(qkv, V, kind):
    _check(kind, qkv, [1030], 2, 1, V)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,zero", [([1300, 0, 37, 700], (1, 3)), ([513, 1, 1024, 512], (2,)), ([1537], (0,))],
                         ids=str)
def test_lengths(kind, lens, zero):
    _check(kind, "bf16", lens, 3, 1, 80, zero=zero)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_max_len_above_the_longest(kind):
    _check(kind, "bf16", [900, 300], 2, 2, 128, max_len=1 << 30)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_degenerate_decays(kind):
    """Decays of 0, of -1 and of 1 at the ends of chunks and segments."""
    def edit(d):
        _slow(d)
        T = d["a"].shape[0]
        d["a"][3 + 255] = 0
        d["a"][3 + 256] = 1
        d["a"][3 + 600:3 + 640] = 0
        d["a"][T - 200:T - 190] = -1
    _check(kind, "bf16", [1100], 2, 1, 64, edit=edit)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_in_place(kind):
    """The last state goes where the first one stands, while the first segment starts from it: many heads, so that
    segments run at different times."""
    lens, H, V = [2100, 1025], 24, 80
    d = ref.draw(kind, "bf16", lens, H, 8, V, seed=5)
    _slow(d)
    S = d["S0"].clone()
    y = torch.empty(d["v"].shape, device="cuda")
    _go(kind, "bf16", d, H, 8, V, S, None, S, None, y, 2100)
    torch.cuda.synchronize()
    yr, Sr = ref.run(kind, d, lens, d["S0"])
    assert ref.slab_err(S, Sr) <= TOL and ref.slab_err(y, yr) <= TOL


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_replays_and_streams(kind):
    """Replays of a captured call between eager ones, and two calls at once with a workspace each: bit for bit."""
    lens, H, V = [1400, 90], 4, 128
    ds = [ref.draw(kind, "bf16", lens, H, 4, V, seed=30 + i) for i in range(2)]
    Ss = [torch.empty(2, H, 128, V, device="cuda") for _ in ds]
    ys = [torch.empty(d["v"].shape, device="cuda") for d in ds]

    def go(i, stream=None):
        _go(kind, "bf16", ds[i], H, 4, V, ds[i]["S0"], None, Ss[i], None, ys[i], 1400, stream=stream,
            workspace=works[i])

    import rank_state_read_amd as lib
    need = lib.sketchssm_prefill_workspace(lib.make_shape(2, H, 128, V, 16, 1, 79, 49, kind, "bf16", 4), 2, 1490, 1400)
    works = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in ds]
    for i in range(2):
        go(i)
    torch.cuda.synchronize()
    eager = [x.clone() for x in Ss + ys]

    def clear():
        for x in Ss + ys:
            x.fill_(float("nan"))
        for x in works:
            x.fill_(255)
        torch.cuda.synchronize()

    def same(what):
        torch.cuda.synchronize()
        assert all(torch.equal(x, e) for x, e in zip(Ss + ys, eager)), what

    graphs = [torch.cuda.CUDAGraph() for _ in ds]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            go(i)
    streams = [torch.cuda.Stream() for _ in ds]
    for rep in range(3):
        clear()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        same(f"replay {rep}")
        clear()
        for i in range(2):
            go(i, stream=streams[i])
        same(f"streams {rep}")


@pytest.mark.timeout(300)
@pytest.mark.parametrize("V", [64, 80, 96, 112])
@pytest.mark.parametrize("H,Hk", [(48, 8), (16, 2), (12, 4), (20, 1)])
def test_many_heads_of_a_key_head(H, Hk, V):
    """Blocks of two heads where widths and numbers allow them, of one elsewhere, cut into segments and not."""
    for lens in ([1100, 80], [70, 33, 0, 64, 65, 20, 7, 90, 31, 32, 33, 44, 51, 12]):
        _check("mamba2", "bf16", lens, H, Hk, V, zero=(1,), cut=False)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind,qkv", [("kda", "bf16"), ("kda", "f32"), ("gdn", "f32"), ("mamba2", "f32")])
def test_many_sequences(kind, qkv):
    """More sequences than a wave has lanes, and enough of them for blocks of all 128 value columns."""
    _check(kind, qkv, [33 + (7 * i) % 40 for i in range(70)], 6, 6, 128, zero=range(0, 70, 3), cut=False)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_long_sequence_among_many_short_ones(kind):
    """One sequence cut into segments, the others shorter than one, more of them than a wave has lanes; first, in the
    middle and last."""
    for at in (0, 40, 69):
        lens = [(3 * i) % 11 for i in range(70)]
        lens[at] = 2049
        _check(kind, "bf16", lens, 4, 2, 80, zero=range(0, 70, 4))
