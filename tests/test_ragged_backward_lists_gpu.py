"""Lists whose offsets go backwards over idle entries: the sequences in them do not overlap, so each has its result,
and it has to be the same whichever form takes the call.

Tolerance: the ragged calls' 1e-4 of a slab's largest value."""
import random

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


def _check(call, kind, qkv, spans, H, V, max_len, skip=(), T=None, tail=False):
    """Sequence 2 i of the call has tokens spans[i]; what lies between two spans in the list is idle, as it runs
    backwards or its row is -1.  Those in `skip` are idle too, for their row."""
    import rank_state_read_amd as lib
    T = T or max(b for a, b in spans)
    lens = [b - a for a, b in spans]
    d = ref.draw(kind, qkv, [T], H, H, V, seed=len(spans), state_rows=len(spans))
    d["a"] = d["a"] ** 0.1
    off = [x for span in spans for x in span]
    n = len(off) - 1
    rows = [i // 2 if i % 2 == 0 and i // 2 not in skip else -1 for i in range(n)]
    rows0 = [i // 2 for i in range(n)]
    S, y = torch.full((len(spans), H, 128, V), 7.0, device="cuda"), torch.full(d["v"].shape, 9.0, device="cuda")
    sh = lib.make_shape(len(spans), H, 128, V, 16, 1, 79, 49, kind, qkv, H)
    args = (sh, d["S0"], _i32(rows0), S, _i32(rows), _i32(off), max_len, d["q"], d["k"], d["v"], d["a"], d["beta"], y)
    print(f"  {call} {kind} {qkv} {len(spans)} spans", flush=True)
    if call == "rmw_seq":
        lib.sketchssm_rmw_seq(*args)
    else:
        need = lib.sketchssm_prefill_workspace(sh, n, T, max_len)
        work = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
        lib.sketchssm_prefill(*args, workspace=work[:need])
        torch.cuda.synchronize()
        assert (work[need:] == 255).all()
        if tail:  # cut into segments
            assert need > lib.sketchssm_prefill_workspace(sh, n, T, 64)
    torch.cuda.synchronize()
    seen = torch.zeros(T, dtype=torch.bool)
    for i, (a, b) in enumerate(spans):
        if i in skip:
            assert (S[i] == 7).all()
            continue
        one = dict(d, offsets=torch.tensor([a, b]))
        yr, Sr = ref.run(kind, one, [lens[i]], d["S0"][i:i + 1])
        eS, ey = ref.slab_err(S[i:i + 1], Sr), ref.slab_err(y[a:b], yr[a:b])
        assert eS <= TOL and ey <= TOL, f"sequence {2 * i}: y {ey:.2e}, S {eS:.2e}"
        seen[a:b] = True
    assert (y[~seen.cuda()] == 9).all()


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind,qkv", [(k, q) for k in KINDS for q in ("bf16", "f32")])
@pytest.mark.parametrize("call", ["rmw_seq", "prefill"])
def test_later_tokens_first(call, kind, qkv):
    _check(call, kind, qkv, [(60, 100), (0, 50)], 4, 80, 50, T=107)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_segments(kind):
    """The same of sequences that are cut."""
    _check("prefill", kind, "bf16", [(1400, 2600), (0, 1300)], 4, 80, 1300, tail=True)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [20, 70])
def test_many_in_any_order(n, kind):
    """Backwards, and shuffled with idle entries that overlap the others: below and above a wave's lanes."""
    rng = random.Random(n)
    ends = [0]
    for _ in range(n):
        ends.append(ends[-1] + rng.randrange(0, 70))
    spans = list(zip(ends, ends[1:]))
    _check("prefill", kind, "bf16", spans[::-1], 2, 64, 70)
    rng.shuffle(spans)
    _check("prefill", kind, "bf16", spans, 2, 64, 70, skip=range(0, n, 7))


@pytest.mark.timeout(300)
@pytest.mark.parametrize("long", [False, True])
def test_overlaps_keep_to_their_workspace(long):
    """Sequences that overlap have no defined results, and may ask for more slots than there are: nothing outside the
    workspace and the rows and tokens they name is touched, and what comes before them in the list is right."""
    import rank_state_read_amd as lib
    H, V, B, T = 4, 64, 60, 1200 if long else 300
    d = ref.draw("gdn", "bf16", [T], H, H, V, seed=4, state_rows=B)
    n = 2 * 50 - 1
    off = [0 if i % 2 == 0 else T for i in range(n + 1)]
    S, y = torch.full((B, H, 128, V), 7.0, device="cuda"), torch.full(d["v"].shape, 9.0, device="cuda")
    sh = lib.make_shape(B, H, 128, V, 16, 1, 79, 49, "gdn", "bf16", H)
    need = lib.sketchssm_prefill_workspace(sh, n, T, T)
    assert (need > lib.sketchssm_prefill_workspace(sh, n, T, 64)) == long
    work = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    rows = _i32([i // 2 for i in range(n)])
    lib.sketchssm_prefill(sh, d["S0"], rows, S, rows, _i32(off), T, d["q"], d["k"], d["v"], d["a"], d["beta"], y,
                          workspace=work[:need])
    torch.cuda.synchronize()
    assert (work[need:] == 255).all() and (S[50:] == 7).all()
    Sr = ref.run("gdn", dict(d, offsets=torch.tensor([0, T])), [T], d["S0"][:1])[1]
    assert ref.slab_err(S[:1], Sr) <= TOL


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("call", ["rmw_seq", "prefill"])
def test_offsets_out_of_range_around_good_ones(call, kind):
    """Entries below 0, backwards and past the end: what lies in range between them has its values."""
    import rank_state_read_amd as lib
    H, V, T = 2, 64, 150
    d = ref.draw(kind, "bf16", [T], H, H, V, seed=8, state_rows=6)
    off = _i32([-4, 20, 10, 30, 60, T + 1, T + 20])
    S, y = torch.full((6, H, 128, V), 7.0, device="cuda"), torch.full(d["v"].shape, 9.0, device="cuda")
    fn = lib.sketchssm_rmw_seq if call == "rmw_seq" else lib.sketchssm_prefill
    fn(lib.make_shape(6, H, 128, V, 16, 1, 79, 49, kind, "bf16", H), d["S0"], None, S, None, off, T, d["q"], d["k"],
       d["v"], d["a"], d["beta"], y)
    torch.cuda.synchronize()
    for i, (a, b) in ((2, (10, 30)), (3, (30, 60))):
        yr, Sr = ref.run(kind, dict(d, offsets=torch.tensor([a, b])), [b - a], d["S0"][i:i + 1])
        assert ref.slab_err(S[i:i + 1], Sr) <= TOL and ref.slab_err(y[a:b], yr[a:b]) <= TOL
    assert (S[[0, 1, 4, 5]] == 7).all() and (y[:10] == 9).all() and (y[60:] == 9).all()
