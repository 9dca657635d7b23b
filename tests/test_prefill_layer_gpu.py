"""The ragged calls as a layer's owner makes them: fresh and continued prompts of listed rows, tokens of some rows,
other streams, and what a bad token or a short workspace does.

Tolerance: the ragged calls' 1e-4 of a slab's largest value."""
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


def _layer(kind, B, H, V, Hk):
    import numpy as np
    from rank_state_read_amd.layer import SketchLayer
    return SketchLayer(B=B, H=H, K=128, V=V, W=16, G=1, basis_rows=79, rank_cap=49, kind=kind, qkv="bf16",
                       rank=np.zeros(H, np.int32), group=np.zeros(H, np.int32),
                       basis=np.zeros((1, 79, 128), np.float32), kq_heads=Hk)


def _part(d, spans):
    idx = torch.cat([torch.arange(a, b) for a, b in spans]).cuda()
    out = {key: None if d[key] is None else d[key][idx].contiguous() for key in ("q", "k", "v", "a", "beta")}
    off = [0]
    for a, b in spans:
        off.append(off[-1] + b - a)
    return out, _i32(off), max(b - a for a, b in spans), idx


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_fresh_then_continued_then_tokens(kind):
    """Rows 4, 0 and 2 of a layer: a first piece of each prompt into stale states, the rest, then a few tokens each."""
    lens, cut1, cut2 = [150, 40, 90], [100, 33, 20], [144, 38, 90]
    H, V, Hk, rows = 8, 80, 2, [4, 0, 2]
    d = ref.draw(kind, "bf16", lens, H, Hk, V, seed=3)
    L = _layer(kind, 5, H, V, Hk)
    L.S.fill_(3.0)  # what another sequence left there
    off = d["offsets"].tolist()
    yr, Sr = ref.run(kind, d, lens, torch.zeros(3, H, 128, V, device="cuda"))
    x, o, n, idx = _part(d, [(off[i], off[i] + cut1[i]) for i in range(3)])
    y = L.prefill(o, n, x["q"], x["k"], x["v"], x["a"], x["beta"], rows=_i32(rows))
    assert ref.slab_err(y, yr[idx]) <= TOL
    x, o, n, idx = _part(d, [(off[i] + cut1[i], off[i] + cut2[i]) for i in range(3)])
    y = L.prefill(o, n, x["q"], x["k"], x["v"], x["a"], x["beta"], rows=_i32(rows), fresh=False)
    assert ref.slab_err(y, yr[idx]) <= TOL
    x, o, n, idx = _part(d, [(off[i] + cut2[i], off[i] + lens[i]) for i in range(3)])
    y = L.rmw_seq(o, n, x["q"], x["k"], x["v"], x["a"], x["beta"], rows=_i32(rows))
    assert ref.slab_err(y, yr[idx]) <= TOL and ref.slab_err(L.S[rows], Sr) <= TOL
    assert (L.S[[1, 3]] == 3).all()


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
def test_call_on_another_stream_owns_its_memory(kind):
    """A call queued behind other work of a side stream, its y and workspace taken by the call: memory that the
    current stream allocates and overwrites meanwhile is not theirs."""
    lens, H, V = [300, 170], 8, 64
    d = ref.draw(kind, "bf16", lens, H, H, V, seed=4)
    L = _layer(kind, 2, H, V, H)
    side, busy = torch.cuda.Stream(), torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            for _ in range(20):
                busy.add_(1)
        y = L.prefill(d["offsets"], 300, d["q"], d["k"], d["v"], d["a"], d["beta"], stream=stream)
        for _ in range(8):
            torch.empty(1 << 24, dtype=torch.uint8, device="cuda").fill_(255)
            torch.empty(y.numel(), device="cuda").fill_(float("nan"))
        torch.cuda.synchronize()
        yr, Sr = ref.run(kind, d, lens, torch.zeros(2, H, 128, V, device="cuda"))
        assert ref.slab_err(y, yr) <= TOL and ref.slab_err(L.S, Sr) <= TOL


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("call", ["prefill", "rmw_seq"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_token_stays_in_its_sequence(bad, call, kind):
    """A token of inf or NaN spoils its own sequence from (at most) 31 tokens before it on, and no other one."""
    lens, H, V, at = [70, 100, 66], 4, 80, 80
    d = ref.draw(kind, "bf16", lens, H, H, V, seed=6)
    for key in ("q", "k", "v"):
        d[key][70 + at] = bad
    L = _layer(kind, 3, H, V, H)
    fn = L.prefill if call == "prefill" else L.rmw_seq
    L.S.zero_()
    y = fn(d["offsets"], 100, d["q"], d["k"], d["v"], d["a"], d["beta"])
    clean = {key: None if d[key] is None else torch.nan_to_num(d[key], 0, 0, 0) if key in "qkv" else d[key]
             for key in d}
    yr, Sr = ref.run(kind, clean, lens, torch.zeros(3, H, 128, V, device="cuda"))
    fine = list(range(70 + at - 31)) + list(range(170, 236))
    assert ref.slab_err(y[fine], yr[fine]) <= TOL and ref.slab_err(L.S[[0, 2]], Sr[[0, 2]]) <= TOL
    assert not torch.isfinite(y[70 + at]).all()


@pytest.mark.timeout(120)
def test_workspace_of_the_callers():
    """One byte too few is refused, the stated size does, whatever stands behind it."""
    import rank_state_read_amd as lib
    lens, H, V = [200, 90], 4, 96
    d = ref.draw("gdn", "f32", lens, H, H, V, seed=7)
    sh = lib.make_shape(2, H, 128, V, 16, 1, 79, 49, "gdn", "f32", H)
    S, y = torch.empty(2, H, 128, V, device="cuda"), torch.empty(d["v"].shape, device="cuda")
    need = lib.sketchssm_prefill_workspace(sh, 2, 290, 200)
    assert need > 0
    work = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")

    def go(w):
        lib.sketchssm_prefill(sh, None, None, S, None, d["offsets"], 200, d["q"], d["k"], d["v"], d["a"], d["beta"], y,
                              workspace=w)

    with pytest.raises(lib.SketchSSMError):
        go(work[:need - 1])
    with pytest.raises(ValueError):
        go(torch.empty(need, dtype=torch.uint8))  # on the host
    with pytest.raises(ValueError):
        go(work[:2 * need:2])
    go(work[:need])
    torch.cuda.synchronize()
    yr, Sr = ref.run("gdn", d, lens, torch.zeros(2, H, 128, V, device="cuda"))
    assert ref.slab_err(S, Sr) <= TOL and ref.slab_err(y, yr) <= TOL
    assert (work[need:] == 77).all()
