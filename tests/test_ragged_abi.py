"""Argument checks of the ragged calls and the gated norm: refused on the host before any launch (no GPU needed)."""
import ctypes

import pytest

from rank_state_read_amd import binding as B

FAKE = 1 << 20  # a 16-byte-aligned stand-in address, never dereferenced
NAMES = ["S0", "n_rows0", "rows0", "S", "rows", "offsets", "n_seqs", "total", "max_len", "q", "k", "v", "a", "beta", "y"]


def _shape(kind="gdn", **kw):
    d = dict(B=4, H=8, K=128, V=80, W=16, G=1, basis_rows=79, rank_cap=49, kind=kind, qkv="bf16", kq_heads=0)
    d.update(kw)
    return B.make_shape(**d)


def _call(entry, shape, **over):
    a = dict(S0=FAKE, n_rows0=4, rows0=FAKE, S=FAKE, rows=FAKE, offsets=FAKE, n_seqs=2, total=10, max_len=6, q=FAKE,
             k=FAKE, v=FAKE, a=FAKE, beta=FAKE, y=FAKE)
    ws, size = over.pop("workspace", 1 << 24), over.pop("workspace_bytes", 1 << 40)
    a.update(over)
    args = [None if shape is None else ctypes.byref(shape)] + [a[n] for n in NAMES]
    L = B.lib()
    return L.sketchssm_rmw_seq(*args, None) if entry == "rmw_seq" else L.sketchssm_prefill(*args, ws, size, None)


@pytest.mark.parametrize("entry", ["rmw_seq", "prefill"])
def test_ragged_argument_errors(entry):
    gdn, mamba = _shape(), _shape("mamba2")
    assert _call(entry, None) == 1
    assert _call(entry, _shape(V=72)) == 2
    assert _call(entry, _shape(kq_heads=3)) == 2
    for key in ("S", "offsets", "q", "k", "v", "a", "y"):
        assert _call(entry, gdn, **{key: None}) == 1, key
    assert _call(entry, gdn, beta=None) == 1          # the delta rule needs beta
    assert _call(entry, mamba) == 1                   # Mamba-2 takes none
    assert _call(entry, gdn, S0=None) == 1            # rows0 without S0
    assert _call(entry, gdn, n_rows0=0) == 2
    assert _call(entry, gdn, n_rows0=1 << 17) == 2    # first states past 2^31 elements
    for key in ("n_seqs", "total", "max_len"):
        assert _call(entry, gdn, **{key: -1}) == 1, key
    for key in ("S0", "rows0", "S", "rows", "offsets", "q", "k", "v", "a", "beta", "y"):
        assert _call(entry, gdn, **{key: FAKE + 4}) == 3, key
    assert _call(entry, gdn, n_seqs=1 << 28) == 2     # blocks past 2^31
    assert _call(entry, gdn, n_seqs=0) == 0           # nothing to do


def test_prefill_workspace():
    gdn = _shape()
    assert _call("prefill", gdn, workspace=(1 << 24) + 8) == 3
    need = B.sketchssm_prefill_workspace(gdn, 3, 5000, 4000)
    assert B.sketchssm_prefill_workspace(gdn, -1, 5000, 4000) == 0
    assert B.sketchssm_prefill_workspace(_shape(V=72), 3, 5000, 4000) == 0
    if need:
        big = dict(n_seqs=3, total=5000, max_len=4000)
        assert _call("prefill", gdn, workspace=None, workspace_bytes=0, **big) == 1
        assert _call("prefill", gdn, workspace_bytes=need - 1, **big) == 2


def test_gated_norm_argument_errors():
    sh = _shape()

    def call(shape=sh, y=FAKE, skip=None, D=None, z=FAKE, w=FAKE, w_heads=8, heads=2, gate=2, eps=1e-5, n=3, out=FAKE):
        return B.lib().sketchssm_gated_norm(None if shape is None else ctypes.byref(shape), y, skip, D, z, w, w_heads,
                                           heads, gate, eps, n, out, None)

    assert call(shape=None) == 1
    assert call(shape=_shape(V=40)) == 2
    assert call(y=None) == 1 and call(out=None) == 1 and call(w=None) == 1
    assert call(z=None) == 1                      # a gate needs z
    assert call(gate=0) == 1                      # no gate takes none
    assert call(gate=4) == 1 and call(gate=-1) == 1
    assert call(skip=FAKE) == 1 and call(D=FAKE) == 1
    assert call(heads=3) == 2 and call(heads=0) == 2 and call(heads=16) == 2
    assert call(w_heads=2) == 2
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(n=-1) == 1 and call(n=0) == 0
    for key in ("y", "z", "w", "out"):
        assert call(**{key: FAKE + 8}) == 3, key
    assert call(shape=_shape(H=256), w_heads=256, heads=1, n=1 << 23) == 2  # groups past 2^31


def test_binding_refuses_wrong_tensors():
    """Types and shapes are refused before an address is taken."""
    torch = pytest.importorskip("torch")
    sh = _shape(V=64)
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    good = dict(S0=f(3, 8, 128, 64), rows0=i(2), S=f(4, 8, 128, 64), rows=i(2), offsets=i(3), max_len=5, q=b(9, 8, 128),
                k=b(9, 8, 128), v=b(9, 8, 64), a=f(9, 8), beta=f(9, 8), y=f(9, 8, 64))
    bad = dict(S0=f(3, 8, 64, 128), rows0=i(3), S=f(3, 8, 128, 64), rows=i(2).long(), offsets=i(3)[None], q=f(9, 8, 128),
               k=b(9, 4, 128), v=b(8, 8, 64), a=f(9, 8, 128), beta=b(9, 8), y=b(9, 8, 64))
    for fn in (B.sketchssm_rmw_seq, B.sketchssm_prefill):
        for key, x in bad.items():
            with pytest.raises(ValueError):
                fn(sh, **dict(good, **{key: x}))
        with pytest.raises(ValueError, match="device tensor"):
            fn(sh, **good)  # all as they should be, but on the host
    with pytest.raises(ValueError, match="rows"):
        B.sketchssm_rmw_seq(sh, **dict(good, rows=None, rows0=i(5), offsets=i(6)))
