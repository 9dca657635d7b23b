"""Argument checks of the tree calls and the 8-bit cache: refused on the host before any launch (no GPU needed)."""
import ctypes

import pytest

from rank_state_read_amd import binding as B

FAKE = 1 << 20  # a 16-byte-aligned stand-in address, never dereferenced


def _shape(kind="gdn", **kw):
    d = dict(B=4, H=8, K=128, V=80, W=16, G=1, basis_rows=79, rank_cap=49, kind=kind, qkv="bf16", kq_heads=0)
    d.update(kw)
    return B.make_shape(**d)


def _plan(kind="gdn", ranks=(0, 3, 0, 5, 6, 7, 8, 9), **kw):
    return B.Plan(_shape(kind, **kw), list(ranks), [0] * len(ranks))


READ = ["S", "Z", "frames", "kbuf", "vbuf", "abuf", "bbuf", "pos", "rows", "offsets", "n_seqs", "total", "max_nodes",
        "parents", "q", "k", "v", "a", "beta", "y"]
ACCEPT = ["kbuf", "vbuf", "abuf", "bbuf", "pos", "new_pos", "rows", "offsets", "n_seqs", "total", "parents", "accepted",
          "k", "v", "a", "beta"]
NUMBERS = {"n_seqs": 2, "total": 10, "max_nodes": 6}


def _read(plan, **over):
    a = {n: NUMBERS.get(n, FAKE) for n in READ}
    a.update(over)
    return B.lib().sketchssm_tree_read(None if plan is None else plan.handle, *[a[n] for n in READ], None)


def _accept(shape, **over):
    a = {n: NUMBERS.get(n, FAKE) for n in ACCEPT}
    a["new_pos"] = 2 * FAKE
    a.update(over)
    return B.lib().sketchssm_tree_accept(None if shape is None else ctypes.byref(shape), *[a[n] for n in ACCEPT], None)


def test_read_argument_errors():
    mixed, dense, sketch, mamba = _plan(), _plan(ranks=[0] * 8), _plan(ranks=[4] * 8), _plan("mamba2")
    assert _read(None) == 1
    for key in ("S", "Z", "frames", "kbuf", "vbuf", "abuf", "bbuf", "offsets", "parents", "q", "k", "v", "a", "beta", "y"):
        assert _read(mixed, **{key: None}) == 1, key
    for key in NUMBERS:
        assert _read(mixed, **{key: -1}) == 1, key
    assert _read(mixed, max_nodes=65) == 2
    assert _read(mixed, n_seqs=1 << 27) == 2
    assert _read(mamba) == 1 and _read(mamba, bbuf=None) == 1 and _read(mamba, beta=None) == 1
    for key in READ:
        if key not in NUMBERS:
            assert _read(mixed, **{key: FAKE + 4}) == 3, key
    # nothing to do
    assert _read(mixed, n_seqs=0) == 0 and _read(mixed, total=0) == 0 and _read(mixed, max_nodes=0) == 0
    assert _read(mixed, n_seqs=0, pos=None, kbuf=None, vbuf=None, abuf=None, bbuf=None, rows=None) == 0
    assert _read(dense, n_seqs=0, Z=None, frames=None) == 0 and _read(sketch, n_seqs=0, S=None) == 0
    assert _read(mixed, n_seqs=0, total=0, parents=None, q=None, k=None, v=None, a=None, beta=None, y=None) == 0


def test_accept_argument_errors():
    gdn, mamba = _shape(), _shape("mamba2")
    assert _accept(None) == 1 and _accept(_shape(V=72)) == 2
    for key in ("kbuf", "vbuf", "abuf", "bbuf", "pos", "new_pos", "offsets", "parents", "accepted", "k", "v", "a", "beta"):
        assert _accept(gdn, **{key: None}) == 1, key
    assert _accept(mamba) == 1 and _accept(mamba, beta=None) == 1 and _accept(mamba, bbuf=None) == 1
    assert _accept(gdn, new_pos=FAKE) == 1  # in place
    assert _accept(gdn, n_seqs=-1) == 1 and _accept(gdn, total=-1) == 1
    assert _accept(gdn, n_seqs=1 << 30) == 2
    for key in ACCEPT:
        if key not in NUMBERS:
            assert _accept(gdn, **{key: FAKE + 4}) == 3, key


def test_cache_argument_errors():
    sh, L = _shape(), B.lib()

    def store(shape=sh, S=FAKE, rows=FAKE, codes=FAKE, scales=FAKE, slots=FAKE, n_slots=4, n=2, fmt=0):
        return L.sketchssm_cache_store(None if shape is None else ctypes.byref(shape), S, rows, codes, scales, slots,
                                       n_slots, n, fmt, None)

    def load(shape=sh, S=FAKE, rows=FAKE, codes=FAKE, scales=FAKE, slots=FAKE, n_slots=4, n=2, fmt=0):
        return L.sketchssm_cache_load(None if shape is None else ctypes.byref(shape), codes, scales, slots, n_slots, S,
                                      rows, n, fmt, None)

    for call in (store, load):
        assert call(shape=None) == 1 and call(shape=_shape(V=40)) == 2
        for key in ("S", "codes", "scales"):
            assert call(**{key: None}) == 1, key
        assert call(fmt=2) == 1 and call(fmt=-1) == 1 and call(n=-1) == 1 and call(n_slots=-1) == 1
        for key in ("S", "codes", "scales", "rows", "slots"):
            assert call(**{key: FAKE + 8}) == 3, key
        assert call(n=1 << 20) == 2  # more threads than a launch counts
        assert call(n=0) == 0 and call(n=0, rows=None, slots=None) == 0


def _tensors(torch):
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    plan = _plan(V=64)
    window = dict(kbuf=b(16, 8, 4, 128), vbuf=b(16, 8, 4, 64), abuf=f(16, 8, 4), bbuf=f(16, 8, 4), pos=i(4))
    tree = dict(rows=i(2), offsets=i(3), parents=i(9), k=b(9, 8, 128), v=b(9, 8, 64), a=f(9, 8), beta=f(9, 8))
    bad = dict(kbuf=b(16, 4, 8, 128), vbuf=f(16, 8, 4, 64), abuf=f(16, 8, 4, 128), bbuf=f(4, 8, 16), pos=i(3), rows=i(3),
               offsets=i(3)[None], parents=i(8), k=b(9, 4, 128), v=b(9, 8, 80), a=b(9, 8), beta=f(8, 8))
    return plan, dict(window, **tree), bad, f, b, i


def test_binding_refuses_wrong_tensors():
    """Types and shapes are refused before an address is taken."""
    torch = pytest.importorskip("torch")
    plan, common, bad, f, b, i = _tensors(torch)
    good = dict(common, S=f(4, 8, 128, 64), Z=f(plan.z_elems), frames=f(plan.frame_elems), max_nodes=6, q=b(9, 8, 128),
                y=f(9, 8, 64))
    for key, x in dict(bad, S=f(3, 8, 128, 64), Z=f(plan.z_elems - 1), frames=b(plan.frame_elems), q=f(9, 8, 128),
                       y=b(9, 8, 64), max_nodes=1 << 32).items():
        with pytest.raises(ValueError):
            B.sketchssm_tree_read(plan, **dict(good, **{key: x}))
    with pytest.raises(ValueError, match="rows"):
        B.sketchssm_tree_read(plan, **dict(good, rows=None, offsets=i(6)))
    with pytest.raises(ValueError, match="device tensor"):
        B.sketchssm_tree_read(plan, **good)  # all as they should be, but on the host
    good = dict(common, new_pos=i(4), accepted=i(2))
    for key, x in dict(bad, new_pos=i(5), accepted=i(3)).items():
        with pytest.raises(ValueError):
            B.sketchssm_tree_accept(plan.shape, **dict(good, **{key: x}))
    with pytest.raises(ValueError, match="device tensor"):
        B.sketchssm_tree_accept(plan.shape, **good)


def test_binding_refuses_wrong_caches():
    torch = pytest.importorskip("torch")
    sh = _shape(V=64)
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    good = dict(S=torch.zeros(4, 8, 128, 64), rows=i(2), slots=i(2), codes=torch.zeros(5, 8, 128, 64, dtype=torch.int8),
                scales=torch.zeros(5, 8, 128, dtype=torch.bfloat16), format="i8")
    bad = dict(S=torch.zeros(4, 8, 64, 128), rows=i(3), slots=i(2).long(), codes=good["codes"].view(torch.float8_e4m3fn),
               scales=torch.zeros(5, 8, 128), format="e4m3")
    for fn in (B.sketchssm_cache_store, B.sketchssm_cache_load):
        for key, x in bad.items():
            with pytest.raises(ValueError):
                fn(sh, **dict(good, **{key: x}))
        with pytest.raises(KeyError):
            fn(sh, **dict(good, format="i4"))
        with pytest.raises(ValueError, match="rows"):
            fn(sh, **dict(good, rows=None, slots=i(5)))
        with pytest.raises(ValueError, match="slots"):
            fn(sh, **dict(good, slots=None, rows=i(6)))
        with pytest.raises(ValueError, match="device tensor"):
            fn(sh, **good)


def test_state_cache_object():
    torch = pytest.importorskip("torch")
    from rank_state_read_amd.layer import StateCache
    c = StateCache(3, 2, 128, 64, "e4m3", device="cpu")
    assert c.codes.shape == (3, 2, 128, 64) and c.codes.dtype == torch.float8_e4m3fn
    assert c.scales.shape == (3, 2, 128) and c.scales.dtype == torch.bfloat16
    with pytest.raises(KeyError):
        StateCache(3, 2, 128, 64, "fp8", device="cpu")


def test_outputs_apart_from_inputs():
    """y may not overlap a node's inputs, new_pos not pos: other blocks still read them."""
    plan = _plan()
    far = {n: (i + 1) << 30 for i, n in enumerate(READ) if n not in NUMBERS}
    nbytes = {"q": 10 * 8 * 128 * 2, "k": 10 * 8 * 128 * 2, "v": 10 * 8 * 80 * 2, "a": 10 * 8 * 4, "beta": 10 * 8 * 4}
    for key, n in nbytes.items():
        for y in (far[key], far[key] + n - 16, far[key] - 10 * 8 * 80 * 4 + 16):
            assert _read(plan, **dict(far, y=y)) == 1, key
    for new in (FAKE, FAKE + 16, FAKE - 16):
        assert _accept(_shape(B=8), new_pos=new) == 1
