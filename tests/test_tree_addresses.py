"""Addresses in place of tensors, and arguments left out, in the tree and cache calls: they pass through to the library as
in every other call, so that it is the library that answers (no GPU needed: the tensors are on the host, which is refused
last of all)."""
import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd import binding as B  # noqa: E402

FAKE = 1 << 20  # never dereferenced
f = torch.zeros


def b(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def i(n):
    return torch.zeros(n, dtype=torch.int32)


SHAPE = B.make_shape(4, 8, 128, 64, 16, 1, 79, 49, "gdn", "bf16", 0)


@pytest.mark.parametrize("given", [FAKE, None])
@pytest.mark.parametrize("key", ["S", "kbuf", "vbuf", "abuf", "bbuf", "pos", "rows", "parents", "q", "k", "a", "beta", "y"])
def test_tree_read(key, given):
    plan = B.Plan(SHAPE, [0] * 8, [0] * 8)
    d = dict(S=f(4, 8, 128, 64), Z=None, frames=None, kbuf=b(16, 8, 4, 128), vbuf=b(16, 8, 4, 64), abuf=f(16, 8, 4),
             bbuf=f(16, 8, 4), pos=i(4), rows=i(2), offsets=i(3), max_nodes=6, parents=i(9), q=b(9, 8, 128), k=b(9, 8, 128),
             v=b(9, 8, 64), a=f(9, 8), beta=f(9, 8), y=f(9, 8, 64))
    with pytest.raises(ValueError, match="device tensor"):
        B.sketchssm_tree_read(plan, **dict(d, **{key: given}))


@pytest.mark.parametrize("fn", [B.sketchssm_cache_store, B.sketchssm_cache_load])
def test_caches(fn):
    d = dict(S=f(4, 8, 128, 64), rows=i(2), slots=i(2), codes=torch.zeros(5, 8, 128, 64, dtype=torch.int8), scales=b(5, 8, 128),
             format="i8")
    for key in ("rows", "slots", "scales"):
        with pytest.raises(ValueError, match="device tensor"):
            fn(SHAPE, **dict(d, **{key: FAKE}))
    for lists in (dict(rows=FAKE, slots=FAKE), dict(rows=FAKE, slots=None), dict(rows=None, slots=FAKE)):
        with pytest.raises(ValueError, match="number of pairs"):  # no tensor says it
            fn(SHAPE, **dict(d, **lists))
