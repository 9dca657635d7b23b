"""The model's tree and cache calls on stand-in layers (no GPU): every layer is called once and in order with the
model's lists, gated outputs where a layer has a norm, and inconsistent set-ups are refused."""
import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd.model import SketchModel  # noqa: E402


class _Layer:
    W, B = 4, 3

    def __init__(self, name, log, norm=None):
        self.name, self.log, self.norm = name, log, norm

    def tree_read(self, offsets, max_nodes, parents, q, k, v, a, beta=None, pos=None, rows=None, stream=None):
        self.log.append((self.name, "read", offsets, max_nodes, parents, q, k, v, a, beta, pos, rows, stream))
        return f"y-{self.name}"

    def tree_accept(self, offsets, parents, accepted, k, v, a, beta=None, *, pos, rows=None, new_pos=None, stream=None):
        self.log.append((self.name, "accept", offsets, parents, accepted, k, v, a, beta, pos, rows, new_pos, stream))
        return "new" if new_pos is None else new_pos

    def gated_norm(self, y, z, v=None, stream=None):
        self.log.append((self.name, "norm", y, z, v, stream))
        return f"n-{self.name}"

    def flush_seq(self, rows, n, stream=None):
        self.log.append((self.name, "flush", rows, n, stream))

    def new_cache(self, n, fmt):
        return (self.name, n, fmt)

    def cache_store(self, c, rows, slots, stream=None):
        self.log.append((self.name, "store", c, rows, slots, stream))

    def cache_load(self, c, slots, rows, stream=None):
        self.log.append((self.name, "load", c, slots, rows, stream))

    def zeros_like(self, x, stream=None):
        return f"0-{x}"


def _tokens(n):
    return [{"q": f"q{i}", "k": f"k{i}", "v": f"v{i}", "a": f"a{i}"} for i in range(n)]


def test_read_and_accept():
    log = []
    m = SketchModel([_Layer(0, log), _Layer(1, log, norm=(None, 1, "silu", 1e-5, None))])
    toks = _tokens(2)
    toks[1]["z"], toks[1]["beta"] = "z1", "b1"
    assert m.tree_read(toks, "par", "off", 9, pos="pos", rows="rows", stream=5) == ["y-0", "n-1"]
    assert log == [(0, "read", "off", 9, "par", "q0", "k0", "v0", "a0", None, "pos", "rows", 5),
                   (1, "read", "off", 9, "par", "q1", "k1", "v1", "a1", "b1", "pos", "rows", 5),
                   (1, "norm", "y-1", "z1", "v1", 5)]
    log.clear()
    assert m.tree_accept(toks, "par", "off", "acc", "pos", rows="rows") == "new"
    assert log == [(0, "accept", "off", "par", "acc", "k0", "v0", "a0", None, "pos", "rows", None, None),
                   (1, "accept", "off", "par", "acc", "k1", "v1", "a1", "b1", "pos", "rows", "new", None)]
    assert m.pos == 0


def test_caches():
    log = []
    m = SketchModel([_Layer(i, log) for i in range(2)])
    caches = m.new_cache(7, "e4m3")
    assert caches == [(0, 7, "e4m3"), (1, 7, "e4m3")]
    m.cache_store(caches, "rows", "slots", stream=3)
    assert log == [(i, "store", caches[i], "rows", "slots", 3) for i in range(2)]
    log.clear()
    m.cache_load(caches, "slots", "rows")
    assert log == [x for i in range(2) for x in ((i, "load", caches[i], "slots", "rows", None),
                                                 (i, "flush", "rows", "0-rows", None))]
    log.clear()
    m.flush_seq("rows", "n")
    assert log == [(i, "flush", "rows", "n", None) for i in range(2)]


def test_refusals():
    log = []
    m = SketchModel([_Layer(0, log), _Layer(1, log, norm=(None, 1, "silu", 1e-5, None))])
    with pytest.raises(ValueError, match="per layer"):
        m.tree_read(_tokens(1), "par", "off", 1)
    with pytest.raises(ValueError, match="per layer"):
        m.tree_accept(_tokens(3), "par", "off", "acc", "pos")
    with pytest.raises(ValueError, match="no gate"):
        m.tree_read(_tokens(2), "par", "off", 1)
    for call in (m.cache_store, m.cache_load):
        with pytest.raises(ValueError, match="per layer"):
            call([1], "rows", "slots")
    assert log == []
