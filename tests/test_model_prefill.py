"""The model's prompt call on stand-in layers (no GPU): every layer sees its packed prompts once and in order, the
first sketches follow, gated outputs where tokens hold a gate, and inconsistent set-ups are refused."""
import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd.model import SketchModel  # noqa: E402


class _Layer:
    W, B = 4, 3

    def __init__(self, name, log):
        self.name, self.log = name, log

    def flush(self, n, stream=None):
        self.log.append((self.name, "flush", n, stream))

    def prefill(self, offsets, max_len, q, k, v, a, beta=None, stream=None):
        self.log.append((self.name, "prefill", offsets.tolist(), max_len, q, beta, stream))
        return f"y-{self.name}"

    def read(self, pos, q, k, v, a, beta=None, stream=None):
        self.log.append((self.name, "read", pos))
        return f"y-{self.name}"

    def gated_norm(self, y, z, v=None, stream=None):
        self.log.append((self.name, "norm", y, z, v, stream))
        return f"n-{self.name}"


def _tokens(n, **more):
    return [dict({"q": i, "k": None, "v": f"v{i}", "a": None}, **more) for i in range(n)]


def test_prompts_then_first_sketches():
    log = []
    m = SketchModel([_Layer(i, log) for i in range(2)])
    m.pos = 3
    off = torch.tensor([0, 5, 5, 9], dtype=torch.int32)
    assert m.prefill(_tokens(2), off, 5, stream=7) == ["y-0", "y-1"]
    assert log == [(i, "prefill", [0, 5, 5, 9], 5, i, None, 7) for i in range(2)] + [(i, "flush", 0, 7) for i in
                                                                                      range(2)]
    assert m.pos == 0


def test_gated_outputs():
    log = []
    m = SketchModel([_Layer(i, log) for i in range(2)])
    toks = _tokens(2)
    toks[1]["z"], toks[1]["beta"] = "z1", "b1"
    off = torch.zeros(4, dtype=torch.int32)
    assert m.prefill(toks, off, 0) == ["y-0", "n-1"]
    assert (1, "norm", "y-1", "z1", "v1", None) in log and log[1][5] == "b1"
    log.clear()
    assert m.decode_step(toks) == ["y-0", "n-1"]
    assert log == [(0, "read", 0), (1, "read", 0), (1, "norm", "y-1", "z1", "v1", None)]


def test_refusals():
    m = SketchModel([_Layer(i, []) for i in range(2)])
    with pytest.raises(ValueError, match="per layer"):
        m.prefill(_tokens(1), torch.zeros(4, dtype=torch.int32), 1)
    with pytest.raises(ValueError, match="per sequence"):
        m.prefill(_tokens(2), torch.zeros(3, dtype=torch.int32), 1)
