"""Which layers of a model are normed: those with set_norm, whatever their gate, and what their tokens have to hold is
asked for before any layer has run (stand-in layers, no GPU)."""
import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd.layer import SketchLayer  # noqa: E402
from rank_state_read_amd.model import SketchModel  # noqa: E402
from test_model_prefill import _Layer, _tokens  # noqa: E402

OFF = torch.zeros(4, dtype=torch.int32)


def _layer(name, log, gate):
    L = _Layer(name, log)
    L.norm, L.device = None, "cpu"
    if gate is not None:
        SketchLayer.set_norm(L, torch.ones(64), 1, gate)
    return L


def _calls(tokens, gates):
    for call in (lambda m, t: m.prefill(t, OFF, 0), lambda m, t: m.decode_step(t)):
        log = []
        yield log, call, SketchModel([_layer(i, log, g) for i, g in enumerate(gates)]), tokens


@pytest.mark.parametrize("gate", ["none", 0])
def test_norm_without_gate(gate):
    """A norm that takes no gate is applied to tokens without one."""
    for log, call, m, toks in _calls(_tokens(2), [gate, None]):
        assert call(m, toks) == ["n-0", "y-1"]
        assert [e for e in log if e[1] == "norm"] == [(0, "norm", "y-0", None, "v0", None)]


def test_gate_of_a_layer_without_norm():
    """Tokens may hold a gate that the caller applies: such a layer returns its y, as it did before there were norms."""
    for log, call, m, toks in _calls(_tokens(2, z="z"), [None, "silu"]):
        assert call(m, toks) == ["y-0", "n-1"]


@pytest.mark.parametrize("gate,z", [("silu", None), ("silu_first", None), (3, None), ("none", "z"), (0, "z")])
def test_gate_missing_or_too_many(gate, z):
    """Refused before the first layer's state or window has changed."""
    toks = _tokens(2)
    toks[1]["z"] = z
    for log, call, m, toks in _calls(toks, [None, gate]):
        with pytest.raises(ValueError, match="layer 1.*z"):
            call(m, toks)
        assert log == [] and m.pos == 0
