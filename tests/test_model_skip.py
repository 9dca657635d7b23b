"""A Mamba-2 layer's skip is D x, and its update takes dt x: the model's tokens may hold x beside v (stand-in layers,
no GPU)."""
import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd.model import SketchModel  # noqa: E402
from test_model_prefill import _Layer, _tokens  # noqa: E402


def _skips(log):
    return [e[4] for e in log if e[1] == "norm"]


def test_skip_takes_x_where_the_tokens_hold_it():
    log = []
    m = SketchModel([_Layer(i, log) for i in range(3)])
    toks = _tokens(3, z="z")
    toks[0]["x"], toks[2]["x"] = "x0", None  # the others: v is x itself
    m.prefill(toks, torch.zeros(4, dtype=torch.int32), 0)
    assert _skips(log) == ["x0", "v1", "v2"]
    log.clear()
    m.decode_step(toks)
    assert _skips(log) == ["x0", "v1", "v2"]
