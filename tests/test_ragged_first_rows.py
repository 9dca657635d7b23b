"""A list of first rows needs the states it names: without them the binding's calls are refused, as the C calls are,
and never start from zero instead (no GPU needed: refused before anything is launched)."""
import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd import binding as B  # noqa: E402


class _Called(Exception):
    pass


def _args():
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    sh = B.make_shape(4, 8, 128, 64, 16, 1, 79, 49, "gdn", "bf16", 0)
    return dict(shape=sh, S0=f(3, 8, 128, 64), rows0=i(2), S=f(4, 8, 128, 64), rows=i(2), offsets=i(3), max_len=5,
                q=b(9, 8, 128), k=b(9, 8, 128), v=b(9, 8, 64), a=f(9, 8), beta=f(9, 8), y=f(9, 8, 64))


@pytest.mark.parametrize("fn", [B.sketchssm_rmw_seq, B.sketchssm_prefill])
@pytest.mark.parametrize("S0", ["none", "no rows"])
def test_first_rows_without_first_states(fn, S0):
    args = dict(_args(), S0=None if S0 == "none" else torch.zeros(0, 8, 128, 64))
    with pytest.raises(ValueError, match="rows0"):
        fn(**args)


@pytest.mark.parametrize("S0", ["given", "none"])
def test_what_the_library_gets(S0):
    """The list goes with its states; without both every sequence starts from zero."""
    args = _args()
    if S0 == "none":
        args.update(S0=None, rows0=None)
    got = B._ragged(**args)
    assert got[1:4] == ([args["S0"].data_ptr(), 3, args["rows0"].data_ptr()] if S0 == "given" else [None, 0, None])


def test_layer_with_fresh_rows(monkeypatch):
    """A layer's prompt call that names first rows but starts its rows from zero contradicts itself."""
    from rank_state_read_amd.layer import SketchLayer
    L = SketchLayer.__new__(SketchLayer)
    a = _args()
    L.shape, L.S, L.device = a["shape"], a["S"], a["S"].device
    call = lambda **kw: L.prefill(a["offsets"], 5, a["q"], a["k"], a["v"], a["a"], a["beta"], a["rows"],  # noqa: E731
                                  rows0=a["rows0"], y=a["y"], **kw)
    with pytest.raises(ValueError, match="rows0"):
        call()

    def on_device(device, stream):
        raise _Called
    monkeypatch.setattr(B, "_on_device", on_device)
    for kw in (dict(S0=a["S0"]), dict(fresh=False)):  # these go on to the library
        with pytest.raises(_Called):
            call(**kw)
