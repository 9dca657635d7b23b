"""Numbers that do not fit the C calls' 32 bits are refused by the binding: cut to 32 bits a bound of 2^32 would become
0 and idle every sequence (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

from rank_state_read_amd import binding as B  # noqa: E402
from test_ragged_first_rows import _args  # noqa: E402


@pytest.mark.parametrize("max_len", [-2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63 - 1])
@pytest.mark.parametrize("fn", [B.sketchssm_rmw_seq, B.sketchssm_prefill])
def test_max_len(fn, max_len):
    with pytest.raises(ValueError, match="max_len"):
        fn(**dict(_args(), max_len=max_len))


def test_workspace():
    sh = _args()["shape"]
    ok = dict(n_seqs=2, total_tokens=500, max_len=400)
    assert B.sketchssm_prefill_workspace(sh, **ok) > 0
    assert B.sketchssm_prefill_workspace(sh, **dict(ok, max_len=2 ** 31 - 1)) > 0
    assert B.sketchssm_prefill_workspace(sh, **dict(ok, n_seqs=-1)) == 0  # as the C call says
    for key in ok:
        with pytest.raises(ValueError, match=key):
            B.sketchssm_prefill_workspace(sh, **dict(ok, **{key: 2 ** 32 + 400}))
