"""The gated norm at the widths between which its teams change, against its formula in 64 bits (the bounds are
those of `_norm_case`)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_ragged_gpu import _need_gpu, _norm_case  # noqa: E402,F401


@pytest.mark.timeout(300)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("H,V,heads", [(6, 128, 1), (6, 128, 2), (6, 96, 3), (20, 64, 10), (8, 128, 8), (13, 80, 13),
                                       (32, 64, 32), (26, 80, 26), (32, 128, 32), (52, 80, 52), (64, 128, 64),
                                       (103, 80, 103), (128, 128, 128), (129, 128, 129)])
def test_widths(qkv, H, V, heads):
    for n in (1, 18):
        _norm_case(qkv, H, V, n, heads, "sigmoid", True, False, seed=n)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("n", [2730, 2731, 4097])
def test_number_of_groups(n):
    """Groups of 160 values around the number at which their team changes (8190, 8193 and 12291 of them)."""
    _norm_case("bf16", 6, 80, n, 2, "silu", False, False, seed=n)
