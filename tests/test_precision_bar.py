"""What the bars of test_prefill_precision_gpu.py can see, by the same arithmetic on the CPU: fp32 products as sums of
products of bf16 terms, with three terms and with two, terms cut off and terms rounded."""
import numpy as np
import pytest

U = 2.0 ** -24
BAR = 16 * U


def _bits(x):
    return x.astype(np.float32).view(np.uint32)


def _cut(x):
    return (_bits(x) & np.uint32(0xFFFF0000)).view(np.float32)


def _round(x):
    b = _bits(x)
    return ((b + np.uint32(0x7FFF) + ((b >> np.uint32(16)) & np.uint32(1))) & np.uint32(0xFFFF0000)).view(np.float32)


def _terms(x, how, n):
    out = []
    for _ in range(n):
        out.append(how(x))
        x = x - out[-1]
    return out, x


def _product(a, b, how_a, how_b, n):
    """a b with terms i of a and j of b where i + j < n."""
    ta, tb = _terms(a, how_a, n)[0], _terms(b, how_b, n)[0]
    return sum(ta[i].astype(np.float64) @ tb[j] for i in range(n) for j in range(n - i))


@pytest.fixture(scope="module")
def operands():
    g = np.random.default_rng(0)
    return g.standard_normal((256, 128)).astype(np.float32), g.standard_normal((128, 256)).astype(np.float32)


@pytest.mark.parametrize("how", [_cut, _round])
def test_three_terms_hold_the_number(operands, how):
    assert (_terms(operands[0], how, 3)[1] == 0).all()


def _off(operands, *how):
    a, b = operands
    want = a.astype(np.float64) @ b
    return np.linalg.norm(_product(a, b, *how) - want) / np.linalg.norm(want)


def test_two_terms_are_above_the_bar(operands):
    assert _off(operands, _cut, _cut, 3) <= 2 * U and _off(operands, _round, _cut, 3) <= U
    assert _off(operands, _cut, _cut, 2) >= 400 * U > BAR  # one-sided
    assert _off(operands, _round, _cut, 2) >= 150 * U > BAR
    assert _off(operands, _round, _round, 2) >= 60 * U > BAR


def test_lean(operands):
    """Two operands that are cut lean to one side, one that is rounded takes the lean away (positive operands)."""
    a, b = (np.abs(x) for x in operands)
    want = a.astype(np.float64) @ b
    mean = lambda *how: float(((_product(a, b, *how) - want) / want).mean()) / U  # noqa: E731
    assert mean(_cut, _cut, 3) < -0.5 and abs(mean(_round, _cut, 3)) < 0.02
