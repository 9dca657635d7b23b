"""How near the exact recurrence the ragged calls come: as near as fp32 arithmetic, which the 1e-4 of a slab that the
other tests ask for does not show.

Errors are taken as 2-norms, of a sequence's y and last state, relative to the exact ones, with keys of length 1 and
decays and beta in (0, 1], where rounding errors do not grow.  With u = 2^-24 a rounding to nearest is off by u / sqrt(3)
of the value in the mean square, and independent ones add as squares.  An output passes at most about 30 of them in a
sum of 128 channels and 32 tokens (an instruction adds 32 products at a time, in 3 or 6 terms each): 3.2 u.  The state,
w and y are such sums one after the other: 5.5 u.  The state's own error is carried on: where a chunk's decays leave
0.95 of it (the slow decays below), it grows by 1 / sqrt(1 - 0.95^2) = 3.2 of a chunk's 1.6 u, and a cut sequence's join
is a sum of 128 more, 3.3 u.  All of them together: 8.4 u.  The bar is 16 u, twice that.  Two bf16 terms of an operand
instead of three would put a product off by 75 u to 450 u (test_precision_bar.py)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ragged_reference as ref  # noqa: E402

U = 2.0 ** -24
BAR = 16 * U
KINDS = ["mamba2", "gdn", "kda"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rank_state_read_amd import binding
    binding.lib()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _go(call, kind, qkv, d, lens, H, Hk, V, S0):
    import rank_state_read_amd as lib
    n = len(lens)
    sh = lib.make_shape(n, H, 128, V, 16, 1, 79, 49, kind, qkv, Hk)
    S, y = torch.empty(n, H, 128, V, device="cuda"), torch.empty(d["v"].shape, device="cuda")
    fn = lib.sketchssm_rmw_seq if call == "rmw_seq" else lib.sketchssm_prefill
    fn(sh, S0, None, S, None, d["offsets"], max(lens), d["q"], d["k"], d["v"], d["a"], d["beta"], y)
    torch.cuda.synchronize()
    return y, S


def _err(got, want):
    return float((got.double() - want).norm() / want.norm())


def _check(call, kind, qkv, lens, H, Hk, V, seed=0, slow=False):
    d = ref.draw(kind, qkv, lens, H, Hk, V, seed)
    if slow:
        d["a"] = d["a"] ** 0.02
    y, S = _go(call, kind, qkv, d, lens, H, Hk, V, d["S0"])
    yr, Sr = ref.run(kind, d, lens, d["S0"])
    off = d["offsets"].tolist()
    worst = (0.0, 0.0)
    for i, n in enumerate(lens):
        if n:
            worst = max(worst[0], _err(y[off[i]:off[i + 1]], yr[off[i]:off[i + 1]])), max(worst[1], _err(S[i], Sr[i]))
    print(f"  {call} {kind} {qkv} H={H}/{Hk} V={V} {len(lens)} sequences: y {worst[0] / U:.1f} u, S {worst[1] / U:.1f} u",
          flush=True)
    assert max(worst) <= BAR
    return d, y, yr


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [64, 80, 96, 112, 128])
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
def test_chunks(qkv, V, kind):
    _check("prefill", kind, qkv, [300, 45], 6, 3, V)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
def test_recurrent(qkv, kind):
    _check("rmw_seq", kind, qkv, [9, 1, 40], 6, 3, 80)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [80, 128])
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
def test_segments(qkv, V, kind):
    import rank_state_read_amd as lib
    sh = lib.make_shape(1, 2, 128, V, 16, 1, 79, 49, kind, qkv, 1)
    assert lib.sketchssm_prefill_workspace(sh, 1, 1030, 1030) > lib.sketchssm_prefill_workspace(sh, 1, 1030, 64)
    _check("prefill", kind, qkv, [1030], 2, 1, V, slow=True)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind,qkv", [("kda", "bf16"), ("kda", "f32"), ("gdn", "f32"), ("mamba2", "f32")])
def test_all_columns_in_a_block(kind, qkv):
    _check("prefill", kind, qkv, [33 + (7 * i) % 40 for i in range(70)], 6, 6, 128)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("V", [80, 96])
def test_two_heads_in_a_block(V):
    _check("prefill", "mamba2", "bf16", [70, 33, 64, 65, 40, 90, 31, 32, 33, 44, 51, 35], 48, 8, V)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
def test_no_growth_along_a_sequence(qkv, kind):
    """With these decays (0.93 a token) a state forgets in 100 tokens, so the errors of the last 500 of 2500 tokens
    are those of the first 500, a mean over more than 60000 values on both sides; twice that leaves room for the start."""
    d, y, yr = _check("prefill", kind, qkv, [2500], 2, 1, 64)
    first, last = _err(y[:500], yr[:500]), _err(y[-500:], yr[-500:])
    print(f"    first {first / U:.2f} u, last {last / U:.2f} u", flush=True)
    assert last <= 2 * first


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind,qkv", [("mamba2", "bf16"), ("mamba2", "f32"), ("kda", "bf16")])
def test_products_lean_to_no_side(kind, qkv):
    """Products of fp32 operands leave out what is below the terms they take, which must not have the sign of the
    product every time.  With positive operands throughout, decays of 1 (whose products are exact) and for KDA beta = 0
    (y is the product of q and the first state alone), the errors' mean is 0: of the 5.5 u in the mean square, those of
    sums are independent from value to value, and those of a token's products (P) are shared by the columns of a head,
    so at least 64 tokens of 16 heads are independent, 5.5 u / 32 = 0.17 u.  The bar is 1.5 times that.  (Both operands
    cut off instead of one of them rounded: -0.69 u a product, test_precision_bar.py.)"""
    H, V, lens = 16, 80, [64]
    d = ref.draw(kind, qkv, lens, H, H, V, seed=5)
    for key in ("q", "k", "v"):
        d[key] = d[key].abs()
    if d["beta"] is not None:
        d["beta"].zero_()
    d["a"].fill_(1)
    S0 = d["S0"].abs()
    y, S = _go("prefill", kind, qkv, d, lens, H, H, V, S0)
    yr, Sr = ref.run(kind, d, lens, S0)
    e = ((y.double() - yr) / yr).mean().item()
    eS = ((S.double() - Sr) / Sr).mean().item()
    print(f"  {kind} {qkv}: mean error of y {e / U:.3f} u, of S {eS / U:.3f} u", flush=True)
    assert abs(e) <= 0.25 * U
    assert abs(eS) <= 0.25 * U
