"""The order in which the ragged calls take their sequences, which no result may depend on.

Tolerance: the ragged calls' 1e-4 of a slab's largest value."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import ragged_reference as ref  # noqa: E402

TOL = 1e-4
KINDS = ["mamba2", "gdn", "kda"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rank_state_read_amd import binding
    binding.lib()


def _go(call, kind, H, V, d, S0, rows0, S, rows, offsets, max_len, y):
    import rank_state_read_amd as lib
    sh = lib.make_shape(S.shape[0], H, 128, V, 16, 1, 79, 49, kind, "bf16", H)
    fn = lib.sketchssm_rmw_seq if call == "rmw_seq" else lib.sketchssm_prefill
    fn(sh, S0, rows0, S, rows, torch.tensor(offsets, dtype=torch.int32, device="cuda"), max_len, d["q"], d["k"],
       d["v"], d["a"], d["beta"], y)
    torch.cuda.synchronize()


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("call", ["rmw_seq", "prefill"])
@pytest.mark.parametrize("n", [64, 65, 130, 200])
def test_a_few_long_sequences_among_many(n, call, kind):
    """More waves than the CUs hold at once; long sequences first, in the middle and last."""
    lens = [i % 4 for i in range(n)]
    for at, length in ((0, 40), (n // 2, 61), (n - 2, 17), (n - 1, 50)):
        lens[at] = length
    H, V = 16, 128
    d = ref.draw(kind, "bf16", lens, H, H, V, seed=n)
    S, y = torch.full((n, H, 128, V), 7.0, device="cuda"), torch.empty(d["v"].shape, device="cuda")
    _go(call, kind, H, V, d, d["S0"], None, S, None, d["offsets"].tolist(), 61, y)
    yr, Sr = ref.run(kind, d, lens, d["S0"])
    assert ref.slab_err(S, Sr) <= TOL and ref.slab_err(y, yr) <= TOL


@pytest.mark.timeout(300)
@pytest.mark.parametrize("call", ["rmw_seq", "prefill"])
@pytest.mark.parametrize("n", [60, 140])
def test_every_other_sequence_out_of_range(n, call):
    """Sequences that run backwards stay idle and keep none of the others from their turn.  (The others all read
    the same tokens, so only their states are looked at.)"""
    H, V, T = 16, 128, 40
    d = ref.draw("gdn", "bf16", [T], H, H, V, seed=3, state_rows=n)
    S, y = torch.full((n, H, 128, V), 7.0, device="cuda"), torch.empty(d["v"].shape, device="cuda")
    _go(call, "gdn", H, V, d, d["S0"], None, S, None, [T * (i % 2) for i in range(n + 1)], T, y)
    Sr = torch.stack([ref.run("gdn", d, [T], d["S0"][i:i + 1])[1][0] for i in range(0, n, 2)])
    assert ref.slab_err(S[::2], Sr) <= TOL
    assert (S[1::2] == 7).all()


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("longest", [15, 16, 17, 27, 28, 29])
def test_lengths_where_the_form_changes(longest, kind):
    """The longest prompt decides between the recurrent and the chunked form; a larger max_len changes no result
    beyond the tolerance."""
    lens, H, V = [longest, 1, 0, longest - 1], 4, 80
    d = ref.draw(kind, "bf16", lens, H, H, V, seed=longest)
    yr, Sr = ref.run(kind, d, lens, d["S0"])
    for max_len in (longest, 64, 2 ** 31 - 1):
        S, y = torch.empty(4, H, 128, V, device="cuda"), torch.empty(d["v"].shape, device="cuda")
        _go("prefill", kind, H, V, d, d["S0"], None, S, None, d["offsets"].tolist(), max_len, y)
        assert ref.slab_err(S, Sr) <= TOL and ref.slab_err(y, yr) <= TOL
