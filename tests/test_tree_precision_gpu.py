"""How near the definition tree reads come: as near as fp32 arithmetic, which the 1e-4 of a slab that the other tests
ask for does not show.

Where a sum has one term that is not zero, y is that term bit for bit: a float32 operand that enters a product in bf16
parts must enter with all its 24 bits, whichever operand it is (the state, the frame, the sketch, or the products P by way
of a decay or beta).  The parts' partial sums, 8 and 16 leading bits of the operand, are fp32 numbers, so nothing rounds.

For random operands errors are taken as 2-norms of a call's y relative to the exact one; u = 2^-24, and a rounding to
nearest is off by u / sqrt(3) of the value in the mean square, independent ones adding as squares.  Decays and beta are
in (0, 1] and keys have length 1, so no error grows on the way.  A path has up to 80 tokens (16 held, 64 nodes):
  the carried query, or the decays   two roundings a token at most (KDA: a correction and a decay; GDN: a correction, and
                                     the decays' product beside it; Mamba-2: one), sqrt(2 80 / 3) = 7.3 u
  x S, or F x, or q k                sums of 128 products whose partial sums grow evenly, sqrt(128 / 2 / 3) = 4.6 u
  Z^T (F x)                          64 products more, sqrt(64 / 2 / 3) = 3.3 u
  P v                                80 rows, sqrt(80 / 2 / 3) = 3.7 u
Together, as if all fell on one value: sqrt(7.3^2 + 4.6^2 + 3.3^2 + 3.7^2) = 10 u.  The bar is twice that, 20 u.  An
operand cut to two bf16 parts loses up to 2^-16 of its leading bit, 0.4 2^-16 = 100 u of its own part of y in the mean
square; behind long paths, whose values make up most of y, that is less than the bar, and the cases of one term show it."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import tree_reference as ref  # noqa: E402

K, W = ref.K, ref.W
U = 2.0 ** -24
BAR = 20 * U
KINDS = ["mamba2", "gdn", "kda"]
RANKS = {"dense": [0, 0, 0, 0], "sketch": [6, 17, 64, 1]}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rank_state_read_amd import binding
    binding.lib()


def _read(d, rows, H, Hk, V, qkv):
    from rank_state_read_amd import Plan, sketchssm_tree_read
    B = d["S"].shape[0]
    plan = Plan(ref.shape_of(B, H, V, d["kind"], qkv, Hk), d["ranks"], d["groups"])
    y = torch.full(d["v"].shape, 9.0, device="cuda")
    sketchssm_tree_read(plan, d["S"], d["Z"], d["frames"], d["kbuf"], d["vbuf"], d["abuf"], d["bbuf"], d["pos"],
                        torch.tensor(rows, dtype=torch.int32, device="cuda"), d["offsets"], max(d["sizes"]), d["parents"],
                        d["q"], d["k"], d["v"], d["a"], d["beta"], y)
    torch.cuda.synchronize()
    return y


# -- random operands --------------------------------------------------------------------------------------------
@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("ranks", ["dense", "sketch"])
@pytest.mark.parametrize("V", [64, 80, 128])
@pytest.mark.parametrize("sizes,how", [([13, 5], "tree"), ([30, 17], "tree"), ([64, 47, 7], "tree"), ([64, 33], "chain")],
                         ids=str)
def test_random_operands(sizes, how, V, ranks, qkv, kind):
    H, Hk, B = 4, 2, len(sizes) + 1
    d = ref.draw(kind, qkv, sizes, B, H, Hk, V, RANKS[ranks], [16, 9, 0, 5][:B], V, how)
    rows = list(range(1, B)) if how == "tree" else list(range(B - 1))
    y, want = _read(d, rows, H, Hk, V, qkv), ref.read(d, rows)
    e = float((y.double() - want).norm() / want.norm()) / U
    print(f"  {kind} {qkv} V={V} {ranks} {how} {sizes}: {e:.2f} u", flush=True)
    assert e <= BAR / U


# -- one term ---------------------------------------------------------------------------------------------------
def _quiet(kind, qkv, sizes, V, ranks, held, B=3, H=4, Hk=4):
    """Tokens that change nothing: keys and values 0, decays 1."""
    d = ref.draw(kind, qkv, sizes, B, H, Hk, V, ranks, [held] * B, 11, "chain")
    for key in ("k", "v", "q", "kbuf", "vbuf"):
        d[key].zero_()
    d["a"].fill_(1), d["abuf"].fill_(1)
    return d


SIZES = [[11], [29], [64]]


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("V", [80, 128])
def test_the_state(V, sizes, qkv, kind):
    """q picks one key: y is that row of the state."""
    d = _quiet(kind, qkv, sizes, V, RANKS["dense"], 7)
    at = [(37 * n + 5) % K for n in range(sizes[0])]
    for n, c in enumerate(at):
        d["q"][n, :, c] = 1
    y = _read(d, [2], 4, 4, V, qkv)
    for n, c in enumerate(at):
        assert torch.equal(y[n], d["S"][2, :, c]), n


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("V", [80, 128])
@pytest.mark.parametrize("which", ["frame", "sketch"])
def test_the_sketch(which, V, sizes, qkv, kind):
    """frame: the sketch has a 1 in row i, column i, so that y's column i is F[i, key]; sketch: F picks key i for row i,
    so that y is the sketch's row of the queried key."""
    ranks, B, row = RANKS["sketch"], 3, 1
    d = _quiet(kind, qkv, sizes, V, ranks, 7)
    at = [(37 * n + 5) % K if which == "frame" else (5 * n) % 64 for n in range(sizes[0])]
    for n, c in enumerate(at):
        d["q"][n, :, c] = 1
    if which == "frame":
        d["Z"].zero_()
    else:
        d["frames"].zero_()
    want, z0 = torch.zeros(sizes[0], 4, V, device="cuda"), 0
    for h, (g, r) in enumerate(zip(d["groups"], ranks)):
        f0 = d["frame"][g, r]
        Z = d["Z"][z0 * B * V:(z0 + r) * B * V].view(B, r, V)[row]
        for i in range(r):
            if which == "frame":
                Z[i, i] = 1
            else:
                d["frames"][f0 + i, i] = 1
        for n, c in enumerate(at):
            if which == "frame":
                want[n, h, :r] = d["frames"][f0:f0 + r, c]
            elif c < r:
                want[n, h] = Z[c]
        z0 += r
    assert torch.equal(_read(d, [row], 4, 4, V, qkv), want)


@pytest.mark.timeout(300)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("qkv", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("V", [80, 128])
@pytest.mark.parametrize("token", ["held", "root"])
def test_the_path(token, V, sizes, qkv, kind):
    """One token of a chain, a held-back one or the first node, has a value, 1 in column 3; one later node has a decay
    with 24 bits.  From that node on y's column is the decay; before it, 1.  For the delta rule beta has 24 bits instead,
    and y's column is beta from the token on."""
    d = _quiet(kind, qkv, sizes, V, RANKS["dense"], 7)
    d["S"].zero_()
    d["q"][:, :, 9] = 1
    key, value, beta = (("kbuf", "vbuf", "bbuf") if token == "held" else ("k", "v", "beta"))
    at = (4, slice(None), 2) if token == "held" else (0, slice(None))
    d[key][at + (9,)] = 1
    d[value][at + (3,)] = 1
    g = torch.Generator().manual_seed(5)
    x = (0.5 + 0.5 * torch.rand(4, generator=g)).cuda()  # per head
    want = torch.zeros(sizes[0], 4, V, device="cuda")
    if kind == "mamba2":
        d["a"][5, :] = x
        want[:5, :, 3] = 1
        want[5:, :, 3] = x
    else:
        d[beta][at] = x
        want[:, :, 3] = x
    assert torch.equal(_read(d, [2], 4, 4, V, qkv), want)
