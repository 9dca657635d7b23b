"""States in 8 bits: scales and codes as the definition in 64 bits has them, bit for bit, and what reads back."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import tree_reference as ref  # noqa: E402

K = 128
FORMATS = ["i8", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from rank_state_read_amd import binding
    binding.lib()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(n, H, V, fmt):
    kind = torch.int8 if fmt == "i8" else torch.float8_e4m3fn
    codes = torch.full((n, H, K, V), 77, dtype=torch.int8, device="cuda").view(kind)
    return codes, torch.full((n, H, K), 3.0, dtype=torch.bfloat16, device="cuda")


def roundtrip(S, fmt, rows, slots, n_slots, rows2=None):
    from rank_state_read_amd import sketchssm_cache_load, sketchssm_cache_store
    B, H, _, V = S.shape
    sh = ref.shape_of(B, H, V, "gdn", "bf16", 0)
    codes, scales = _cache(n_slots, H, V, fmt)
    sketchssm_cache_store(sh, S, _i32(rows), codes, scales, _i32(slots), fmt)
    out = torch.full_like(S, 9.0)
    sketchssm_cache_load(sh, codes, scales, _i32(slots), out, _i32(rows if rows2 is None else rows2), fmt)
    torch.cuda.synchronize()
    return codes, scales, out


def _states(B, H, V, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, H, K, V, generator=g) * torch.exp(spread * torch.randn(B, H, K, 1, generator=g))).cuda()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("V", [64, 80, 96, 112, 128])
@pytest.mark.parametrize("H", [1, 5, 32])
def test_widths(H, V, fmt):
    S = _states(4, H, V, V)
    codes, scales, out = roundtrip(S, fmt, [2, 0, 3], [5, 1, 4], 7, [1, 2, 0])
    for src, slot, dst in zip([2, 0, 3], [5, 1, 4], [1, 2, 0]):
        s, x = ref.quantised(S[src], fmt)
        assert torch.equal(scales[slot].double(), s)
        assert torch.equal(out[dst].double(), x)
    assert (out[3] == 9).all()
    for slot in (0, 2, 3, 6):
        assert (scales[slot] == 3).all() and (codes[slot].view(torch.int8) == 77).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_exponent(fmt):
    """Rows over all of fp32's exponents: the scale's lower end, values that read back as 0, the largest."""
    S = _states(1, 2, 64, 3, 0.3)
    e = torch.linspace(-150, 125, K)
    S = S.clamp(-4, 4) * torch.exp2(e.floor()).cuda()[None, None, :, None]
    _, scales, out = roundtrip(S, fmt, [0], [0], 1)
    s, x = ref.quantised(S[0], fmt)
    assert torch.equal(scales[0].double(), s) and torch.equal(out[0].double(), x.float().double())


@pytest.mark.parametrize("fmt", FORMATS)
def test_ties_and_borders(fmt):
    """Values halfway between two codes, one step of fp32 to either side of them, and maxima at the scales' borders."""
    V = 128
    S = torch.zeros(1, 1, K, V)
    g = torch.Generator().manual_seed(7)
    lim = 127.0 if fmt == "i8" else 448.0
    for r in range(K):
        s = float(torch.tensor(2.0 ** (r % 9 - 4) * (1 + (r % 128) / 128)).to(torch.bfloat16)) if fmt == "i8" else 2.0 ** (r % 9 - 4)
        if fmt == "i8":
            mid = (torch.randint(-127, 127, (V,), generator=g) + 0.5) * s
        else:
            c = torch.randint(0, 126, (V,), generator=g).to(torch.uint8)
            lo, hi = c.view(torch.float8_e4m3fn).float(), (c + 1).view(torch.float8_e4m3fn).float()
            mid = (lo + hi) / 2 * s * torch.where(torch.rand(V, generator=g) < 0.5, -1.0, 1.0)
        inf = torch.tensor(float("inf"))
        mid[1::3] = torch.nextafter(mid[1::3], inf)
        mid[2::3] = torch.nextafter(mid[2::3], -inf)
        top = torch.tensor(lim * s)
        mid[0] = [top, torch.nextafter(top, inf), torch.nextafter(top, -inf)][r % 3]
        S[0, 0, r] = mid
    S = S.cuda()
    _, scales, out = roundtrip(S, fmt, [0], [0], 1)
    s, x = ref.quantised(S[0], fmt)
    assert torch.equal(scales[0].double(), s) and torch.equal(out[0].double(), x)


@pytest.mark.parametrize("fmt", FORMATS)
def test_special_rows(fmt):
    """Zero rows; rows with an infinity or a NaN read back as NaN, their neighbours as they are."""
    S = _states(1, 1, 80, 5)
    S[0, 0, 3] = 0
    S[0, 0, 5, 7], S[0, 0, 6, 79], S[0, 0, 9, 0] = float("inf"), float("nan"), -float("inf")
    S[0, 0, 10], S[0, 0, 11] = -0.0, 1e-45
    _, scales, out = roundtrip(S, fmt, [0], [0], 1)
    bad = [5, 6, 9]
    good = [r for r in range(K) if r not in bad]
    assert out[0, 0, bad].isnan().all() and scales[0, 0, bad].isnan().all()
    s, x = ref.quantised(S[0, 0, good], fmt)
    assert torch.equal(out[0, 0, good].double(), x) and torch.equal(scales[0, 0, good].double(), s)
    assert (out[0, 0, [3, 10, 11]] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_all_codes(fmt):
    """A load of every code there is."""
    from rank_state_read_amd import sketchssm_cache_load
    kind = torch.int8 if fmt == "i8" else torch.float8_e4m3fn
    codes = torch.arange(K * 64).to(torch.uint8).view(1, 1, K, 64).cuda()
    scales = torch.exp2(torch.arange(K) % 40 - 20.0).view(1, 1, K).to(torch.bfloat16).cuda()
    S = torch.zeros(1, 1, K, 64, device="cuda")
    sketchssm_cache_load(ref.shape_of(1, 1, 64, "gdn", "bf16", 0), codes.view(kind), scales, None, S, None, fmt)
    x = codes.view(kind).float() * scales.float()[..., None]
    assert torch.equal(S.isnan(), x.isnan()) and torch.equal(S.nan_to_num(), x.nan_to_num())


def test_lists():
    """Shared and empty slots, pairs out of range, rows and slots in order where a list is left out."""
    from rank_state_read_amd import sketchssm_cache_load, sketchssm_cache_store
    S = _states(4, 3, 64)
    sh = ref.shape_of(4, 3, 64, "gdn", "bf16", 0)
    codes, scales = _cache(3, 3, 64, "i8")
    sketchssm_cache_store(sh, S, None, codes, scales, None, "i8")  # rows 0 .. 2
    x = [ref.quantised(S[i], "i8")[1] for i in range(3)]
    out = torch.full_like(S, 9.0)
    sketchssm_cache_load(sh, codes, scales, _i32([2, 2, -1, 3]), out, _i32([0, 3, 1, 2]), "i8")
    assert torch.equal(out[0].double(), x[2]) and torch.equal(out[3].double(), x[2])
    assert (out[1] == 0).all() and (out[2] == 9).all()
    out.fill_(9.0)
    sketchssm_cache_load(sh, codes, scales, _i32([1, 1, -(1 << 31), 0]), out, _i32([-1, 4, 1 << 30, 2]), "i8")
    assert torch.equal(out[2].double(), x[0]) and (out[[0, 1, 3]] == 9).all()
    out.fill_(9.0)
    sketchssm_cache_load(sh, codes, scales, None, out, None, "i8")
    assert all(torch.equal(out[i].double(), x[i]) for i in range(3)) and (out[3] == 9).all()
    before = codes.clone(), scales.clone()
    sketchssm_cache_store(sh, S, _i32([4, -1, 0, 1]), codes, scales, _i32([0, 1, 3, -1]), "i8")
    assert torch.equal(codes, before[0]) and torch.equal(scales, before[1])
    sketchssm_cache_load(sh, codes, scales, _i32([]), out, _i32([]), "i8")
