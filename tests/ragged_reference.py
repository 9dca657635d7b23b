"""Plain 64-bit references of the ragged calls and the gated norm, token by token from the definitions, and
the inputs their tests draw.  They share no code with the library."""
import torch

K = 128


def draw(kind, qkv, lens, H, Hk, V, seed=0, lead=0, tail=0, device="cuda", state_rows=None):
    """Inputs of sequences of the given lengths, behind `lead` and before `tail` tokens that belong to none
    (filled with NaN: nothing may read them)."""
    g = torch.Generator().manual_seed(seed)
    n, T = len(lens), sum(lens)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = torch.bfloat16 if qkv == "bf16" else torch.float32
    k = rn(T, Hk, K)
    d = {"q": rn(T, Hk, K).to(dt), "k": (k / k.norm(dim=-1, keepdim=True)).to(dt), "v": rn(T, H, V).to(dt),
         "a": torch.exp(-0.1 * torch.nn.functional.softplus(rn(T, H, K) if kind == "kda" else rn(T, H))),
         "beta": None if kind == "mamba2" else torch.sigmoid(rn(T, H))}
    pad = lambda x, m: torch.full((m,) + tuple(x.shape[1:]), float("nan"), dtype=x.dtype)  # noqa: E731
    d = {key: None if x is None else torch.cat([pad(x, lead), x, pad(x, tail)]).to(device) for key, x in d.items()}
    off = [lead]
    for length in lens:
        off.append(off[-1] + length)
    d["offsets"] = torch.tensor(off, dtype=torch.int32, device=device)
    d["S0"] = (0.05 * rn(state_rows or n, H, K, V)).to(device)
    return d


def run(kind, d, lens, S0, upto=None):
    """(y, last states) of every sequence in 64 bits; S0 [n, H, K, V] its first states.  y of other tokens is 0."""
    f = lambda x: x.double()  # noqa: E731
    T, H, V = d["v"].shape
    share = H // d["q"].shape[1]
    y = torch.zeros(T, H, V, dtype=torch.float64, device=d["v"].device)
    S = f(S0).clone()
    off = d["offsets"].tolist()
    for i, length in enumerate(lens):
        s = S[i]
        for t in range(off[i], off[i] + length):
            k = f(d["k"][t]).repeat_interleave(share, 0)[:, :, None]
            q = f(d["q"][t]).repeat_interleave(share, 0)[:, :, None]
            a = f(d["a"][t])
            s = (a[:, :, None] if kind == "kda" else a[:, None, None]) * s
            u = f(d["v"][t])[:, None, :]
            if kind != "mamba2":
                u = f(d["beta"][t])[:, None, None] * (u - (k * s).sum(1, keepdim=True))
            s = s + k * u
            y[t] = (q * s).sum(1)
        S[i] = s
    return y, S


def norm(y, skip, D, z, w, heads, gate, eps):
    """The gated norm's formula in 64 bits."""
    x = y.double()
    n, H, V = x.shape
    if skip is not None:
        x = x + D.double()[None, :, None] * skip.double()
    s = None if z is None else 1 / (1 + torch.exp(-z.double()))
    if gate == "silu_first":
        x = x * (z.double() * s)
    g = x.reshape(n, H // heads, heads * V)
    g = g / torch.sqrt((g * g).mean(-1, keepdim=True) + eps)
    x = g.reshape(n, H, V) * w.double()
    return x * z.double() * s if gate == "silu" else x * s if gate == "sigmoid" else x


def slab_err(got, ref, floor=1e-30):
    """Largest error over the slabs (all but the last dims of one head's vector or state), relative to the slab's max."""
    got, ref = got.double(), ref.double()
    dims = tuple(range(2, ref.dim()))
    if not ref.numel():
        return 0.0
    den = ref.abs().amax(dims).clamp(min=floor)
    return float(((got - ref).abs().amax(dims) / den).max())
