"""A plain 64-bit reference of the tree calls and of the 8-bit cache, from their definitions, and the inputs their
tests draw.  It shares no code with the library."""
import random

import torch

K, W = 128, 16


def shape_of(B, H, V, kind, qkv, Hk, G=2):
    from rank_state_read_amd import make_shape
    return make_shape(B, H, K, V, W, G, 79, 64, kind, qkv, Hk)


def trees(sizes, seed=0, how="tree"):
    """Parents of each sequence's nodes: random trees, chains, stars (every node a first token) or combs (two chains)."""
    rng = random.Random(seed)
    pick = {"tree": lambda j: rng.randint(-1, j - 1), "chain": lambda j: j - 1, "star": lambda j: -1,
            "comb": lambda j: max(j - 2, -1)}[how]
    return [[pick(j) for j in range(n)] for n in sizes]


def path(parents, node):
    """Nodes from the root to `node`."""
    out = []
    while node >= 0:
        out.insert(0, node)
        node = parents[node]
    return out


def draw(kind, qkv, sizes, B, H, Hk, V, ranks, held, seed=0, how="tree", lead=0, tail=0, device="cuda"):
    """Inputs of trees of the given sizes on state rows `rows`, behind `lead` and before `tail` nodes that belong to
    none; those and every window slot that holds no token are NaN (nothing may read them).  held: tokens per row."""
    g = torch.Generator().manual_seed(seed)
    n, T = len(sizes), sum(sizes)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = torch.bfloat16 if qkv == "bf16" else torch.float32
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    decay = lambda *s: torch.exp(-0.1 * torch.nn.functional.softplus(rn(*s)))  # noqa: E731
    kda, delta = kind == "kda", kind != "mamba2"
    nan = float("nan")
    pad = lambda x, m: torch.full((m,) + tuple(x.shape[1:]), nan, dtype=x.dtype)  # noqa: E731
    d = {"q": rn(T, Hk, K).to(dt), "k": unit(rn(T, Hk, K)).to(dt), "v": rn(T, H, V).to(dt),
         "a": decay(T, H, K) if kda else decay(T, H), "beta": torch.sigmoid(rn(T, H)) if delta else None}
    d = {key: None if x is None else torch.cat([pad(x, lead), x, pad(x, tail)]) for key, x in d.items()}
    d.update({"kbuf": unit(rn(W, Hk, B, K)).to(dt), "vbuf": rn(W, H, B, V).to(dt),
              "abuf": decay(W, H, B, K) if kda else decay(W, H, B),
              "bbuf": torch.sigmoid(rn(W, H, B)) if delta else None})
    for b in range(B):
        for key in ("kbuf", "vbuf", "abuf", "bbuf"):
            if d[key] is not None:
                d[key][max(0, min(W, held[b])):, :, b] = nan
    par = trees(sizes, seed, how)
    flat = [p for t in par for p in t]
    off = [lead]
    for size in sizes:
        off.append(off[-1] + size)
    groups = [h * 2 // H for h in range(H)]
    pairs = sorted({(gr, r) for gr, r in zip(groups, ranks) if r})
    fr, at = {}, 0
    for p in pairs:
        fr[p], at = at, at + p[1]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    d.update({"S": 0.05 * rn(B, H, K, V), "Z": 0.3 * rn(B * V * sum(ranks)) if sum(ranks) else None,
              "frames": rn(at, K) / K ** 0.5 if at else None, "pos": i32(held), "offsets": i32(off),
              "parents": i32([-7] * lead + flat + [-7] * tail)})
    d = {key: x.to(device) if isinstance(x, torch.Tensor) else x for key, x in d.items()}
    d.update({"par": par, "groups": groups, "ranks": list(ranks), "frame": fr, "kind": kind, "sizes": list(sizes)})
    return d


def first_states(d, rows):
    """What stands before each sequence's window, [n, H, K, V]: the state, or F^T Z of a sketch head (a query reads it
    as Z^T F q)."""
    S = d["S"][rows].double()
    B, H, _, V = d["S"].shape
    z = 0
    for h, (g, r) in enumerate(zip(d["groups"], d["ranks"])):
        if r:
            F = d["frames"][d["frame"][g, r]:d["frame"][g, r] + r].double()
            Z = d["Z"][z * B * V:(z + r) * B * V].view(B, r, V)[rows].double()
            for i in range(len(rows)):
                S[i, h] = F.t().contiguous() @ Z[i]
            z += r
    return S


def step(kind, S, k, v, a, beta, share):
    """S [H, K, V] after one token."""
    k = k.double().repeat_interleave(share, 0)[:, :, None]
    S = (a.double()[:, :, None] if kind == "kda" else a.double()[:, None, None]) * S
    u = v.double()[:, None, :]
    if kind != "mamba2":
        u = beta.double()[:, None, None] * (u - (k * S).sum(1, keepdim=True))
    return S + k * u


def read(d, rows, held=None):
    """(y of every node in 64 bits, its largest possible sum of magnitudes is not tracked); other nodes' y is 0."""
    T, H, V = d["v"].shape
    share, off = H // d["q"].shape[1], d["offsets"].tolist()
    y = torch.zeros(T, H, V, dtype=torch.float64, device=d["v"].device)
    pos = d["pos"].tolist() if held is None else held
    at = lambda x, *i: None if x is None else x[i]  # noqa: E731
    for i, (row, S0) in enumerate(zip(rows, first_states(d, rows))):
        root = S0
        for j in range(pos[row]):
            root = step(d["kind"], root, d["kbuf"][j, :, row], d["vbuf"][j, :, row], d["abuf"][j, :, row],
                        None if d["bbuf"] is None else d["bbuf"][j, :, row], share)
        states = {-1: root}
        for j, p in enumerate(d["par"][i]):
            t = off[i] + j
            states[j] = step(d["kind"], states[p], d["k"][t], d["v"][t], d["a"][t], at(d["beta"], t), share)
            y[t] = (d["q"][t].double().repeat_interleave(share, 0)[:, :, None] * states[j]).sum(1)
    return y


def quantised(x, fmt):
    """(scales, values read back) of state rows in 64 bits; scales as the definition has them: the least number of the
    format's kind that is not below max|x| / 127 (or 448)."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    lim = 127.0 if fmt == "i8" else 448.0
    least = top.clamp(min=lim * 2.0 ** -100)
    m, e = torch.frexp(least / torch.full_like(top, lim))  # m in [1/2, 1): 8 significant bits, or 1
    two = lambda e: torch.exp2(e.double())  # noqa: E731
    s = torch.ceil(m * 256) / 256 * two(e) if fmt == "i8" else two(e - (m == 0.5).int())
    t = x / s
    if fmt == "i8":
        c = torch.round(t)
    else:
        q = two((torch.frexp(t)[1] - 4).clamp(min=-9))
        c = torch.round(t / q) * q
    return s[..., 0], c * s
