"""The operators around the decode path, as they are measured: prefill of ragged prompts (the chunked form
of the state update), the recurrent form for a few tokens of listed state rows, and the gated norm behind a
layer's output.

``own`` selects who computes a pass: elementary torch operations in 32 bits, or the library's entry points.
Per state head with key dim K and value dim V, S a K x V state:

  prefill, rmw_seq   S <- M S + beta k v^T,  y = S^T q  for every token of a sequence in turn, with
                     Mamba-2 M = a I (beta = 1), GDN M = a (I - beta k k^T), KDA M = (I - beta k k^T) diag(a);
                     a sequence starts from a cached state or from zero, and its last state is written
  gated_norm         x = y + D skip;  then norm(x silu(z)) w, norm(x) w silu(z) or norm(x) w sigmoid(z),
                     norm over groups of consecutive heads, x / sqrt(mean(x^2) + eps)
"""
import math
import random

import torch

own = False

K = 128
KINDS = ("mamba2", "gdn", "kda")
GATES = ("none", "silu_first", "silu", "sigmoid")
EPS = 1e-5


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _seq(name, op, kind, H, Hk, V, dtype, n, tokens, start="zeros", lens=0):
    c = {"op": op, "kind": kind, "H": H, "Hk": Hk, "V": V, "dtype": dtype, "n": n, "tokens": tokens,
         "start": start, "lens": lens}
    return dict(c, name=name) if name else c


def _norm(name, H, V, dtype, rows, heads, gate, skip):
    c = {"op": "gated_norm", "H": H, "V": V, "dtype": dtype, "tokens": rows, "heads": heads, "gate": gate, "skip": skip}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one long prompt through a Gated DeltaNet layer: few heads, a long serial axis
        _seq("prefill gdn long", "prefill", "gdn", 32, 32, 128, "bf16", 1, 16384),
        # a prefill batch of several prompts of different lengths, keys shared by two heads
        _seq("prefill gdn batch", "prefill", "gdn", 32, 16, 128, "bf16", 9, 16001, "mixed", 3),
        # one prompt through the Nano-shaped Mamba-2 layer, keys and queries per group
        _seq("prefill mamba2 prompt", "prefill", "mamba2", 128, 8, 80, "bf16", 1, 4096),
        # the same layer, a batch of prompts that continue cached prefixes
        _seq("prefill mamba2 batch", "prefill", "mamba2", 128, 8, 80, "bf16", 7, 16003, "cache", 5),
        # a KDA layer's prefill batch: one decay per key channel
        _seq("prefill kda batch", "prefill", "kda", 32, 32, 128, "bf16", 4, 8190, "mixed", 7),
        # a short prompt on its own, where latency counts
        _seq("prefill gdn short", "prefill", "gdn", 32, 32, 128, "bf16", 1, 77),
        # float32 activations at another width
        _seq("prefill gdn float32", "prefill", "gdn", 32, 32, 96, "f32", 3, 3001, "zeros", 9),
        # one token of one sequence: the smallest call
        _seq("rmw_seq gdn one token", "rmw_seq", "gdn", 32, 32, 128, "bf16", 1, 1, "cache"),
        # a serving batch of the Nano-shaped layer with a few drafted tokens for some rows
        _seq("rmw_seq mamba2 batch", "rmw_seq", "mamba2", 128, 8, 80, "bf16", 192, 500, "cache", 11),
        # drafted tokens of a KDA layer
        _seq("rmw_seq kda drafts", "rmw_seq", "kda", 32, 32, 128, "bf16", 96, 480, "cache", 13),
        # a decode step's output of the Nano-shaped layer: gate, then norm over a group of 16 heads
        _norm("gated_norm decode", 128, 80, "bf16", 256, 16, "silu_first", True),
        # a prefill's output of a Gated DeltaNet layer: a norm per head, then the gate
        _norm("gated_norm prefill", 32, 128, "bf16", 16001, 1, "silu", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "rmw_seq", "gated_norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    V = rng.choice([64, 80, 96, 112, 128])
    if op == "gated_norm":
        H = rng.choice([8, 12, 32, 40, 128])
        heads = rng.choice([h for h in (1, 2, 4, 16, H) if H % h == 0])
        return _norm(None, H, V, dtype, _log(rng, 1, 16001 * 32 // H), heads, rng.choice(GATES), rng.random() < 0.4)
    kind = rng.choice(KINDS)
    H = rng.choice([8, 16, 32, 40, 64] + ([128] if kind == "mamba2" else []))
    Hk = H // rng.choice([1, 1, 2, 8] if kind != "mamba2" else [1, 8, 8])
    lens, start = rng.randrange(1 << 16), rng.choice(["zeros", "cache", "mixed"])
    if op == "rmw_seq":
        n = _log(rng, 1, 256)
        tokens = min(n * rng.randint(1, 8), 500 * 128 // H)
        return _seq(None, op, kind, H, Hk, V, dtype, min(n, tokens), tokens, start, lens)
    tokens = _log(rng, 17, (8190 if kind == "kda" else 16001) * 32 // max(H, 32))
    return _seq(None, op, kind, H, Hk, V, dtype, min(_log(rng, 1, 24), tokens), tokens, start, lens)


def _lengths(case):
    """A split of the tokens into n lengths of at least one token, uneven where there are several."""
    n, rng = case["n"], random.Random(case["lens"])
    w = [0.3 + rng.expovariate(1.0) for _ in range(n)]
    got = [1 + int((case["tokens"] - n) * x / sum(w)) for x in w]
    got[rng.randrange(n)] += case["tokens"] - sum(got)
    return got


# ---------------------------------------------------------------------------
# inputs: the distributions of the layer's activations
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    T, H, V = case["tokens"], case["H"], case["V"]
    if case["op"] == "gated_norm":
        y, z, x = rn(T, H, V), rn(T, H, V).to(dt), rn(T, H, V).to(dt)
        return {"case": case, "y": y, "z": None if case["gate"] == "none" else z, "x": x if case["skip"] else None,
                "D": 1 + 0.2 * rn(H) if case["skip"] else None, "w": 1 + 0.1 * rn(H, V),
                "out": torch.empty((T, H, V), dtype=dt, device="cuda")}
    Hk, n, kda = case["Hk"], case["n"], case["kind"] == "kda"
    lens = _lengths(case)
    k = rn(T, Hk, K)
    k = (k / k.norm(dim=-1, keepdim=True)).to(dt)
    a = torch.exp(-0.1 * torch.nn.functional.softplus(rn(T, H, K) if kda else rn(T, H)))
    order = list(range(n))
    random.Random(seed).shuffle(order)
    zero = {"zeros": lambda i: True, "cache": lambda i: False, "mixed": lambda i: i % 2 == 0}[case["start"]]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"case": case, "k": k, "q": rn(T, Hk, K).to(dt), "v": rn(T, H, V).to(dt), "a": a,
            "beta": None if case["kind"] == "mamba2" else torch.sigmoid(rn(T, H)),
            "S0": None if case["start"] == "zeros" else 0.02 * rn(n, H, K, V), "S": torch.zeros(n, H, K, V, device="cuda"),
            "rows": i32(order), "rows0": i32([-1 if zero(i) else r for i, r in enumerate(order)]),
            "offsets": i32([sum(lens[:i]) for i in range(n + 1)]), "max_len": max(lens),
            "y": torch.empty(T, H, V, device="cuda")}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own_norm(state) if op == "gated_norm" else _own_seq(state)
    return _plain_norm(state) if op == "gated_norm" else _plain_seq(state)


_shapes = {}


def _shape(c, n):
    """The layer's descriptor, which a program makes once."""
    from rank_state_read_amd import make_shape
    key = (n, c["H"], c["V"], c.get("kind"), c["dtype"], c.get("Hk"))
    if key not in _shapes:
        _shapes[key] = make_shape(n, c["H"], K, c["V"], 16, 1, 79, 49, c.get("kind", "gdn"), c["dtype"], c.get("Hk", 0))
    return _shapes[key]


def _own_seq(s):
    from rank_state_read_amd import sketchssm_prefill, sketchssm_rmw_seq
    c = s["case"]
    call = sketchssm_prefill if c["op"] == "prefill" else sketchssm_rmw_seq
    call(_shape(c, c["n"]), s["S0"], None if s["S0"] is None else s["rows0"], s["S"], s["rows"], s["offsets"], s["max_len"],
         s["q"], s["k"], s["v"], s["a"], s["beta"], s["y"])
    return {"y": s["y"], "S": s["S"]}


def _own_norm(s):
    from rank_state_read_amd import sketchssm_gated_norm
    c = s["case"]
    sketchssm_gated_norm(_shape(c, 1), s["y"], s["x"], s["D"], s["z"], s["w"], c["heads"], c["gate"], EPS, s["out"])
    return s["out"]


def _padded(s, C):
    """The ragged arrays in 32 bits as [n, H, L, ...], L a multiple of C: tokens past a sequence's end decay by 1
    and write nothing."""
    c, off = s["case"], s["offsets"].long()
    L = -(-s["max_len"] // C) * C
    at = off[:-1, None] + torch.arange(L, device="cuda")
    live = at < off[1:, None]
    at = torch.where(live, at, torch.zeros_like(at))
    share = c["H"] // c["Hk"]

    def pad(x, fill, rep=1):
        x = x.float()[at]
        x = torch.where(live.view(live.shape + (1,) * (x.dim() - 2)), x, torch.full_like(x, fill))
        return x.transpose(1, 2).repeat_interleave(rep, dim=1)

    q, k, v, a = pad(s["q"], 0, share), pad(s["k"], 0, share), pad(s["v"], 0), pad(s["a"], 1)
    beta = torch.ones_like(v[..., 0]) if s["beta"] is None else pad(s["beta"], 0)
    return q, k, v, a, beta, at, live


def _states(s):
    """The sequences' first states, [n, H, K, V]."""
    if s["S0"] is None:
        return torch.zeros_like(s["S"])
    r = s["rows0"].long()
    return torch.where((r >= 0).view(-1, 1, 1, 1), s["S0"][r.clamp(min=0)], torch.zeros_like(s["S"]))


def _inverse(N, C):
    """(I + N)^-1 of strictly lower triangular C x C matrices: (I - N)(I + N^2)(I + N^4)..."""
    inv, p = torch.eye(C, device="cuda") - N, N
    for _ in range(C.bit_length() - 2):
        p = p @ p
        inv = inv + inv @ p
    return inv


def _plain_seq(s):
    """The chunked form: within a chunk the updates u solve a triangular system, between chunks the state moves on.

    With G_i the decays' product up to token i and G_ij that after j up to i: A_ij = k_i G_ij k_j (j < i),
    P_ij = q_i G_ij k_j (j <= i), T = (I + diag(beta) A)^-1 diag(beta) (I for Mamba-2),
    u = T (v - (G k) S), y = (G q) S + P u, S <- G_C S + sum_j G_Cj k_j u_j."""
    kind = s["case"]["kind"]
    C = 16 if kind == "kda" else 64
    q, k, v, a, beta, at, live = _padded(s, C)
    n, H, L, V = v.shape
    cut = lambda x: x.reshape((n, H, L // C, C) + x.shape[3:])  # noqa: E731
    q, k, v, a, beta = cut(q), cut(k), cut(v), cut(a), cut(beta)
    i = torch.arange(C, device="cuda")
    after, upto = i[:, None] > i, i[:, None] >= i
    S, y = _states(s), torch.empty_like(v)
    if kind != "kda":  # the decays' products leave the sums over channels
        G = torch.where(after, a[..., :, None], 1.0).cumprod(-2) * upto
        kk, P = k @ k.transpose(-1, -2).contiguous() * (G * after), q @ k.transpose(-1, -2).contiguous() * G
        gam = a.cumprod(-1)[..., None]
        gk, gq, kend = gam * k, gam * q, (k * G[..., -1, :, None]).transpose(-1, -2).contiguous()
        gend = gam[..., -1, :, None]
        if kind == "gdn":
            T = _inverse(beta[..., None] * kk, C) * beta[..., None, :]
            v, gk = T @ v, T @ gk
    for m in range(L // C):
        if kind == "kda":
            am, km, qm = a[:, :, m], k[:, :, m], q[:, :, m]
            G = torch.where(after[..., None], am[..., :, None, :], 1.0).cumprod(-3) * upto[..., None]
            kG = km[..., None, :, :] * G
            kk, Pm = (km[..., :, None, :] * kG).sum(-1) * after, (qm[..., :, None, :] * kG).sum(-1)
            T = _inverse(beta[:, :, m, :, None] * kk, C) * beta[:, :, m, None, :]
            gam = am.cumprod(-2)
            u = T @ (v[:, :, m] - (gam * km) @ S)
            y[:, :, m] = (gam * qm) @ S + Pm @ u
            S = gam[..., -1, :, None] * S + kG[..., -1, :, :].transpose(-1, -2).contiguous() @ u
        else:
            u = v[:, :, m] if kind == "mamba2" else v[:, :, m] - gk[:, :, m] @ S
            y[:, :, m] = gq[:, :, m] @ S + P[:, :, m] @ u
            S = gend[:, :, m] * S + kend[:, :, m] @ u
    s["y"][at[live]] = y.reshape(n, H, L, V).transpose(1, 2)[live]
    s["S"][s["rows"].long()] = S
    return {"y": s["y"], "S": s["S"]}


def _plain_norm(s):
    c = s["case"]
    x = s["y"]
    if s["x"] is not None:
        x = x + s["D"][:, None] * s["x"].float()
    z = None if s["z"] is None else s["z"].float()
    if c["gate"] == "silu_first":
        x = x * z / (1 + torch.exp(-z))
    shape = x.shape
    x = x.reshape(shape[0], c["H"] // c["heads"], -1)
    x = (x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)).reshape(shape) * s["w"]
    if c["gate"] == "silu":
        x = x * z / (1 + torch.exp(-z))
    if c["gate"] == "sigmoid":
        x = x / (1 + torch.exp(-z))
    return x.to(s["out"].dtype)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda x: x.double()  # noqa: E731
    if case["op"] == "gated_norm":
        x, z = f64(s["y"]), None if s["z"] is None else f64(s["z"])
        if case["skip"]:
            x = x + f64(s["D"]).view(1, -1, 1) * f64(s["x"])
        sig = None if z is None else torch.special.expit(z)
        if case["gate"] == "silu_first":
            x = x * (z * sig)
        rows = x.view(x.shape[0], -1, case["heads"] * case["V"])
        x = (rows * torch.rsqrt(rows.square().mean(2, True) + EPS)).view_as(x) * f64(s["w"])
        return x * (z * sig) if case["gate"] == "silu" else x * sig if case["gate"] == "sigmoid" else x
    # token by token, all sequences side by side; a sequence that has ended stands still
    off, rows, rows0 = s["offsets"].tolist(), s["rows"].tolist(), s["rows0"].tolist()
    n, H, share, T = case["n"], case["H"], case["H"] // case["Hk"], case["tokens"]
    lens = [off[i + 1] - off[i] for i in range(n)]
    by_len = sorted(range(n), key=lambda i: -lens[i])
    S = torch.stack([torch.zeros_like(s["S"][0]) if rows0[i] < 0 else s["S0"][rows0[i]] for i in by_len]).double()
    first = torch.tensor([off[i] for i in by_len], device="cuda")
    y = torch.empty(T, H, case["V"], dtype=torch.float64, device="cuda")
    for t in range(max(lens)):
        m = sum(length > t for length in lens)
        at = first[:m] + t
        k = f64(s["k"][at]).repeat_interleave(share, 1)[..., None]
        q = f64(s["q"][at]).repeat_interleave(share, 1)[..., None]
        v, a = f64(s["v"][at])[:, :, None], f64(s["a"][at])
        live = S[:m]
        live *= a[..., None] if case["kind"] == "kda" else a[..., None, None]
        if case["kind"] != "mamba2":
            v = f64(s["beta"][at])[..., None, None] * (v - (k * live).sum(2, True))
        live += k * v
        y[at] = (q * live).sum(2)
    out = torch.empty_like(S)
    out[[rows[i] for i in by_len]] = S
    return {"y": y, "S": out}


def work(case):
    e, T, H, V = 2 if case["dtype"] == "bf16" else 4, case["tokens"], case["H"], case["V"]
    if case["op"] == "gated_norm":
        n = T * H * V
        moved = 4 * n + e * n + (e * n if case["gate"] != "none" else 0) + (e * n if case["skip"] else 0) + 4 * H * V
        return {"bytes": moved, "flops": 12 * n}
    kda, delta, n = case["kind"] == "kda", case["kind"] != "mamba2", case["n"]
    cached = {"zeros": 0, "cache": n, "mixed": n // 2}[case["start"]]
    per_token = e * (2 * case["Hk"] * K + H * V) + 4 * H * ((K if kda else 1) + (1 if delta else 0) + V)
    return {"bytes": T * per_token + 4 * (n + cached) * H * K * V, "flops": T * H * K * V * (6 if delta else 4)}
