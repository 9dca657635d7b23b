"""More operators around the decode path, as they are measured: trees of drafted tokens read over a row's cache
(its sketch or state, and its window), the accepted path kept in the window, and states cached in 8 bits.

``own`` selects who computes a pass: elementary torch operations in 32 bits (64 where a quantised value is next to a
border), or the library's entry points.  Per state head with key dim K and value dim V, S the K x V state of the last
flush, held-back window tokens 1..p behind it and a node's ancestors behind those:

  tree_read    a node's query is carried back through its ancestors, itself first, and the window, x <- M^T x, every
               token adding beta (k . x) v on the way; what arrives reads the state, S^T x (a dense head), or the
               sketch, Z^T F x.  M is a I (Mamba-2), a (I - beta k k^T) (GDN), (I - beta k k^T) diag(a) (KDA)
  tree_accept  the tokens on the path to a row's accepted node go to its next window slots
  cache_fork   state rows are stored in 8 bits, one scale per key row of V values, and read back into other rows:
               i8 has the least bf16 scale s >= 2^-100 with 127 s >= max|x| and codes round(x / s), e4m3 the least
               power of two s >= 2^-100 with 448 s >= max|x| and the code nearest x / s; ties to even
  cache_load   stored rows are read back, one slot into several rows, or zero where a row has no slot
"""
import math
import random

import torch

own = False

K, W = 128, 16
KINDS = ("mamba2", "gdn", "kda")
FORMATS = ("i8", "e4m3")


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _tree(name, op, kind, H, Hk, V, dtype, n, nodes, rank=0, shape="tree", lens=0):
    """n trees of `nodes` nodes in all; rank: mean rank of the sketch heads (0: every head reads its state)."""
    c = {"op": op, "kind": kind, "H": H, "Hk": Hk, "V": V, "dtype": dtype, "n": n, "nodes": nodes, "rank": rank,
         "shape": shape, "lens": lens}
    return dict(c, name=name) if name else c


def _cache(name, op, H, V, fmt, n, slots, lens=0):
    c = {"op": op, "H": H, "V": V, "fmt": fmt, "n": n, "slots": slots, "lens": lens}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of one sequence over its state and window: the smallest call
        _tree("tree_read gdn one token", "tree_read", "gdn", 32, 32, 128, "bf16", 1, 1),
        # a serving batch of a Gated DeltaNet layer, about 16 drafted tokens per sequence, verified on the state
        _tree("tree_read gdn batch", "tree_read", "gdn", 32, 16, 128, "bf16", 128, 2049, 0, "tree", 3),
        # the Nano-shaped Mamba-2 layer, small trees over the sketch of mean rank 6
        _tree("tree_read mamba2 sketch", "tree_read", "mamba2", 128, 8, 80, "bf16", 192, 1501, 6, "tree", 5),
        # the same layer, wide trees verified on the state
        _tree("tree_read mamba2 wide", "tree_read", "mamba2", 128, 8, 80, "bf16", 64, 3001, 0, "tree", 7),
        # a KDA layer over the sketch of mean rank 10: one decay per key channel
        _tree("tree_read kda sketch", "tree_read", "kda", 32, 32, 128, "bf16", 160, 1603, 10, "tree", 9),
        # float32 activations, drafted chains, another width
        _tree("tree_read gdn float32 chains", "tree_read", "gdn", 32, 32, 96, "f32", 40, 301, 0, "chain", 11),
        # a verified batch of the Nano-shaped layer keeps its accepted tokens
        _tree("tree_accept mamba2 batch", "tree_accept", "mamba2", 128, 8, 80, "bf16", 192, 1501, 0, "tree", 13),
        # one sequence of a KDA layer
        _tree("tree_accept kda one", "tree_accept", "kda", 32, 32, 128, "bf16", 1, 17, 0, "tree", 15),
        # a batch of Nano-shaped prompts' states into the prefix cache and out again for new sequences
        _cache("cache_fork nano batch", "cache_fork", 128, 80, "i8", 48, 61, 17),
        # one delta-rule sequence forked
        _cache("cache_fork one", "cache_fork", 32, 128, "e4m3", 1, 3, 19),
        # a batch that starts from a few cached prefixes, some rows from none
        _cache("cache_load prefixes", "cache_load", 32, 128, "e4m3", 96, 7, 21),
        # few rows from a larger cache at a width between
        _cache("cache_load few", "cache_load", 40, 112, "i8", 5, 33, 23),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree_read", "tree_read", "tree_read", "tree_accept", "cache_fork", "cache_load"])
    V, lens = rng.choice([64, 80, 96, 112, 128]), rng.randrange(1 << 16)
    if op.startswith("cache"):
        H = rng.choice([8, 12, 32, 40, 128])
        n = _log(rng, 1, 47 * 128 * 80 // (H * V))
        return _cache(None, op, H, V, rng.choice(FORMATS), n, n + rng.randrange(9) if op == "cache_fork" else
                      _log(rng, 1, 48), lens)
    kind, dtype = rng.choice(KINDS), rng.choice(["bf16", "bf16", "bf16", "f32"])
    H = rng.choice([8, 16, 32, 40, 64] + ([128] if kind == "mamba2" else []))
    Hk = H // rng.choice([1, 1, 2, 8] if kind != "mamba2" else [1, 8, 8])
    n = _log(rng, 1, min(192, 64 * 128 * 80 // (H * V)))
    nodes = min(n * _log(rng, 1, 50), 2048 * 32 // H)
    rank = rng.choice([0, 0, 6, 21]) if op == "tree_read" else 0
    return _tree(None, op, kind, H, Hk, V, dtype, min(n, nodes), nodes, rank, rng.choice(["tree", "tree", "chain"]), lens)


def _plan_of(case):
    """What a case's sequences are, apart from the values: per sequence its number of nodes, their parents (-1: the
    window's last token), its held-back tokens and its accepted node; per head its rank and group."""
    rng = random.Random(case["lens"])
    n, cap, chain = case["n"], 64, case["shape"] == "chain"
    w = [0.3 + rng.random() for _ in range(n)]
    sizes = [min(cap, 1 + int((case["nodes"] - n) * x / sum(w))) for x in w]
    left, i = case["nodes"] - sum(sizes), 0
    while left:
        add = min(left, cap - sizes[i], 1 + left // n)
        sizes[i], left, i = sizes[i] + add, left - add, (i + 1) % n
    trees, held, taken = [], [], []
    for size in sizes:
        par = [j - 1 if chain or rng.random() < 0.3 else rng.randint(-1, j - 1) for j in range(size)]
        depth = []
        for p in par:
            depth.append(1 if p < 0 else depth[p] + 1)
        p = rng.randint(0, W)
        fits = [j for j in range(size) if depth[j] <= W - p]
        trees.append((par, depth))
        held.append(p)
        taken.append(rng.choice(fits) if fits and rng.random() < 0.9 else -1)
    H, G = case["H"], min(8, case["H"])
    ranks = [min(49, 1 + int(rng.expovariate(1.0) * case["rank"])) if case["rank"] and rng.random() > 0.03 else 0
             for _ in range(H)]
    return {"sizes": sizes, "trees": trees, "held": held, "taken": taken, "ranks": ranks,
            "groups": [h * G // H for h in range(H)], "G": G}


def _frames(plan):
    """The distinct (group, rank) pairs of sketch heads in order, and each one's first row of the frames array."""
    pairs = sorted({(g, r) for g, r in zip(plan["groups"], plan["ranks"]) if r})
    first, at = {}, 0
    for pair in pairs:
        first[pair] = at
        at += pair[1]
    return first, at


# ---------------------------------------------------------------------------
# inputs: the distributions of the layer's activations and states
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    n, H, V = case["n"], case["H"], case["V"]
    order = list(range(n))
    random.Random(seed).shuffle(order)
    if case["op"].startswith("cache"):
        i8 = case["fmt"] == "i8"
        slots = random.Random(seed + 1)
        spread = lambda *s: 0.05 * torch.exp(rn(*s))  # noqa: E731  (key rows of a state differ in size)
        if case["op"] == "cache_fork":
            return {"case": case, "S": rn(n, H, K, V) * spread(n, H, K, 1), "rows": i32(order),
                    "codes": torch.zeros(case["slots"], H, K, V, device="cuda").to(torch.int8 if i8 else
                                                                                  torch.float8_e4m3fn),
                    "scales": torch.zeros(case["slots"], H, K, dtype=torch.bfloat16, device="cuda"),
                    "slots": i32(slots.sample(range(case["slots"]), n)), "rows2": i32(order[::-1]),
                    "S2": torch.zeros(n, H, K, V, device="cuda")}
        x = rn(case["slots"], H, K, V).clamp(-4, 4)
        codes = torch.round(x * 31).to(torch.int8) if i8 else (x * 112).to(torch.float8_e4m3fn)
        scales = (spread(case["slots"], H, K) / 128).to(torch.bfloat16)
        if not i8:
            scales = torch.exp2(torch.floor(torch.log2(scales.float()))).to(torch.bfloat16)
        return {"case": case, "codes": codes, "scales": scales, "rows": i32(order),
                "slots": i32([slots.randrange(case["slots"]) if slots.random() < 0.9 else -1 for _ in range(n)]),
                "S": torch.zeros(n, H, K, V, device="cuda")}
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    Hk, T, kda, delta = case["Hk"], case["nodes"], case["kind"] == "kda", case["kind"] != "mamba2"
    plan = _plan_of(case)
    B = n + 2  # the cache has rows that the call does not name

    def keys(*s):
        k = rn(*s)
        return (k / k.norm(dim=-1, keepdim=True)).to(dt)

    decay = lambda *s: torch.exp(-0.1 * torch.nn.functional.softplus(rn(*s)))  # noqa: E731
    off, rows = [0], [r + 1 for r in order]
    for size in plan["sizes"]:
        off.append(off[-1] + size)
    pos = [0] * B
    for r, p in zip(rows, plan["held"]):
        pos[r] = p
    s = {"case": case, "plan": plan, "offsets": i32(off), "parents": i32([p for par, _ in plan["trees"] for p in par]),
         "rows": i32(rows), "max_nodes": max(plan["sizes"]), "pos": i32(pos),
         "depth": max(d for _, depth in plan["trees"] for d in depth),
         "k": keys(T, Hk, K), "v": rn(T, H, V).to(dt), "a": decay(T, H, K) if kda else decay(T, H),
         "beta": torch.sigmoid(rn(T, H)) if delta else None,
         "kbuf": keys(W, Hk, B, K), "vbuf": rn(W, H, B, V).to(dt),
         "abuf": decay(W, H, B, K) if kda else decay(W, H, B), "bbuf": torch.sigmoid(rn(W, H, B)) if delta else None}
    if case["op"] == "tree_accept":
        return dict(s, accepted=i32(plan["taken"]), new_pos=torch.zeros_like(s["pos"]))
    z = B * V * sum(plan["ranks"])
    rows_f = _frames(plan)[1]
    return dict(s, q=rn(T, Hk, K).to(dt), S=0.05 * rn(B, H, K, V), Z=0.05 * rn(z) if z else None,
                frames=rn(rows_f, K) / math.sqrt(K) if rows_f else None, y=torch.empty(T, H, V, device="cuda"))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    return {"tree_read": _own_read if own else _plain_read, "tree_accept": _own_accept if own else _plain_accept,
            "cache_fork": _own_fork if own else _plain_fork, "cache_load": _own_load if own else _plain_load}[op](state)


def _shape(s, B, kind="gdn", dtype="bf16", Hk=0, G=1):
    """The layer's descriptor, which a program makes once."""
    if "shape" not in s:
        from rank_state_read_amd import make_shape
        c = s["case"]
        s["shape"] = make_shape(B, c["H"], K, c["V"], W, G, 79, 49, kind, dtype, Hk)
    return s["shape"]


def _tree_shape(s):
    c = s["case"]
    return _shape(s, s["pos"].numel(), c["kind"], c["dtype"], c["Hk"], s["plan"]["G"])


def _own_read(s):
    from rank_state_read_amd import Plan, sketchssm_tree_read
    if "handle" not in s:  # the layer's plan, made once too
        s["handle"] = Plan(_tree_shape(s), s["plan"]["ranks"], s["plan"]["groups"])
    sketchssm_tree_read(s["handle"], s["S"], s["Z"], s["frames"], s["kbuf"], s["vbuf"], s["abuf"], s["bbuf"], s["pos"],
                        s["rows"], s["offsets"], s["max_nodes"], s["parents"], s["q"], s["k"], s["v"], s["a"], s["beta"],
                        s["y"])
    return s["y"]


def _own_accept(s):
    from rank_state_read_amd import sketchssm_tree_accept
    sketchssm_tree_accept(_tree_shape(s), s["kbuf"], s["vbuf"], s["abuf"], s["bbuf"], s["pos"], s["new_pos"], s["rows"],
                          s["offsets"], s["parents"], s["accepted"], s["k"], s["v"], s["a"], s["beta"])
    return {key: s[key] for key in ("kbuf", "vbuf", "abuf", "bbuf", "new_pos") if s[key] is not None}


def _own_fork(s):
    from rank_state_read_amd import sketchssm_cache_load, sketchssm_cache_store
    c = s["case"]
    shape = _shape(s, c["n"])
    sketchssm_cache_store(shape, s["S"], s["rows"], s["codes"], s["scales"], s["slots"], c["fmt"])
    sketchssm_cache_load(shape, s["codes"], s["scales"], s["slots"], s["S2"], s["rows2"], c["fmt"])
    return {"S2": s["S2"], "scales": s["scales"]}


def _own_load(s):
    from rank_state_read_amd import sketchssm_cache_load
    c = s["case"]
    sketchssm_cache_load(_shape(s, c["n"]), s["codes"], s["scales"], s["slots"], s["S"], s["rows"], c["fmt"])
    return s["S"]


def _plain_read(s):
    c = s["case"]
    H, share, n, N = c["H"], c["H"] // c["Hk"], c["n"], s["max_nodes"]
    delta, kda = c["kind"] != "mamba2", c["kind"] == "kda"
    first, rows = s["offsets"][:-1].long()[:, None], s["rows"].long()
    i = torch.arange(N, device="cuda")[None]
    live = i < s["offsets"][1:].long()[:, None] - first
    at = torch.where(live, first + i, first)
    heads = lambda t: t.float().repeat_interleave(share, -2)  # noqa: E731
    x = heads(s["q"][at])  # [n, N, H, K]
    acc = torch.zeros(n, N, H, c["V"], device="cuda")

    def back(x, acc, k, v, a, beta, on):
        """The carried queries and their sums past one token each (of those that have it: on)."""
        w = (x * k).sum(-1)
        if delta:
            w = w * beta
        acc = torch.where(on[..., None, None], acc + w[..., None] * v, acc)
        if delta:
            x = torch.where(on[..., None, None], (x - w[..., None] * k) * (a if kda else a[..., None]), x)
        else:
            x = torch.where(on[..., None, None], x * a[..., None], x)
        return x, acc

    node, par = torch.where(live, i, -1), s["parents"].long()
    for _ in range(s["depth"]):
        tok = first + node.clamp(min=0)
        x, acc = back(x, acc, heads(s["k"][tok]), s["v"][tok].float(), s["a"][tok], s["beta"][tok] if delta else None,
                      node >= 0)
        node = torch.where(node >= 0, par[tok], node)
    held = s["pos"].long()[rows][:, None]
    for slot in reversed(range(W)):
        k, v = heads(s["kbuf"][slot].transpose(0, 1)[rows]), s["vbuf"][slot].transpose(0, 1)[rows].float()
        a, beta = s["abuf"][slot].transpose(0, 1)[rows], s["bbuf"][slot].transpose(0, 1)[rows] if delta else None
        x, acc = back(x, acc, k[:, None], v[:, None], a[:, None], beta[:, None] if delta else None, held > slot)
    x, y = x.transpose(1, 2).contiguous(), acc.transpose(1, 2).contiguous()  # [n, H, N, ...]
    plan, (frame, _), B = s["plan"], _frames(s["plan"]), s["pos"].numel()
    dense = torch.tensor([h for h in range(H) if plan["ranks"][h] == 0], device="cuda", dtype=torch.long)
    if len(dense) == H:
        y = y + x @ s["S"][rows]
    elif len(dense):
        y[:, dense] += x[:, dense] @ s["S"][rows[:, None], dense[None]]
    z = 0
    for h in range(H):
        r = plan["ranks"][h]
        if r:
            f0 = frame[plan["groups"][h], r]
            Zh = s["Z"][z * c["V"]:(z + B * r) * c["V"]].view(B, r, c["V"])
            y[:, h] += (x[:, h] @ s["frames"][f0:f0 + r].t().contiguous()) @ Zh[rows]
            z += B * r
    s["y"][at[live]] = y.transpose(1, 2)[live]
    return s["y"]


def _plain_accept(s):
    first, rows, node = s["offsets"][:-1].long(), s["rows"].long(), s["accepted"].long()
    par, old = s["parents"].long(), s["pos"].long()[s["rows"].long()]
    path = []  # accepted node first
    for _ in range(W):
        path.append(node)
        node = torch.where(node >= 0, par[first + node.clamp(min=0)], node)
    length = torch.stack([m >= 0 for m in path]).sum(0)
    for t, m in enumerate(path):
        on = m >= 0
        slot = torch.where(on, old + length - 1 - t, 0)
        tok = first + m.clamp(min=0)
        for buf, new in ((s["kbuf"], s["k"]), (s["vbuf"], s["v"]), (s["abuf"], s["a"]), (s["bbuf"], s["beta"])):
            if buf is not None:
                new = new[tok]
                buf[slot, :, rows] = torch.where(on.view((-1,) + (1,) * (new.dim() - 1)), new, buf[slot, :, rows])
    s["new_pos"].copy_(s["pos"])
    s["new_pos"][rows] = (old + length).int()
    return {key: s[key] for key in ("kbuf", "vbuf", "abuf", "bbuf", "new_pos") if s[key] is not None}


def _plain_fork(s):
    rows, slots = s["rows"].long(), s["slots"].long()
    x = s["S"][rows]
    top = x.abs().amax(-1).double()
    if s["case"]["fmt"] == "i8":
        bits = (top / torch.full_like(top, 127)).float().clamp(min=2.0 ** -100).view(torch.int32) & -65536
        scale = bits.view(torch.float32)
        scale = torch.where(scale.double() * 127 < top, (bits + 65536).view(torch.float32), scale)
        codes = torch.round(x.double() / scale.double()[..., None]).to(torch.int8)
    else:
        m, e = torch.frexp(top / torch.full_like(top, 448))
        scale = torch.exp2(torch.where(m == 0.5, e - 1, e).clamp(min=-100).float())
        codes = (x / scale[..., None]).to(torch.float8_e4m3fn)
    s["scales"][slots] = scale.to(torch.bfloat16)
    codes = codes.float()
    s["S2"][s["rows2"].long()] = codes * scale[..., None]
    return {"S2": s["S2"], "scales": s["scales"]}


def _plain_load(s):
    slots = s["slots"].long()
    on = slots >= 0
    at = slots.clamp(min=0)
    codes = s["codes"].view(torch.uint8)[at].view(s["codes"].dtype)
    x = codes.float() * s["scales"][at].float()[..., None]
    s["S"][s["rows"].long()] = torch.where(on.view(-1, 1, 1, 1), x, torch.zeros_like(x))
    return s["S"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree_read": _exact_read, "tree_accept": _exact_accept, "cache_fork": _exact_fork,
            "cache_load": _exact_load}[case["op"]](s)


def _exact_read(s):
    """Forwards: every node has its own state, its parent's with one token applied; a sketch head's first state is
    F^T Z, which the carried query reads as Z^T F does."""
    c, plan = s["case"], s["plan"]
    H, V, share, B = c["H"], c["V"], c["H"] // c["Hk"], s["pos"].numel()
    frame, _ = _frames(plan)
    off, rows = s["offsets"].tolist(), s["rows"].tolist()
    first = torch.empty(c["n"], H, K, V, dtype=torch.float64, device="cuda") if any(plan["ranks"]) else None
    if first is not None:
        at = 0
        for h, (g, r) in enumerate(zip(plan["groups"], plan["ranks"])):
            if r:
                Z = s["Z"][at * V:(at + B * r) * V].view(B, r, V)[rows].double()
                f0 = frame[g, r]
                first[:, h] = torch.einsum("rk,nrv->nkv", s["frames"][f0:f0 + r].double(), Z)
                at += B * r
            else:
                first[:, h] = s["S"][rows, h].double()
    y = torch.empty(c["nodes"], H, V, dtype=torch.float64, device="cuda")

    def after(S, k, v, a, beta):
        k = k.double().repeat_interleave(share, 0)[:, :, None]
        S = S * (a.double()[:, :, None] if c["kind"] == "kda" else a.double()[:, None, None])
        u = v.double()[:, None]
        if c["kind"] != "mamba2":
            u = beta.double()[:, None, None] * (u - (k * S).sum(1, keepdim=True))
        return torch.addcmul(S, k, u)

    for i, row in enumerate(rows):
        root = s["S"][row].double() if first is None else first[i]
        for j in range(plan["held"][i]):
            root = after(root, s["kbuf"][j, :, row], s["vbuf"][j, :, row], s["abuf"][j, :, row],
                         None if s["bbuf"] is None else s["bbuf"][j, :, row])
        par, states = plan["trees"][i][0], {-1: root}
        last = {p: j for j, p in enumerate(par)}  # each state is let go behind its last child
        for j, p in enumerate(par):
            t = off[i] + j
            S = after(states[p], s["k"][t], s["v"][t], s["a"][t], None if s["beta"] is None else s["beta"][t])
            y[t] = (s["q"][t].double().repeat_interleave(share, 0)[:, :, None] * S).sum(1)
            if j in last:
                states[j] = S
            if last[p] == j:
                del states[p]
    return y


def _exact_accept(s):
    """The same copies, one token at a time."""
    bufs = [(s[b], s[t]) for b, t in (("kbuf", "k"), ("vbuf", "v"), ("abuf", "a"), ("bbuf", "beta")) if s[b] is not None]
    off, plan, pos = s["offsets"].tolist(), s["plan"], s["pos"].tolist()
    for i, row in enumerate(s["rows"].tolist()):
        path, node = [], plan["taken"][i]
        while node >= 0:
            path.insert(0, node)
            node = plan["trees"][i][0][node]
        for m in path:
            for buf, new in bufs:
                buf[pos[row], :, row] = new[off[i] + m]
            pos[row] += 1
    out = {key: s[key].double() for key in ("kbuf", "vbuf", "abuf", "bbuf") if s[key] is not None}
    return dict(out, new_pos=torch.tensor(pos, dtype=torch.int32, device="cuda"))


def _exact_fork(s):
    x = s["S"].double()
    out, scales = torch.zeros_like(x), s["scales"].double()
    for src, slot, dst in zip(s["rows"].tolist(), s["slots"].tolist(), s["rows2"].tolist()):
        v = x[src]
        top = v.abs().amax(-1, keepdim=True)
        if s["case"]["fmt"] == "i8":  # 8 significant bits, rounded up
            full = top / torch.full_like(top, 127)
            step = torch.exp2(torch.floor(torch.log2(full)) - 7)
            scale = (torch.ceil(full / step) * step).clamp(min=2.0 ** -100)
            out[dst] = torch.round(v / scale) * scale
        else:  # 4 significant bits down to 2^-6, then steps of 2^-9
            scale = torch.exp2(torch.ceil(torch.log2(top / torch.full_like(top, 448)))).clamp(min=2.0 ** -100)
            t = v / scale
            step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
            out[dst] = torch.round(t / step) * step * scale
        scales[slot] = scale[..., 0]
    return {"S2": out, "scales": scales}


def _exact_load(s):
    out = torch.zeros(s["S"].shape, dtype=torch.float64, device="cuda")
    for row, slot in zip(s["rows"].tolist(), s["slots"].tolist()):
        if slot >= 0:
            out[row] = s["codes"][slot].float().double() * s["scales"][slot].double()[:, :, None]
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    H, V, n = case["H"], case["V"], case["n"]
    if case["op"].startswith("cache"):
        item = n * H * K
        small, large = item * (V + 2), item * V * 4
        if case["op"] == "cache_fork":
            return {"bytes": 2 * (small + large), "flops": 6 * item * V}
        used = min(n, case["slots"]) * H * K * (V + 2)
        return {"bytes": used + large, "flops": item * V}
    e, Hk, T = 2 if case["dtype"] == "bf16" else 4, case["Hk"], case["nodes"]
    kda, delta = case["kind"] == "kda", case["kind"] != "mamba2"
    plan = _plan_of(case)
    token = e * (Hk * K + H * V) + 4 * H * ((K if kda else 1) + (1 if delta else 0))
    if case["op"] == "tree_accept":
        kept = sum(depth[m] for (_, depth), m in zip(plan["trees"], plan["taken"]) if m >= 0)
        return {"bytes": 2 * kept * token + 8 * n, "flops": 0}
    ranks = plan["ranks"]
    first = 4 * n * V * sum(r or K for r in ranks) + 4 * K * _frames(plan)[1]
    flops = T * sum(2 * r * (K + V) if r else 2 * K * V for r in ranks)
    steps = sum(len(d) * p + sum(d) for (_, d), p in zip(plan["trees"], plan["held"]))
    flops += steps * H * ((4 if delta else 2) * K + 2 * V)
    return {"bytes": first + sum(plan["held"]) * token + T * (token + e * Hk * K + 4 * H * V + 4), "flops": flops}
