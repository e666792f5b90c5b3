"""Timed cases of the operators of drafted decoding: rotary positions in every
layout and scaled for long contexts, attention of trees of drafted tokens over
a cache, and the acceptance of a tree's path with the move of its cells.

A tree of n drafted tokens stands in cells base .. base + n - 1 of its
sequence's cache, in the order of its nodes; the cells before base are the
sequence's earlier tokens.  A node's position is base + its depth, and it sees
the earlier cells, its ancestors and itself.  A step holds the nodes of several
trees as consecutive rows: tree i has rows row0[i] .. row0[i + 1] - 1.

A case's "op":
  table    cos and sin of positions, the frequencies scaled for long contexts
  rope     rows of q, k, v heads: q and k rotated (the whole head or its first
           n_rot elements, adjacent pairs or halves; normed before where
           "norm"), q out, k and v to their cells of an fp16 cache
  tree     attention of the nodes of one or more trees over their sequences'
           caches; bit j of row t's mask (int32 words) says that it sees cell
           base + j
  accept   the path that a tree's target tokens accept, and its keys and values
           moved to the cells behind the sequence's earlier tokens, every layer
"""
import math

import torch

own = False

EPS = 1e-5
_L = None


def _lib():
    global _L
    if _L is None:
        import llama_decoder_forward_02_gb300 as L
        _L = L
    return _L


def _stream():
    return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the table of a context of the ~1B shape, frequencies stretched by bands
        {"name": "table 4096 hd64 bands", "op": "table", "n_pos": 4096, "n_rot": 64, "theta": 500000.0,
         "scaling": "bands", "factor": 8.0, "orig": 1024},
        # the table of a very long context, frequencies stretched by a ramp
        {"name": "table 131072 hd128 ramp", "op": "table", "n_pos": 131072, "n_rot": 128, "theta": 500000.0,
         "scaling": "ramp", "factor": 4.0, "orig": 32768},
        # a tree of 16 drafted tokens of the 8B shape
        {"name": "rope T16 tree", "op": "rope", "T": 16, "H": 32, "Hkv": 8, "hd": 128, "n_rot": 128, "layout": "pairs",
         "norm": False, "tree": True, "n_seq": 1, "n_ctx": 4096},
        # one ubatch of the ~1B shape in a model whose rotation takes half of each head, as halves
        {"name": "rope T512 hd64 part", "op": "rope", "T": 512, "H": 32, "Hkv": 8, "hd": 64, "n_rot": 32,
         "layout": "halves", "norm": False, "tree": False, "n_seq": 2, "n_ctx": 4096},
        # a long prompt's rows at once, whole heads as halves, normed
        {"name": "rope T4096 halves", "op": "rope", "T": 4096, "H": 32, "Hkv": 8, "hd": 128, "n_rot": 128,
         "layout": "halves", "norm": True, "tree": False, "n_seq": 1, "n_ctx": 4608},
        # a small tree of the ~1B shape early in its context
        {"name": "tree 8 of 700 hd64", "op": "tree", "H": 32, "Hkv": 8, "hd": 64, "n_ctx": 4096, "trees": "700+8",
         "window": 0, "kv": "f16", "holes": False},
        # a usual tree of the 8B shape behind a 2048-token prompt
        {"name": "tree 16 of 2100", "op": "tree", "H": 32, "Hkv": 8, "hd": 128, "n_ctx": 4096, "trees": "2100+16",
         "window": 0, "kv": "f16", "holes": False},
        # a wide tree in a 32k context
        {"name": "tree 64 of 32000", "op": "tree", "H": 32, "Hkv": 8, "hd": 128, "n_ctx": 32768, "trees": "32000+64",
         "window": 0, "kv": "f16", "holes": False},
        # a usual tree in a 32k context with an FP8 cache
        {"name": "tree 16 of 32000 e4m3", "op": "tree", "H": 32, "Hkv": 8, "hd": 128, "n_ctx": 32768,
         "trees": "32000+16", "window": 0, "kv": "e4m3", "holes": False},
        # eight sequences of different lengths, a tree each
        {"name": "tree 8 ragged", "op": "tree", "H": 32, "Hkv": 8, "hd": 128, "n_ctx": 8192,
         "trees": "1882+16,1582+12,2911+16,3415+9,2775+16,2634+5,1781+16,748+14", "window": 0, "kv": "f16",
         "holes": False},
        # a tree of 16 over the 32 layers of the 8B shape
        {"name": "accept 16", "op": "accept", "trees": "100+16", "accepted": "5", "n_layer": 32, "Hkv": 8, "hd": 128,
         "n_ctx": 512},
        # eight trees of 64 over the 32 layers of the 8B shape
        {"name": "accept 8x64", "op": "accept", "trees": ",".join(f"{37 * i}+64" for i in range(8)),
         "accepted": "4,9,1,6,12,3,7,5", "n_layer": 32, "Hkv": 8, "hd": 128, "n_ctx": 512},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rope", "rope", "tree", "tree", "tree", "tree", "accept"])
    hd = rng.choice([32, 64, 128, 128])
    if op == "table":
        return {"op": op, "n_pos": _log(rng, 100, 100000), "n_rot": 8 * rng.randint(1, 16),
                "theta": rng.choice([10000.0, 500000.0, 1000000.0]),
                "scaling": rng.choice(["none", "linear", "bands", "ramp"]), "factor": rng.choice([2.0, 4.0, 8.0, 32.0]),
                "orig": rng.choice([2048, 4096, 8192, 32768])}
    H, Hkv = rng.choice([(32, 8), (16, 8), (8, 1), (8, 8), (40, 8), (12, 4), (6, 2)])
    if op == "rope":
        T = _log(rng, 1, 3000)
        return {"op": op, "T": T, "H": H, "Hkv": Hkv, "hd": hd, "n_rot": rng.choice([hd, hd, 8 * rng.randint(1, hd // 8)]),
                "layout": rng.choice(["pairs", "halves"]), "norm": rng.random() < 0.4, "tree": T <= 64,
                "n_seq": rng.randint(1, 3), "n_ctx": T + rng.randint(1, 500)}
    n = rng.choice([1, 1, 2, rng.randint(3, 8)])
    if op == "accept":
        nodes = [_log(rng, 1, 64) for _ in range(n)]
        trees = [(rng.randint(0, 300), m) for m in nodes]
        return {"op": op, "trees": ",".join("%d+%d" % t for t in trees),
                "accepted": ",".join(str(rng.randint(1, (m + 1) // 2)) for m in nodes),
                "n_layer": _log(rng, 1, 32), "Hkv": Hkv, "hd": hd, "n_ctx": 400}
    nodes = [_log(rng, 1, 200 if n == 1 else 48) for _ in range(n)]
    far = min(30000 if n == 1 else 6000, 60_000_000 // (H * sum(nodes)))       # no dearer than the largest listed case
    trees = [(rng.choice([0, _log(rng, 1, far), _log(rng, 1, far), _log(rng, 1, far)]), m) for m in nodes]
    return {"op": op, "H": H, "Hkv": Hkv, "hd": hd, "n_ctx": max(a + b for a, b in trees) + rng.randint(0, 300),
            "trees": ",".join("%d+%d" % t for t in trees), "window": rng.choice([0, 0, _log(rng, 1, 4000)]),
            "kv": rng.choice(["f16", "f16", "e4m3"]), "holes": rng.random() < 0.25}


# ------------------------------------------------------------------ inputs

def _rand(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale


def _trees(case):
    return [tuple(map(int, t.split("+"))) for t in case["trees"].split(",")]


def _parents(n, g):
    """Each node's parent in its tree: node 0 the root, the rest under a random earlier node."""
    u = torch.rand(n, generator=g)
    return [-1] + [int(u[i] * i) for i in range(1, n)]


def _depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _frequencies(case):
    """Radians a position of each pair, and the factor of cos and sin, in 64 bits."""
    n, theta, s = case["n_rot"], case["theta"], case["factor"]
    f = [theta ** (-2.0 * i / n) for i in range(n // 2)]
    if case["scaling"] == "linear":
        return [x / s for x in f], 1.0
    if case["scaling"] == "bands":
        # wavelengths above orig / 1 are stretched, those below orig / 4 kept, with a straight line between
        out = []
        for x in f:
            keep = min(max((case["orig"] * x / (2 * math.pi) - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            out.append(x * keep + x / s * (1 - keep))
        return out, 1.0
    if case["scaling"] == "ramp":
        # pairs that turn more than 32 times in orig positions are kept, those that turn less than once stretched
        def pair(turns):
            return n * math.log(case["orig"] / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), n - 1)
        out = []
        for i, x in enumerate(f):
            ramp = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            out.append(x / s * ramp + x * (1 - ramp))
        return out, 0.1 * math.log(s) + 1.0
    return f, 1.0


def _table(n_pos, f, m):
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * torch.tensor(f, dtype=torch.float64).cuda()
    return torch.stack((a.cos() * m, a.sin() * m), -1)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    gh = torch.Generator().manual_seed(int(seed))
    op = case["op"]
    s = {"op": op, "case": dict(case), "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if op == "table":
        # other positions for another seed
        s["pos0"] = int(torch.randint(0, 1000, (1,), generator=gh))
        s["f"], s["m"] = _frequencies(case)
        s["out"] = torch.empty((case["n_pos"], case["n_rot"] // 2, 2), device="cuda")
        s["rope"] = None
        return s
    if op == "rope":
        T, H, Hkv, hd, n_seq, n_ctx = (case[k] for k in ("T", "H", "Hkv", "hd", "n_seq", "n_ctx"))
        s["qkv"] = _rand((T, (H + 2 * Hkv) * hd), g, 1.3)
        s["q_gain"], s["k_gain"] = ([1 + _rand((hd,), g, 0.1) for _ in range(2)] if case["norm"] else (None, None))
        base = int(torch.randint(0, n_ctx - T + 1, (1,), generator=gh))
        # a run of consecutive cells for each sequence; a tree's positions go by depth
        seq = torch.arange(T) * n_seq // T
        first = torch.searchsorted(seq, torch.arange(n_seq))
        cell = torch.arange(T) - first[seq] + base
        pos = torch.tensor(_depths(_parents(T, gh))) + base if case["tree"] else cell
        s["cell"], s["pos"], s["seq"] = (v.to(torch.int32).cuda() for v in (cell, pos, seq))
        n = case["n_rot"]
        s["table"] = _table(n_ctx, [10000.0 ** (-2.0 * i / n) for i in range(n // 2)], 1.0).float()
        s["q"] = torch.empty((T, H * hd), dtype=torch.float16, device="cuda")
        s["kc"], s["vc"] = (torch.zeros((n_seq, Hkv, n_ctx, hd), dtype=torch.float16, device="cuda") for _ in range(2))
        p = [0 if s[k] is None else s[k].data_ptr()
             for k in ("qkv", "q_gain", "k_gain", "table", "pos", "cell", "seq", "q", "kc", "vc", "err")]
        s["args"] = (p[0], (H + 2 * Hkv) * hd, p[1], p[2], EPS, p[3], n_ctx, n, int(case["layout"] == "halves"), p[4],
                     p[5], p[6], p[7], 1, p[8], p[9], 0, T, H, Hkv, hd, n_ctx, n_seq, p[10])
        return s
    trees = _trees(case)
    n_tree, nodes = len(trees), [b for _, b in trees]
    T, most = sum(nodes), max(nodes)
    row0 = [0]
    for b in nodes:
        row0.append(row0[-1] + b)
    s.update(T=T, most=most, row0_host=row0, row0=_ints(row0), seq=_ints(list(range(n_tree))[::-1]),
             base=_ints([a for a, _ in trees]))
    Hkv, hd, n_ctx = case["Hkv"], case["hd"], case["n_ctx"]
    if op == "accept":
        # distinct tokens; the accepted nodes lie behind those that the path's cells hold now, as in a tree written by levels
        token, parent, target = [], [], []
        for n, a in zip(nodes, map(int, case["accepted"].split(","))):
            path = [0] + sorted((torch.randperm(n - a, generator=gh)[:a - 1] + a).tolist())
            par = _parents(n, gh)
            tok = torch.randperm(32000, generator=gh)[:2 * n].tolist()
            tgt = tok[n:]
            for x, y in zip(path, path[1:]):
                par[y], tgt[x] = x, tok[y]
            token += tok[:n]
            parent += par
            target += tgt
        s.update(token=_ints(token), parent=_ints(parent), target=_ints(target))
        for k in ("kc", "vc"):
            s[k] = _rand((n_tree, case["n_layer"], Hkv, n_ctx, hd), g).to(torch.float16)
        s.update(path=torch.empty((n_tree, most), dtype=torch.int32, device="cuda"),
                 count=torch.empty(n_tree, dtype=torch.int32, device="cuda"),
                 next=torch.empty(n_tree, dtype=torch.int32, device="cuda"))
        p = {k: s[k].data_ptr() for k in ("token", "parent", "target", "row0", "seq", "base", "kc", "vc", "path", "count",
                                          "next", "err")}
        s["args"] = (p["token"], p["parent"], p["target"], p["row0"], p["seq"], p["base"], p["kc"], p["vc"], 0, p["path"],
                     p["count"], p["next"], T, n_tree, most, case["n_layer"], Hkv, hd, n_ctx, n_tree, p["err"])
        return s
    words = (most + 31) // 32
    mask = torch.zeros((T, words * 32), dtype=torch.bool)
    pos = []
    for (a, n), r in zip(trees, row0):
        par = _parents(n, gh)
        for i, p in enumerate(par):
            if p >= 0:
                mask[r + i] = mask[r + p]
            mask[r + i, i] = True
        pos += [a + d for d in _depths(par)]
    if case["holes"]:
        mask[torch.rand(T, generator=gh) < 0.3] = False          # rows that see no drafted cell, not even their own
    packed = (mask.view(T, words, 32).long() << torch.arange(32)).sum(-1)
    s["mask"] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32).cuda()
    s["pos"] = _ints(pos)
    H = case["H"]
    s["q"] = _rand((T, H * hd), g, 1.5).to(torch.float16)
    for k in ("kc", "vc"):
        v = _rand((n_tree, Hkv, n_ctx, hd), g)
        s[k] = v.to(torch.float16) if case["kv"] == "f16" else v.to(torch.float8_e4m3fn)
    s["o"] = torch.empty((T, H * hd), dtype=torch.float16, device="cuda")
    s["scratch"] = None
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state, state["case"])


def _run_own(s):
    L = _lib()
    op, c = s["op"], s["case"]
    if op == "table":
        if s["rope"] is None:
            kind = {"none": L.LLM_ROPE_NONE, "linear": L.LLM_ROPE_LINEAR, "bands": L.LLM_ROPE_BANDS,
                    "ramp": L.LLM_ROPE_RAMP}[c["scaling"]]
            s["rope"] = L.rope(theta=c["theta"], n_rot=c["n_rot"], scaling=kind, factor=c["factor"], n_ctx_orig=c["orig"])
        L.check(L.llm_op_rope_table(s["rope"], s["pos0"], c["n_pos"], s["out"].data_ptr(), _stream()))
        return s["out"]
    if op == "rope":
        L.check(L.llm_op_rope_kv(*s["args"], _stream()))
        return s["q"], s["kc"], s["vc"]
    if op == "accept":
        L.check(L.llm_op_tree_accept(*s["args"], _stream()))
        return s["path"], s["count"], s["next"], s["kc"], s["vc"]
    if s["scratch"] is None:                                        # the workspace such a program keeps
        n_tree = len(s["row0_host"]) - 1
        size = L.llm_op_attn_tree_scratch_bytes(n_tree, s["most"], c["H"], c["Hkv"], c["hd"], c["n_ctx"])
        s["scratch"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        p = {k: s[k].data_ptr() for k in ("q", "kc", "vc", "row0", "seq", "base", "mask", "pos", "o", "scratch", "err")}
        s["args"] = (p["q"], p["kc"], p["vc"], p["row0"], p["seq"], p["base"], p["mask"], p["pos"], p["o"], s["T"], n_tree,
                     s["most"], c["H"], c["Hkv"], c["hd"], c["n_ctx"], n_tree,
                     L.LLM_KV_F16 if c["kv"] == "f16" else L.LLM_KV_E4M3, c["window"], p["scratch"], size, p["err"])
    L.check(L.llm_op_attn_tree(*s["args"], _stream()))
    return s["o"]


def _plain_table(s, c):
    return _table(s["pos0"] + c["n_pos"], s["f"], s["m"])[s["pos0"]:].float()


def _plain_rope(s, c):
    H, Hkv, hd, n = c["H"], c["Hkv"], c["hd"], c["n_rot"]
    x = s["qkv"].unflatten(-1, (-1, hd))
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_gain"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_gain"]
    cs = s["table"][s["pos"].long()][:, None]
    co, si = cs[..., 0], cs[..., 1]

    def turn(u):
        if c["layout"] == "pairs":
            a, b = u[..., 0:n:2], u[..., 1:n:2]
            r = torch.stack((a * co - b * si, a * si + b * co), -1).flatten(-2)
        else:
            a, b = u[..., :n // 2], u[..., n // 2:n]
            r = torch.cat((a * co - b * si, a * si + b * co), -1)
        return torch.cat((r, u[..., n:]), -1).to(torch.float16)
    at = (s["seq"].long(), slice(None), s["cell"].long())
    s["kc"][at] = turn(k)
    s["vc"][at] = v.to(torch.float16)
    return turn(q).flatten(1), s["kc"], s["vc"]


def _seen(mask, n, base, end, pos, window):
    """What rows see of cells 0 .. end - 1: [rows][end]."""
    cell = torch.arange(end, device="cuda")
    bits = (mask[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32) & 1).bool().flatten(1)[:, :n]
    before = torch.ones((len(mask), base), dtype=torch.bool, device="cuda")
    if window:
        before = cell[:base] > pos[:, None] - window
    return torch.cat((before, bits), 1)


def _plain_tree(s, c):
    H, Hkv, hd = c["H"], c["Hkv"], c["hd"]
    out = []
    for i, (base, n) in enumerate(_trees(c)):
        rows, at, end = slice(s["row0_host"][i], s["row0_host"][i + 1]), len(_trees(c)) - 1 - i, base + n
        k, v = s["kc"][at, :, :end].float(), s["vc"][at, :, :end].float()
        q = s["q"][rows].float().view(n, Hkv, H // Hkv, hd).permute(1, 2, 0, 3).flatten(1, 2) / math.sqrt(hd)
        seen = _seen(s["mask"][rows], n, base, end, s["pos"][rows], c["window"]).repeat(H // Hkv, 1)
        w = (q @ k.transpose(-1, -2)).masked_fill(~seen, -math.inf)
        top = w.amax(-1, keepdim=True)
        w = torch.exp(w - torch.where(top == -math.inf, torch.zeros_like(top), top))
        o = (w @ v) / w.sum(-1, keepdim=True).clamp_min(1e-30)      # a row that sees nothing is zero
        out.append(o.view(Hkv, H // Hkv, n, hd).permute(2, 0, 1, 3).reshape(n, H * hd).to(torch.float16))
    return torch.cat(out)


def _plain_accept(s, c):
    for i, (base, n) in enumerate(_trees(c)):
        r, at = s["row0_host"][i], len(_trees(c)) - 1 - i
        tok, par, tgt = s["token"][r:r + n], s["parent"][r:r + n], s["target"][r:r + n]
        node = torch.arange(n, device="cuda")
        # the child that a node's target accepts is the lowest with that token
        child = (par[None] == node[:, None]) & (tok[None] == tgt[:, None]) & (node[None] > 0)
        has, child = child.any(1), child.int().argmax(1)
        path, live, cur = torch.full((s["most"],), -1, dtype=torch.int32, device="cuda"), True, 0
        count = 0
        hops, nxt = has.tolist(), child.tolist()
        while live:
            path[count] = cur
            count += 1
            live, last = hops[cur], cur
            cur = nxt[cur]
        s["path"][i] = path
        s["count"][i] = count
        s["next"][i] = tgt[last]
        src = base + path[:count].long()
        for cache in (s["kc"], s["vc"]):
            cache[at, :, :, base:base + count] = cache[at, :, :, src]
    return s["path"], s["count"], s["next"], s["kc"], s["vc"]


_PLAIN = {"table": _plain_table, "rope": _plain_rope, "tree": _plain_tree, "accept": _plain_accept}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "table":
        n = case["n_pos"] * case["n_rot"] // 2
        return {"bytes": 8 * n, "flops": 30 * n}
    Hkv, hd = case["Hkv"], case["hd"]
    if op == "rope":
        T, H = case["T"], case["H"]
        return {"bytes": 4 * T * (H + 2 * Hkv) * hd + 2 * T * (H + 2 * Hkv) * hd + 4 * case["n_rot"] * T,
                "flops": T * (H + Hkv) * (case["n_rot"] * 3 + (4 * hd if case["norm"] else 0))}
    trees = _trees(case)
    T = sum(n for _, n in trees)
    if op == "accept":
        moved = sum(int(a) - 1 for a in case["accepted"].split(","))
        return {"bytes": 12 * T + moved * case["n_layer"] * 2 * Hkv * hd * 2 * 2, "flops": 10 * T}
    H, W = case["H"], case["window"]
    size = 2 if case["kv"] == "f16" else 1
    # a tree's depth is about twice the logarithm of its size: its rows see that many of their own cells
    own_cells = [min(n, 2 * math.log(n) + 1) for _, n in trees]
    keys = sum(min(a, W or a) + n for a, n in trees)
    seen = sum(n * (min(a, W or a) + d) for (a, n), d in zip(trees, own_cells))
    return {"bytes": keys * Hkv * hd * 2 * size + 4 * T * H * hd, "flops": 4 * H * hd * seen}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "table":
        p = torch.arange(s["pos0"], s["pos0"] + case["n_pos"], device="cuda").double()
        z = torch.polar(torch.tensor(s["m"], dtype=torch.float64, device="cuda").expand(case["n_pos"], len(s["f"])).contiguous(),
                        torch.outer(p, torch.tensor(s["f"], dtype=torch.float64, device="cuda")))
        return torch.view_as_real(z)
    Hkv, hd, n_ctx = case["Hkv"], case["hd"], case["n_ctx"]
    if op == "rope":
        T, H, n = case["T"], case["H"], case["n_rot"]
        heads = s["qkv"].double().view(T, H + 2 * Hkv, hd)
        spin = torch.view_as_complex(s["table"].double())[s["pos"].long()].view(T, 1, n // 2)
        res = []
        for part, gain in ((heads[:, :H], s["q_gain"]), (heads[:, H:H + Hkv], s["k_gain"])):
            part = part.clone()
            if gain is not None:
                part = part / ((part * part).sum(-1, keepdim=True) / hd + EPS).sqrt() * gain.double()
            even, odd = (slice(0, n, 2), slice(1, n, 2)) if case["layout"] == "pairs" else (slice(0, n // 2), slice(n // 2, n))
            z = torch.complex(part[..., even], part[..., odd]) * spin
            part[..., even], part[..., odd] = z.real, z.imag
            res.append(part)
        caches = []
        for rows in (res[1], heads[:, H + Hkv:]):
            full = torch.zeros((case["n_seq"], Hkv, n_ctx, hd), dtype=torch.float64, device="cuda")
            full[s["seq"].long(), :, s["cell"].long()] = rows
            caches.append(full)
        return (res[0].reshape(T, -1), *caches)
    trees, first = _trees(case), s["row0_host"]
    if op == "accept":
        kc, vc = s["kc"].double(), s["vc"].double()
        token, parent, target = (s[k].tolist() for k in ("token", "parent", "target"))
        paths, counts, nexts = [], [], []
        for i, (base, n) in enumerate(trees):
            r, cur, path = first[i], 0, [0]
            while True:
                kids = [j for j in range(1, n) if parent[r + j] == cur and token[r + j] == target[r + cur]]
                if not kids:
                    break
                cur = kids[0]
                path.append(cur)
            for cache in (kc, vc):
                held = cache[len(trees) - 1 - i]
                held[:, :, base:base + len(path)] = held[:, :, [base + j for j in path]].clone()
            paths.append(path + [-1] * (s["most"] - len(path)))
            counts.append(len(path))
            nexts.append(target[r + cur])
        return _ints(paths), _ints(counts), _ints(nexts), kc, vc
    H = case["H"]
    o = torch.zeros((s["T"], H, hd), dtype=torch.float64, device="cuda")
    q = s["q"].double().view(s["T"], H, hd)
    mask = s["mask"].cpu().long() & 0xffffffff
    for i, (base, n) in enumerate(trees):
        at, end, r = len(trees) - 1 - i, base + n, first[i]
        hidden = torch.zeros((n, end), dtype=torch.bool)
        for j in range(n):
            hidden[:, base + j] = (mask[r:r + n, j // 32] >> (j % 32)) % 2 == 0
        if case["window"]:
            low = s["pos"][r:r + n].cpu().long() - case["window"]
            hidden[:, :base] |= torch.arange(base)[None] <= low[:, None]
        blind = hidden.all(1).cuda()
        hidden = hidden.cuda()
        for h in range(H):
            k, v = (s[x][at, h // (H // Hkv), :end].double() for x in ("kc", "vc"))
            w = torch.softmax((q[r:r + n, h] @ k.T * hd ** -0.5).masked_fill(hidden, -math.inf), -1)
            o[r:r + n, h] = torch.where(blind[:, None], torch.zeros_like(w[:, :1]), w @ v)
    return o.view(s["T"], H * hd)
