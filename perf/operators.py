"""Timed cases of the 4-bit operators: products with 4-bit weights, the per-head
norm and rotation of queries and keys with the append to the cache, and the
attention over a cache held in 4 bits.

Q4_0: a row is cut into blocks of 32 elements; a block keeps an fp16 scale d
and 32 codes c in 0..15 and stands for d * (c - 8).  Codes are held in 32-bit
words of eight: in a group of nb blocks (a cache row of 32 nb elements, or 128
consecutive elements of a weight row), word t * nb + b, t = 0..3, holds the
elements 32 b + 8 t + {0..7}, element 8 t + 2 i in bits 4 i.. and element
8 t + 2 i + 1 in bits 16 + 4 i..  A weight row is chunks of 256 elements: two
groups of 128 (64 bytes each), then the eight scales (144 bytes).  A cache of
one layer is the codes [n_seq][Hkv][n_ctx][hd / 2 bytes], then the scales
[n_seq][Hkv][n_ctx][hd / 32] as fp16.

A case's "op":
  gemv     y[t][n] = sum_k W[n][k] x[t][k], W in Q4_0, x fp16, y fp32
  qk       rows of q, k, v heads: q and k normed per head (where "norm"), rotated
           by position; q out, k and v appended to an fp16 or a Q4_0 cache
  decode   attention of single new tokens over their sequences' Q4_0 caches
  prefill  attention of runs of new tokens over their sequences' Q4_0 caches
"""
import math

import torch

own = False

BLOCK = 32
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
        # the output projection of the ~1B shape for one token: launch and latency count
        {"name": "gemv 2048x2048 T1", "op": "gemv", "N": 2048, "K": 2048, "T": 1},
        # the output projection of the 8B shape for one token
        {"name": "gemv 4096x4096 T1", "op": "gemv", "N": 4096, "K": 4096, "T": 1},
        # gate and up of the 8B shape for one token
        {"name": "gemv 28672x4096 T1", "op": "gemv", "N": 28672, "K": 4096, "T": 1},
        # the down projection of the 8B shape for a step of eight sequences
        {"name": "gemv 4096x14336 T8", "op": "gemv", "N": 4096, "K": 14336, "T": 8},
        # the vocabulary projection of the 8B shape
        {"name": "gemv 128256x4096 T1", "op": "gemv", "N": 128256, "K": 4096, "T": 1},
        # a decode step of three sequences with normed queries and keys
        {"name": "qk T3 f16", "op": "qk", "T": 3, "H": 32, "Hkv": 8, "hd": 128, "n_seq": 4, "n_ctx": 8192,
         "kv": "f16", "norm": True},
        # a long prompt's rows at once, fp16 cache
        {"name": "qk T4096 f16", "op": "qk", "T": 4096, "H": 32, "Hkv": 8, "hd": 128, "n_seq": 1, "n_ctx": 4608,
         "kv": "f16", "norm": True},
        # one ubatch of the ~1B shape into a 4-bit cache, and those rows read back
        {"name": "qk T512 q4 hd64", "op": "qk", "T": 512, "H": 32, "Hkv": 8, "hd": 64, "n_seq": 1, "n_ctx": 4096,
         "kv": "q4", "norm": True},
        # one new token of the 8B shape behind a 2048-token prompt
        {"name": "decode 2100", "op": "decode", "H": 32, "Hkv": 8, "hd": 128, "n_ctx": 4096, "lens": "2100",
         "window": 0},
        # one new token of the 8B shape in a 32k context
        {"name": "decode 32000", "op": "decode", "H": 32, "Hkv": 8, "hd": 128, "n_ctx": 32768, "lens": "32000",
         "window": 0},
        # eight sequences of different lengths, a token each
        {"name": "decode 8 ragged", "op": "decode", "H": 32, "Hkv": 8, "hd": 128, "n_ctx": 8192,
         "lens": "1882,1582,2911,3415,2775,2634,1781,748", "window": 0},
        # the last ubatch of a 2048-token prompt of the 8B shape
        {"name": "prefill 512 of 2048", "op": "prefill", "H": 32, "Hkv": 8, "hd": 128, "n_ctx": 4096,
         "runs": "1536+512", "window": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(32, 8), (16, 8), (8, 1), (8, 8), (40, 8), (12, 4), (6, 2)])


def draw(rng):
    op = rng.choice(["gemv", "gemv", "qk", "decode", "decode", "prefill"])
    if op == "gemv":
        K = 256 * _log(rng, 1, 64)
        return {"op": op, "N": min(_log(rng, 50, 130000), 500_000_000 // K), "K": K, "T": rng.randint(1, 8)}
    H, Hkv = _heads(rng)
    hd = rng.choice([32, 64, 128, 128])
    if op == "qk":
        T = _log(rng, 1, 3000)
        n_seq = rng.randint(1, 3)
        return {"op": op, "T": T, "H": H, "Hkv": Hkv, "hd": hd, "n_seq": n_seq, "n_ctx": T + rng.randint(1, 500),
                "kv": rng.choice(["f16", "q4"]), "norm": rng.random() < 0.7}
    if op == "decode":
        n = rng.randint(1, 8)
        lens = [_log(rng, 1, 30000 if n == 1 else 6000) for _ in range(n)]
        return {"op": op, "H": H, "Hkv": Hkv, "hd": hd, "n_ctx": max(lens) + rng.randint(0, 300),
                "lens": ",".join(map(str, lens)), "window": rng.choice([0, 0, _log(rng, 1, 4000)])}
    runs = [(rng.choice([0, _log(rng, 1, 1500)]), _log(rng, 9, 400)) for _ in range(rng.randint(1, 3))]
    return {"op": op, "H": H, "Hkv": Hkv, "hd": hd, "n_ctx": max(a + b for a, b in runs) + rng.randint(0, 200),
            "runs": ",".join("%d+%d" % r for r in runs), "window": rng.choice([0, 0, _log(rng, 1, 1000)])}


# ------------------------------------------------------------------ inputs

def _rand(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale


def _encode(v):
    """Codes (int64, [..., blocks, 32]) and fp32 scales of values [..., n]."""
    v = v.unflatten(-1, (-1, BLOCK))
    top = v.abs().argmax(-1, keepdim=True)
    d = v.gather(-1, top) / -8
    c = torch.where(d != 0, torch.round(v / torch.where(d != 0, d, torch.ones_like(d))) + 8, torch.full_like(v, 8))
    return c.clamp_(0, 15), d[..., 0]


def _pack(c):
    """Codes [..., nb, 32] of one group as its 16 nb bytes."""
    c = c.to(torch.uint8).unflatten(-1, (4, 2, 2, 2))               # [..., b, t, i/2, i%2, odd]
    byte = c[..., 0, :] | (c[..., 1, :] << 4)                       # [..., b, t, i/2, odd]
    return byte.movedim(-4, -3).transpose(-1, -2).flatten(-4)       # [..., t, b, odd, i/2]


def _unpack(b, nb):
    """The codes [..., nb, 32] of a group's bytes, as fp32."""
    b = b.unflatten(-1, (4, nb, 2, 2))                              # [..., t, b, odd, i/2]
    c = torch.stack((b & 15, b >> 4), -1)                           # [..., t, b, odd, i/2, i%2]
    return c.movedim(-3, -1).transpose(-5, -4).flatten(-4).float()  # [..., b, (t, i/2, i%2, odd)]


def _cache(vals):
    """A cache's bytes for values [n_seq][Hkv][n_ctx][hd]."""
    c, d = _encode(vals)
    return torch.cat((_pack(c).reshape(-1), d.to(torch.float16).reshape(-1).view(torch.uint8)))


def _ints(s):
    return [int(x) for x in s.split(",")]


def _table(n_ctx, hd):
    """cos and sin of pos * 10000^(-2 i / hd), from 64 bits."""
    a = torch.arange(n_ctx, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, hd, 2, dtype=torch.float64) / hd)
    return torch.stack((a.cos(), a.sin()), -1).to(torch.float32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op == "gemv":
        N, K, T = case["N"], case["K"], case["T"]
        W = torch.empty((N, K // 16 * 9), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 26) // K)
        for r in range(0, N, step):
            c, d = _encode(_rand((min(step, N - r), K), g, 0.02))
            codes = _pack(c.unflatten(-2, (-1, 4)))                               # [rows][K / 128][64]
            W[r:r + step].unflatten(-1, (-1, 144))[..., :128] = codes.flatten(-2).unflatten(-1, (-1, 128))
            W[r:r + step].unflatten(-1, (-1, 144))[..., 128:] = (
                d.to(torch.float16).view(torch.uint8).unflatten(-1, (-1, 16)))
        x = _rand((T, K), g).to(torch.float16)
        y = torch.empty((T, N), device="cuda")
        s.update(W=W, x=x, y=y, args=(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, T, K, N))
        return s
    H, Hkv, hd, n_ctx = case["H"], case["Hkv"], case["hd"], case["n_ctx"]
    if op == "qk":
        T, n_seq = case["T"], case["n_seq"]
        qkv = _rand((T, (H + 2 * Hkv) * hd), g, 1.3)
        gains = [1 + _rand((hd,), g, 0.1) if case["norm"] else None for _ in range(2)]
        # runs of consecutive positions, one run for each sequence
        own_of = torch.arange(T) * n_seq // T
        first = torch.tensor([int((own_of == i).nonzero()[0]) if (own_of == i).any() else 0 for i in range(n_seq)])
        base = int(torch.randint(0, n_ctx - T + 1, (1,), generator=g, device="cuda"))
        pos = (torch.arange(T) - first[own_of] + base).to(torch.int32).cuda()
        seq = own_of.to(torch.int32).cuda()
        q = torch.empty((T, H * hd), dtype=torch.float16 if T > 8 else torch.float32, device="cuda")
        rows = n_seq * Hkv * n_ctx
        if case["kv"] == "f16":
            kc, vc = (torch.zeros((n_seq, Hkv, n_ctx, hd), dtype=torch.float16, device="cuda") for _ in range(2))
        else:
            kc, vc = (torch.zeros(rows * (hd // 2 + hd // 16), dtype=torch.uint8, device="cuda") for _ in range(2))
        s.update(qkv=qkv, q_gain=gains[0], k_gain=gains[1], pos=pos, seq=seq, q=q, kc=kc, vc=vc, rope=_table(n_ctx, hd),
                 k_rows=torch.empty((T, Hkv, hd), dtype=torch.float16, device="cuda"),
                 v_rows=torch.empty((T, Hkv, hd), dtype=torch.float16, device="cuda"),
                 err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        p = [0 if v is None else v.data_ptr() for v in (s["qkv"], s["q_gain"], s["k_gain"], s["rope"], pos, seq, q,
                                                        kc, vc, s["k_rows"], s["v_rows"], s["err"])]
        s["args"] = (p[0], (H + 2 * Hkv) * hd, p[1], p[2], EPS, p[3], p[4], p[5], p[6], int(T > 8), p[7], p[8],
                     2 if case["kv"] == "q4" else 0, T, H, Hkv, hd, n_ctx, n_seq, p[11])
        s["k_args"] = (p[7], p[4], p[5], p[9], T, Hkv, hd, n_ctx, n_seq, p[11])
        s["v_args"] = (p[8], p[4], p[5], p[10], T, Hkv, hd, n_ctx, n_seq, p[11])
        return s
    if op == "decode":
        lens = _ints(case["lens"])
        T = n_seq = len(lens)
        pos, seq = torch.tensor(lens, dtype=torch.int32) - 1, torch.arange(T, dtype=torch.int32)
        q = _rand((T, H * hd), g, 1.5)
    else:
        runs = [tuple(map(int, r.split("+"))) for r in case["runs"].split(",")]
        n_seq = len(runs)
        pos = torch.cat([torch.arange(a, a + b, dtype=torch.int32) for a, b in runs])
        seq = torch.cat([torch.full((b,), i, dtype=torch.int32) for i, (a, b) in enumerate(runs)])
        T = len(pos)
        q = _rand((T, H * hd), g, 1.5).to(torch.float16)
    kc, vc = (_cache(_rand((n_seq, Hkv, n_ctx, hd), g)) for _ in range(2))
    o = torch.empty((T, H * hd), dtype=torch.float16, device="cuda")
    s.update(q=q, kc=kc, vc=vc, pos=pos.cuda(), seq=seq.cuda(), pos_host=pos, seq_host=seq, o=o, scratch=None,
             err=torch.zeros(1, dtype=torch.int32, device="cuda"), n_seq=n_seq, T=T)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return _PLAIN[state["op"]](state, state["case"])


def _run_own(s):
    L = _lib()
    op, c = s["op"], s["case"]
    if op == "gemv":
        L.check(L.llm_op_gemv_q4_0(*s["args"], _stream()))
        return s["y"]
    if op == "qk":
        st = _stream()
        L.check(L.llm_op_qk_norm_rope(*s["args"], st))
        if c["kv"] == "f16":
            return s["q"], s["kc"], s["vc"]
        L.check(L.llm_op_kv_rows_q4_0(*s["k_args"], st))
        L.check(L.llm_op_kv_rows_q4_0(*s["v_args"], st))
        return s["q"], s["k_rows"], s["v_rows"]
    if s["scratch"] is None:                                        # the workspace such a program keeps
        size = L.llm_op_attn_decode_q4_0_scratch_bytes if op == "decode" else L.llm_op_attn_prefill_q4_0_scratch_bytes
        s["scratch"] = torch.zeros(size(s["T"], c["H"], c["Hkv"], c["hd"], c["n_ctx"], s["n_seq"]), dtype=torch.uint8,
                                   device="cuda")
        where = (s["pos"], s["seq"]) if op == "decode" else (s["pos_host"], s["seq_host"])
        s["args"] = (s["q"].data_ptr(), s["kc"].data_ptr(), s["vc"].data_ptr(), where[0].data_ptr(),
                     where[1].data_ptr(), s["o"].data_ptr(), s["T"], c["H"], c["Hkv"], c["hd"], c["n_ctx"], s["n_seq"],
                     c["window"], s["scratch"].data_ptr(), s["scratch"].numel(), s["err"].data_ptr())
    call = L.llm_op_attn_decode_q4_0 if op == "decode" else L.llm_op_attn_prefill_q4_0
    L.check(call(*s["args"], _stream()))
    return s["o"]


def _plain_gemv(s, c):
    W = s["W"].unflatten(-1, (-1, 144))                             # [N][K / 256][144]
    codes = _unpack(W[..., :128].unflatten(-1, (2, 64)), 4) - 8     # [N][K / 256][2][4][32]
    d = W[..., 128:].contiguous().view(torch.float16).float().unflatten(-1, (2, 4))
    return s["x"].float() @ (codes * d[..., None]).flatten(1).T


def _rotate(v, cs):
    """Pairs (2 i, 2 i + 1) of v [T][heads][hd] turned by the table's rows cs [T][hd / 2][2]."""
    a, b = v[..., 0::2], v[..., 1::2]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)


def _plain_qk(s, c):
    H, Hkv, hd, T = c["H"], c["Hkv"], c["hd"], c["T"]
    q4 = c["kv"] == "q4"
    x = s["qkv"].unflatten(-1, (-1, hd))
    x = x.double() if q4 else x                                     # codes: values next to a border
    cs = s["rope"][s["pos"].long()].to(x.dtype)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_gain"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_gain"]
    q, k = _rotate(q, cs), _rotate(k, cs)
    q = q.flatten(1).to(s["q"].dtype)
    if q4:
        out = []
        for u in (k, v):
            code, d = _encode(u)
            out.append(((code - 8) * d.to(torch.float16).to(u.dtype)[..., None]).flatten(-2).to(torch.float16))
        return q, out[0], out[1]
    at = (s["seq"].long(), slice(None), s["pos"].long())
    s["kc"][at] = k.to(torch.float16)
    s["vc"][at] = v.to(torch.float16)
    return q, s["kc"], s["vc"]


def _values(cache, n_seq, c):
    """The values [n_seq][Hkv][n_ctx][hd] a cache stands for, fp32."""
    hd = c["hd"]
    n = n_seq * c["Hkv"] * c["n_ctx"]
    codes = _unpack(cache[:n * hd // 2].view(n, hd // 2), hd // 32) - 8
    d = cache[n * hd // 2:].view(torch.float16).float().view(n, hd // 32, 1)
    return (codes * d).view(n_seq, c["Hkv"], c["n_ctx"], hd)


def _softmax(s, seen):
    s = s.masked_fill(~seen, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_decode(s, c):
    T, H, Hkv, hd = s["T"], c["H"], c["Hkv"], c["hd"]
    seq, pos = s["seq"].long(), s["pos"].long()
    k, v = (_values(s[n], s["n_seq"], c)[seq] for n in ("kc", "vc"))            # [T][Hkv][n_ctx][hd]
    q = s["q"].view(T, Hkv, H // Hkv, hd) / math.sqrt(hd)
    key = torch.arange(c["n_ctx"], device="cuda")
    seen = (key <= pos[:, None]) & (key > pos[:, None] - (c["window"] or c["n_ctx"] + 1))
    p = _softmax(q @ k.transpose(-1, -2), seen[:, None, None])
    return (p @ v).flatten(1).to(torch.float16)


def _plain_prefill(s, c):
    T, H, Hkv, hd, n_seq, n_ctx = s["T"], c["H"], c["Hkv"], c["hd"], s["n_seq"], c["n_ctx"]
    k, v = (_values(s[n], n_seq, c).transpose(0, 1).flatten(1, 2) for n in ("kc", "vc"))   # [Hkv][n_seq n_ctx][hd]
    q = s["q"].float().view(T, Hkv, H // Hkv, hd).permute(1, 2, 0, 3) / math.sqrt(hd)      # [Hkv][G][T][hd]
    cell = torch.arange(n_seq * n_ctx, device="cuda")
    key, of = cell % n_ctx, cell // n_ctx
    pos, seq = s["pos"].long()[:, None], s["seq"].long()[:, None]
    seen = (of == seq) & (key <= pos) & (key > pos - (c["window"] or n_ctx + 1))
    p = _softmax(q @ k[:, None].transpose(-1, -2), seen)
    return (p @ v[:, None]).permute(2, 0, 1, 3).flatten(1).to(torch.float16)


_PLAIN = {"gemv": _plain_gemv, "qk": _plain_qk, "decode": _plain_decode, "prefill": _plain_prefill}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "gemv":
        N, K, T = case["N"], case["K"], case["T"]
        return {"bytes": N * K * 9 / 16 + 2 * T * K + 4 * T * N, "flops": 2 * N * K * T}
    H, Hkv, hd = case["H"], case["Hkv"], case["hd"]
    if op == "qk":
        T = case["T"]
        kv = 2 * T * Hkv * hd
        b = 4 * T * (H + 2 * Hkv) * hd + T * H * hd * (2 if T > 8 else 4) + 4 * hd * T
        b += kv * 2 if case["kv"] == "f16" else kv * (2 * 9 / 16 + 2)
        return {"bytes": b, "flops": T * (H + Hkv) * hd * 8}
    W = case["window"]
    if op == "decode":
        T = len(_ints(case["lens"]))
        seen = sum(min(n, W or n) for n in _ints(case["lens"]))
        return {"bytes": seen * Hkv * hd * 2 * 9 / 16 + 6 * T * H * hd, "flops": 4 * H * hd * seen}
    runs = [tuple(map(int, r.split("+"))) for r in case["runs"].split(",")]
    T = sum(b for _, b in runs)
    rows = sum(min(a + b, W + b - 1 if W else a + b) for a, b in runs)
    seen = sum(min(p + 1, W or p + 1) for a, b in runs for p in range(a, a + b))
    return {"bytes": rows * Hkv * hd * 2 * 9 / 16 + 4 * T * H * hd, "flops": 4 * H * hd * seen}


# ------------------------------------------------------------------ the definition in 64 bits

def _place(nb):
    """For element e of a group: its word and the bits its code starts at."""
    e = torch.arange(32 * nb)
    b, r = e // 32, e % 32
    t, i, odd = r // 8, r % 8 // 2, r % 2
    return (t * nb + b).cuda(), (4 * i + 16 * odd).cuda()


def _decoded(words, scales, nb):
    """Values in 64 bits of groups of words [n][4 nb] (int32) with scales [n][nb]."""
    at, shift = _place(nb)
    code = (words.long()[:, at] >> shift) & 15
    return (code - 8).double() * scales.double().repeat_interleave(32, 1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "gemv":
        N, K, T = case["N"], case["K"], case["T"]
        y = torch.empty((T, N), dtype=torch.float64, device="cuda")
        step = max(1, (1 << 25) // K)
        for r in range(0, N, step):
            chunk = s["W"][r:r + step].reshape(-1, 144)
            words = chunk[:, :128].contiguous().view(torch.int32).view(-1, 16)
            scale = chunk[:, 128:].contiguous().view(torch.float16).view(-1, 4)
            y[:, r:r + step] = s["x"].double() @ _decoded(words, scale, 4).view(-1, K).T
        return y
    H, Hkv, hd, n_ctx = case["H"], case["Hkv"], case["hd"], case["n_ctx"]
    if op == "qk":
        T = case["T"]
        heads = s["qkv"].double().view(T, H + 2 * Hkv, hd)
        turn = s["rope"].double()[s["pos"].long()].view(T, 1, hd // 2, 2)
        turn = torch.view_as_complex(turn.contiguous())
        res = []
        for part, gain in ((heads[:, :H], s["q_gain"]), (heads[:, H:H + Hkv], s["k_gain"])):
            if gain is not None:
                part = part / ((part * part).sum(-1, keepdim=True) / hd + EPS).sqrt() * gain.double()
            z = torch.view_as_complex(part.reshape(T, -1, hd // 2, 2).contiguous()) * turn
            res.append(torch.view_as_real(z).reshape(T, -1, hd))
        res.append(heads[:, H + Hkv:])
        q, rows = res[0].reshape(T, -1), res[1:]
        if case["kv"] == "f16":
            caches = []
            for r in rows:
                full = torch.zeros((case["n_seq"], Hkv, n_ctx, hd), dtype=torch.float64, device="cuda")
                full[s["seq"].long(), :, s["pos"].long()] = r
                caches.append(full)
            return (q, *caches)
        held = []
        for r in rows:
            blk = r.reshape(-1, 32)
            hi, lo = blk.max(1).values, blk.min(1).values
            # the element of largest magnitude with its sign; of two the first
            tie = (hi == -lo) & (hi > 0)
            lead = torch.where((blk == hi[:, None]).long().argmax(1) < (blk == lo[:, None]).long().argmax(1), hi, lo)
            m = torch.where(tie, lead, torch.where(hi > -lo, hi, lo))
            level = torch.round(blk * -8 / torch.where(m == 0, 1, m)[:, None]).clamp(-8, 7)
            held.append((level * (m / -8).half().double()[:, None]).view(T, Hkv, hd))
        return (q, *held)
    n = s["n_seq"] * Hkv * n_ctx
    o = torch.empty((s["T"], H, hd), dtype=torch.float64, device="cuda")
    k, v = (_decoded(s[c][:n * hd // 2].view(torch.int32).view(n, hd // 8), s[c][n * hd // 2:].view(torch.float16).view(
        n, hd // 32), hd // 32).view(s["n_seq"], Hkv, n_ctx, hd) for c in ("kc", "vc"))
    q = s["q"].double().view(s["T"], Hkv, H // Hkv, hd)
    # a run of rows of one sequence at a time, each row over its own keys
    start = [i for i in range(s["T"]) if i == 0 or s["seq_host"][i] != s["seq_host"][i - 1]] + [s["T"]]
    for i, j in zip(start, start[1:]):
        at, p = int(s["seq_host"][i]), s["pos_host"][i:j].long().cuda()
        end = int(p[-1]) + 1
        hidden = torch.arange(end, device="cuda")[None] > p[:, None]
        if case["window"]:
            hidden |= torch.arange(end, device="cuda")[None] <= p[:, None] - case["window"]
        for h in range(Hkv):
            score = torch.einsum("tgd,kd->gtk", q[i:j, h], k[at, h, :end]) * hd ** -0.5
            weight = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            o[i:j, h * (H // Hkv):(h + 1) * (H // Hkv)] = torch.einsum("gtk,kd->tgd", weight, v[at, h, :end])
    return o.view(s["T"], H * hd)
