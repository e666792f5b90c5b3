"""Trees of drafted tokens and the operators' definitions in 64 bits, for the tests."""
import numpy as np


def parents(rng, n, kind="random"):
    """Each node's parent, -1 for node 0."""
    if kind == "chain":
        return np.arange(-1, n - 1)
    if kind == "star":
        return np.array([-1] + [0] * (n - 1))
    return np.array([-1] + [int(rng.integers(0, i)) for i in range(1, n)])


def depths(parent):
    d = np.zeros(len(parent), np.int64)
    for i, p in enumerate(parent):
        d[i] = 0 if p < 0 else d[p] + 1
    return d


def ancestors(parent):
    """Boolean [n][n]: row i sees node j."""
    n = len(parent)
    m = np.zeros((n, n), bool)
    for i, p in enumerate(parent):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def pack_mask(seen, max_nodes):
    """Boolean [n][up to max_nodes] -> uint32 words [n][ceil(max_nodes / 32)]."""
    words = (max_nodes + 31) // 32
    full = np.zeros((len(seen), words * 32), bool)
    full[:, :seen.shape[1]] = seen
    w = (full.reshape(len(seen), words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32)


def frequencies(theta, n_rot, scaling, factor=1.0, slow=1.0, fast=4.0, orig=1, attn=0.0):
    """Radians a position of each pair and the factor of cos and sin (scaling as LLM_ROPE_*)."""
    j = np.arange(n_rot // 2, dtype=np.float64)
    f = np.float64(theta) ** (-2 * j / n_rot)
    keep = np.ones_like(f)
    if scaling == 1:
        keep = np.zeros_like(f)
    if scaling == 2:
        keep = (orig * f / (2 * np.pi) - slow) / (fast - slow)
    if scaling == 3:
        def pair(turns):
            return n_rot * np.log(orig / (turns * 2 * np.pi)) / (2 * np.log(theta))
        lo, hi = max(np.floor(pair(fast)), 0), min(np.ceil(pair(slow)), n_rot - 1)
        keep = 1 - (j - lo) / max(hi - lo, 0.001)
    keep = np.clip(keep, 0, 1)
    m = attn if attn > 0 else 0.1 * np.log(factor) + 1 if scaling == 3 else 1.0
    return f * keep + f / factor * (1 - keep), m


def rotate(x, cs, n_rot, layout):
    """x [T][heads][hd] turned by cs [T][n_rot / 2][2]; layout as LLM_ROPE_*."""
    x = x.copy()
    a, b = (slice(0, n_rot, 2), slice(1, n_rot, 2)) if layout == 0 else (slice(0, n_rot // 2), slice(n_rot // 2, n_rot))
    z = (x[..., a] + 1j * x[..., b]) * (cs[..., 0] + 1j * cs[..., 1])[:, None]
    x[..., a], x[..., b] = z.real, z.imag
    return x


def attention(q, k, v, base, seen, pos, window):
    """One tree: q [n][H][hd], k, v [Hkv][cells][hd] (float64), seen [n][n].
    Returns o, and per element the weighted sum of |v|, and per head the largest
    root of the sum of (q k)^2 over a visible cell."""
    n, H, hd = q.shape
    G = H // k.shape[0]
    end = base + n
    vis = np.zeros((n, end), bool)
    vis[:, :base] = True
    if window:
        vis[:, :base] &= np.arange(base)[None] > np.asarray(pos)[:, None] - window
    vis[:, base:] = seen[:, :n]
    o, mag, size = np.zeros((n, H, hd)), np.zeros((n, H, hd)), np.zeros((n, H))
    for h in range(H):
        K, V = k[h // G, :end], v[h // G, :end]
        for t in range(n):
            w = vis[t]
            if not w.any():
                continue
            s = K[w] @ q[t, h] / np.sqrt(hd)
            p = np.exp(s - s.max())
            p /= p.sum()
            o[t, h], mag[t, h] = p @ V[w], p @ np.abs(V[w])
            size[t, h] = np.sqrt(((K[w] * q[t, h]) ** 2).sum(-1)).max()
    return o, mag, size


def accept(token, parent, target):
    """Nodes that stand and the next token."""
    path = [0]
    while True:
        kids = [j for j in range(1, len(token)) if parent[j] == path[-1] and token[j] == target[path[-1]]]
        if not kids:
            return path, target[path[-1]]
        path.append(kids[0])
