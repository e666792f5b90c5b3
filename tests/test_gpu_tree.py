"""The operators of drafted decoding on the GPU against their definitions in 64
bits: rotary tables, the rotation in every layout with the append to the cache,
attention of trees of drafted tokens, and the acceptance of a tree's path.

Tolerances.  An fp16 output is off by half a step, 2^-11 of it (2^-25 below
fp16's smallest normal).  What the fp32 arithmetic before it adds:
  rotation: a norm, two products and a sum, below 12 roundings of 2^-24 of the
      products' magnitudes;
  attention: a score is a sum of hd products, whose partial sums are about
      R = sqrt(sum (q k)^2) large, so its rounding and truncation errors (2^-23 of
      a partial sum each, adding like a random walk) are about sqrt(hd) 2^-23 R,
      2^-23 R after the division by sqrt(hd); eight times that, 2^-20 R, bounds the
      exponent's error, and with it the weights' relative one; 2^-19 more for the
      weights' 22 bits, the exponential and the sums.  Both are relative to the
      weighted sum of |V|."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import tree_util as U
from oracle import llama as O
from q4_util import unpack_cache

pytestmark = pytest.mark.gpu
U16, TINY16 = 2.0 ** -11, 2.0 ** -25


@pytest.fixture(scope="module")
def lib():
    import llama_decoder_forward_02_gb300 as L
    return L


def stream():
    return torch.cuda.current_stream().cuda_stream


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32).cuda()


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- rotary tables

@pytest.mark.parametrize("scaling,n_rot,theta,factor,orig,pos0,n_pos", [
    (0, 128, 500000.0, 1.0, 0, 0, 4096),
    (0, 8, 10000.0, 1.0, 0, 7, 1),
    (1, 64, 10000.0, 4.0, 0, 100, 333),
    (2, 128, 500000.0, 8.0, 8192, 0, 1025),
    (2, 88, 1e6, 2.0, 2048, 99999, 777),
    (3, 128, 10000.0, 32.0, 4096, 131000, 501),
    (3, 64, 500000.0, 1.0, 32768, 0, 63),
    (3, 24, 10000.0, 8.0, 2, 0, 300),          # a context so short that the ramp's ends cross
    (0, 128, 1e7, 1.0, 0, (1 << 30) - 40, 40),
])
def test_table(lib, scaling, n_rot, theta, factor, orig, pos0, n_pos):
    fast = 4.0 if scaling == 2 else 32.0
    r = lib.rope(theta, n_rot, scaling=scaling, factor=factor, n_ctx_orig=orig)
    out = torch.full((n_pos * n_rot + 64,), 7.0, device="cuda")
    assert lib.llm_op_rope_table(r, pos0, n_pos, out.data_ptr(), stream()) == 0
    got = out.cpu().double().numpy()
    assert np.all(got[-64:] == 7.0)
    f, m = U.frequencies(np.float32(theta).astype(np.float64), n_rot, scaling, factor, 1.0, fast, orig)
    a = np.arange(pos0, pos0 + n_pos, dtype=np.float64)[:, None] * f
    ref = np.stack((np.cos(a) * m, np.sin(a) * m), -1)
    # two roundings of 2^-24, the polynomial around the nearest of 512 directions good to 2^-30, the angle itself to
    # 2^-53 of its size in both
    tol = 2.0 ** -23 * np.abs(ref) + m * (2.0 ** -30 + np.abs(a)[..., None] * 2.0 ** -52)
    assert np.all(np.abs(got[:-64].reshape(ref.shape) - ref) <= tol)


def test_table_factor(lib):
    r = lib.rope(10000.0, 64, scaling=3, factor=4.0, n_ctx_orig=1024, attn_factor=0.5)
    out = torch.empty((10, 32, 2), device="cuda")
    assert lib.llm_op_rope_table(r, 0, 10, out.data_ptr(), stream()) == 0
    assert torch.all(out[0, :, 0] == 0.5) and torch.all(out[0, :, 1] == 0)


# ---------------------------------------------------------------- rotation and append

@pytest.mark.parametrize("kt", [0, 1, 2])
@pytest.mark.parametrize("hd,H,Hkv,T,n_rot,layout,norm,qt,pad", [
    (128, 4, 2, 9, 128, 1, True, 1, 0),
    (128, 4, 1, 5, 64, 1, False, 0, 4),
    (128, 2, 2, 33, 24, 1, True, 1, 0),          # halves of 12: partners lie across lanes
    (128, 6, 2, 17, 40, 0, True, 1, 0),
    (64, 8, 2, 7, 64, 1, True, 1, 8),
    (64, 4, 4, 700, 32, 1, False, 1, 0),         # one CTA a row
    (64, 4, 4, 3, 8, 1, True, 0, 0),
    (64, 2, 1, 3, 56, 0, False, 1, 0),
    (32, 3, 1, 13, 32, 1, False, 1, 0),
    (32, 4, 2, 1, 16, 1, True, 1, 0),
    (32, 4, 2, 2, 24, 0, True, 1, 0),
])
def test_rope_kv(lib, hd, H, Hkv, T, n_rot, layout, norm, qt, pad, kt):
    rng = np.random.default_rng(T * hd + n_rot + layout)
    n_ctx, n_seq, n_pos, eps = T + 20, 2, T + 7, 1e-5
    ld = (H + 2 * Hkv) * hd + pad
    x = (rng.standard_normal((T, ld)) * 1.3).astype(np.float32)
    gains = [(1 + 0.1 * rng.standard_normal(hd)).astype(np.float32) if norm else None for _ in range(2)]
    f, _ = U.frequencies(10000.0, n_rot, 0)
    a = np.arange(n_pos)[:, None] * f
    tab = np.stack((np.cos(a), np.sin(a)), -1).astype(np.float32)
    pos = rng.integers(0, n_pos, T)                  # several rows share one
    cell = rng.permutation(n_ctx)[:T]
    seq = rng.integers(0, n_seq, T)
    q = torch.full((T, H * hd), 5.0, dtype=torch.float32 if qt == 0 else torch.float16, device="cuda")
    rows = n_seq * Hkv * n_ctx
    size = rows * {0: 2 * hd, 1: hd, 2: hd // 2 + hd // 16}[kt]
    caches = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    X, G, TB, P, C, S, E = dev(x), [None if g is None else dev(g) for g in gains], dev(tab), ints(pos), ints(cell), ints(seq), err_word()
    args = [X.data_ptr(), ld, *(0 if g is None else g.data_ptr() for g in G), eps, TB.data_ptr(), n_pos, n_rot, layout,
            P.data_ptr(), C.data_ptr(), S.data_ptr(), q.data_ptr(), qt, caches[0].data_ptr(), caches[1].data_ptr(), kt, T,
            H, Hkv, hd, n_ctx, n_seq, E.data_ptr(), stream()]
    assert lib.llm_op_rope_kv(*args) == 0
    assert int(E) == 0
    heads = x[:, :(H + 2 * Hkv) * hd].astype(np.float64).reshape(T, H + 2 * Hkv, hd)
    parts = [heads[:, :H], heads[:, H:H + Hkv], heads[:, H + Hkv:]]
    for i, g in enumerate(gains):
        if g is not None:
            parts[i] = parts[i] / np.sqrt((parts[i] ** 2).mean(-1, keepdims=True) + eps) * g
    cs = tab.astype(np.float64)[pos]
    ref = [U.rotate(parts[0], cs, n_rot, layout), U.rotate(parts[1], cs, n_rot, layout), parts[2]]
    mag = [np.abs(p).max(-1, keepdims=True) * 2 for p in parts]
    f32 = [12 * 2.0 ** -24 * m for m in mag]
    step = (2.0 ** -24, 0) if qt == 0 else (U16, TINY16)
    got = q.cpu().double().numpy().reshape(T, H, hd)
    assert np.all(np.abs(got - ref[0]) <= step[0] * np.abs(ref[0]) + step[1] + f32[0])
    held = np.zeros((n_seq, n_ctx), bool)
    held[seq, cell] = True
    for i in (1, 2):
        raw = caches[i - 1].cpu().numpy()
        if kt == 2:
            c, d = unpack_cache(raw, n_seq, Hkv, n_ctx, hd)
            rc, rd = O.quantize_q4_0(ref[i].reshape(T * Hkv, hd))
            assert np.array_equal(c[seq, :, cell].reshape(T * Hkv, hd), rc)
            dd = d[seq, :, cell].reshape(T * Hkv, -1).astype(np.float64)
            assert np.all(np.abs(dd - rd.astype(np.float64)) <= 2 * U16 * np.abs(dd))      # its rounding, of values 2^-24 apart
            assert np.all(d.transpose(0, 2, 1, 3)[~held] == 0)
            continue
        if kt == 0:
            val, st = raw.view(np.float16).astype(np.float64), (U16, TINY16)
        else:
            val = torch.from_numpy(raw).view(torch.float8_e4m3fn).double().numpy()
            st = (2.0 ** -4, 2.0 ** -10)
        val = val.reshape(n_seq, Hkv, n_ctx, hd)
        assert np.all(np.abs(val[seq, :, cell] - ref[i]) <= st[0] * np.abs(ref[i]) + st[1] + f32[i])
        assert np.all(val.transpose(0, 2, 1, 3)[~held] == 0)


def test_rope_kv_is_qk_norm_rope(lib):
    """Whole heads in pairs with cells at their positions: the same bits."""
    rng = np.random.default_rng(1)
    T, H, Hkv, hd, n_ctx = 40, 4, 2, 64, 64
    x, g = dev(rng.standard_normal((T, (H + 2 * Hkv) * hd)).astype(np.float32)), dev(rng.random(hd).astype(np.float32))
    tab, pos, seq = dev(rng.standard_normal((n_ctx, hd // 2, 2)).astype(np.float32)), ints(np.arange(T)), ints([0] * T)
    out = []
    for general in (False, True):
        q = torch.zeros((T, H * hd), dtype=torch.float16, device="cuda")
        k, v = (torch.zeros((Hkv, n_ctx, hd), dtype=torch.float16, device="cuda") for _ in range(2))
        tail = [seq.data_ptr(), q.data_ptr(), 1, k.data_ptr(), v.data_ptr(), 0, T, H, Hkv, hd, n_ctx, 1, None, stream()]
        head = [x.data_ptr(), (H + 2 * Hkv) * hd, g.data_ptr(), g.data_ptr(), 1e-5, tab.data_ptr()]
        call = (lambda: lib.llm_op_rope_kv(*head, n_ctx, hd, 0, pos.data_ptr(), None, *tail)) if general else \
            (lambda: lib.llm_op_qk_norm_rope(*head, pos.data_ptr(), *tail))
        assert call() == 0
        out.append((q, k, v))
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("layout", [0, 1])
def test_rope_kv_rows_outside(lib, layout):
    T, H, Hkv, hd, n_ctx, n_seq, n_pos = 6, 2, 1, 64, 8, 2, 5
    x = torch.randn((T, (H + 2 * Hkv) * hd), device="cuda")
    tab = torch.ones((n_pos, hd // 2, 2), device="cuda")
    pos, cell, seq = ints([0, 5, -1, 1, 1, 4]), ints([0, 1, 2, 8, 3, 4]), ints([0, 0, 0, 0, 2, 1])
    q = torch.full((T, H * hd), 5.0, dtype=torch.float16, device="cuda")
    k, v = (torch.zeros((n_seq, Hkv, n_ctx, hd), dtype=torch.float16, device="cuda") for _ in range(2))
    E = err_word()
    assert lib.llm_op_rope_kv(x.data_ptr(), (H + 2 * Hkv) * hd, None, None, 0.0, tab.data_ptr(), n_pos, hd, layout,
                              pos.data_ptr(), cell.data_ptr(), seq.data_ptr(), q.data_ptr(), 1, k.data_ptr(), v.data_ptr(), 0,
                              T, H, Hkv, hd, n_ctx, n_seq, E.data_ptr(), stream()) == 0
    assert int(E) == 2
    assert torch.all(q[1:5] == 0) and torch.all(q[0] != 5) and torch.any(q[5] != 0)
    full = (v != 0).any(-1).any(1).cpu().numpy()
    want = np.zeros((n_seq, n_ctx), bool)
    want[0, 0] = want[1, 4] = True
    assert np.array_equal(full, want)


# ---------------------------------------------------------------- attention of trees

class Trees:
    """The inputs of one call: trees of (earlier cells, nodes), as host arrays and on the GPU."""

    def __init__(self, lib, hd, H, Hkv, trees, n_ctx, kt=0, window=0, kind="random", max_nodes=None, seed=0, qs=1.5, spare=0,
                 seen=None):
        rng = np.random.default_rng(seed + 7 * hd + H + len(trees))
        self.lib, self.hd, self.H, self.Hkv, self.n_ctx, self.kt, self.window = lib, hd, H, Hkv, n_ctx, kt, window
        self.trees, self.n_seq = trees, len(trees) + 1
        self.row0 = np.concatenate(([0], np.cumsum([n for _, n in trees])))
        self.T = max(int(self.row0[-1]) + spare, 1)
        self.max_nodes = max_nodes or max(max(n for _, n in trees), 1)
        self.seq = rng.permutation(self.n_seq)[:len(trees)]
        self.par = [U.parents(rng, n, kind) if n else np.zeros(0, int) for _, n in trees]
        self.seen = [U.ancestors(p) for p in self.par] if seen is None else seen
        self.pos = np.zeros(self.T, int)
        mask = np.zeros((self.T, (self.max_nodes + 31) // 32), np.uint32)
        for (b, n), r, p, s in zip(trees, self.row0, self.par, self.seen):
            self.pos[r:r + n] = b + U.depths(p)
            mask[r:r + n] = U.pack_mask(s, self.max_nodes)
        self.q = (rng.standard_normal((self.T, H, hd)) * qs).astype(np.float16)
        kv = [torch.from_numpy(rng.standard_normal((self.n_seq, Hkv, n_ctx, hd)).astype(np.float32)) for _ in range(2)]
        kv = [t.to(torch.float16 if kt == 0 else torch.float8_e4m3fn) for t in kv]
        self.k, self.v = (t.double().numpy() for t in kv)
        self.Q, self.KV = dev(self.q), [t.cuda() for t in kv]
        self.ROW0, self.SEQ, self.BASE = ints(self.row0), ints(self.seq), ints([b for b, _ in trees])
        self.MASK, self.POS = dev(mask.view(np.int32)), ints(self.pos)
        self.size = lib.llm_op_attn_tree_scratch_bytes(len(trees), self.max_nodes, H, Hkv, hd, n_ctx)
        self.SCRATCH = torch.zeros(self.size, dtype=torch.uint8, device="cuda")
        self.O = torch.full((self.T, H * hd), 9.0, dtype=torch.float16, device="cuda")
        self.E = err_word()

    def args(self, scratch=None, o=None):
        s = self.SCRATCH if scratch is None else scratch
        o = self.O if o is None else o
        return [self.Q.data_ptr(), self.KV[0].data_ptr(), self.KV[1].data_ptr(), self.ROW0.data_ptr(), self.SEQ.data_ptr(),
                self.BASE.data_ptr(), self.MASK.data_ptr(), self.POS.data_ptr() if self.window else None, o.data_ptr(), self.T,
                len(self.trees), self.max_nodes, self.H, self.Hkv, self.hd, self.n_ctx, self.n_seq, self.kt, self.window,
                s.data_ptr(), s.numel(), self.E.data_ptr(), stream()]

    def run(self, **kw):
        self.lib.check(self.lib.llm_op_attn_tree(*self.args(**kw)))
        return self.O

    def check(self, o=None, norm=True):
        got = (self.O if o is None else o).cpu().double().numpy().reshape(self.T, self.H, self.hd)
        num = den = 0.0
        for i, ((b, n), r) in enumerate(zip(self.trees, self.row0)):
            if not n:
                continue
            s = self.seq[i]
            ref, mag, size = U.attention(self.q[r:r + n].astype(np.float64), self.k[s], self.v[s], b, self.seen[i],
                                         self.pos[r:r + n], self.window)
            tol = U16 * np.abs(ref) + TINY16 + (2.0 ** -20 * size[..., None] + 2.0 ** -19) * mag
            d = np.abs(got[r:r + n] - ref)
            assert np.all(d <= tol), (i, float((d / tol).max()))
            num, den = num + (d ** 2).sum(), den + (ref ** 2).sum()
        if norm and den:
            # a rounding is uniform within half a step: 2^-11 / sqrt(3) of a value at the foot of its binade, 2.1e-4 over all
            assert np.sqrt(num / den) <= 2.6e-4
        end = int(self.row0[-1])
        assert np.all(got[end:] == 9.0)
        assert int(self.E) == 0


@pytest.mark.parametrize("kt", [0, 1])
@pytest.mark.parametrize("hd,H,Hkv,trees,n_ctx,window", [
    (128, 4, 1, [(0, 1)], 1, 0),
    (128, 4, 1, [(5, 1)], 6, 0),
    (128, 8, 2, [(127, 2)], 160, 0),              # a tree across a tile's edge
    (128, 8, 2, [(128, 16)], 300, 0),
    (128, 32, 8, [(1000, 16)], 1100, 0),
    (128, 8, 8, [(300, 64)], 500, 0),             # one query head a kv head
    (128, 16, 1, [(260, 30)], 290, 0),            # 480 rows of one kv head
    (128, 10, 2, [(77, 13)], 128, 0),             # five query heads a kv head: nodes across row tiles
    (64, 8, 2, [(700, 8), (3, 20), (0, 5)], 900, 0),
    (64, 6, 2, [(200, 33), (64, 1)], 256, 50),
    (32, 4, 2, [(100, 9)], 130, 0),
    (32, 12, 4, [(513, 40), (0, 1), (31, 64)], 600, 100),
    (128, 8, 2, [(900, 12), (450, 7)], 1000, 5),  # a window inside the tree's depth
    (128, 8, 2, [(900, 12)], 1000, 1),
    (64, 4, 2, [(140, 256)], 400, 0),             # the largest tree
])
def test_attention(lib, hd, H, Hkv, trees, n_ctx, window, kt):
    t = Trees(lib, hd, H, Hkv, trees, n_ctx, kt, window, spare=3)
    t.run()
    t.check()
    first = t.O.clone()
    t.O.fill_(9.0)
    t.run()                                       # the scratch is ready again, and the bits are the same
    assert torch.equal(first, t.O)


@pytest.mark.parametrize("kind", ["chain", "star"])
def test_tree_shapes(lib, kind):
    t = Trees(lib, 128, 8, 2, [(200, 100), (90, 40)], 320, kind=kind)
    t.run()
    t.check()


@pytest.mark.parametrize("hd,kt", [(128, 0), (64, 0), (128, 1)])
def test_long_context(lib, hd, kt):
    t = Trees(lib, hd, 8, 2, [(9000, 20), (40, 3)], 9100, kt)
    t.run()
    t.check(norm=False)


@pytest.mark.parametrize("hd,H,kt", [(128, 16, 0), (64, 16, 0), (32, 16, 0), (128, 8, 1), (64, 32, 1)])
@pytest.mark.parametrize("n", [3, 10, 24])
def test_many_tiles_a_split(lib, hd, H, kt, n):
    """Groups enough that a split has several tiles, with few rows and with many."""
    trees = [(1900 - 77 * i, 1 + (i * 5) % 23) for i in range(n)]
    t = Trees(lib, hd, H, 8, trees, 2000, kt, seed=n, spare=2)
    t.run()
    t.check()


@pytest.mark.parametrize("hd,kt", [(128, 0), (128, 1), (64, 0), (64, 1)])
def test_repeats_over_many_tiles(lib, hd, kt):
    """Splits of some twenty tiles: the rings of K and V go round often, whatever the order in which their tiles land."""
    t = Trees(lib, hd, 32, 8, [(9900, 16), (9000, 5), (10000, 1), (7777, 12)], 10016, kt)
    t.run()
    t.check()
    first, flush = t.O.clone(), torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for i in range(12):
        t.O.fill_(9.0)
        if i & 1:
            flush.zero_()                         # K and V from memory, else from L2
        t.run()
        assert torch.equal(first, t.O)


def test_many_trees(lib):
    """More groups than the GPU holds at once, some trees without nodes."""
    trees = [(37 * i % 400, i % 7) for i in range(90)]
    t = Trees(lib, 64, 4, 4, trees, 420, spare=5)
    t.run()
    t.check()


@pytest.mark.parametrize("hd,H,Hkv,kt", [(128, 8, 2, 0), (64, 4, 2, 1)])
def test_rows_that_see_nothing(lib, hd, H, Hkv, kt):
    rng = np.random.default_rng(3)
    trees = [(0, 40), (150, 20), (0, 3)]
    seen = []
    for b, n in trees:
        s = rng.random((n, n)) < 0.2                # any mask, bits of later nodes too
        s[::3] = False
        seen.append(s)
    t = Trees(lib, hd, H, Hkv, trees, 300, kt, seen=seen, max_nodes=45)
    t.run()
    t.check()
    blind = ~seen[0].any(1)
    assert blind.any() and torch.all(t.O[:40].view(40, -1)[torch.from_numpy(blind).cuda()] == 0)


def test_mask_bits_past_the_tree(lib):
    t = Trees(lib, 128, 4, 2, [(130, 10), (20, 6)], 200, max_nodes=70)
    t.MASK[:, 1:] = -1
    t.MASK[:, 0] |= -1 << 10                       # bits of nodes that the first tree does not have
    t.MASK[10:, 0] |= -1 << 6
    t.run()
    t.check()


@pytest.mark.parametrize("kt", [0, 1])
@pytest.mark.parametrize("fill", [float("nan"), float("inf")])
def test_unseen_cells_may_hold_anything(lib, fill, kt):
    """Cells behind the tree, before the window, and nodes that a row does not see."""
    t = Trees(lib, 128, 8, 2, [(700, 12), (128, 5)], 900, kt, window=64)
    bad = float("nan") if kt else fill
    clean = t.run().clone()
    t.check()
    depth = U.depths(t.par[0])
    lone = 11                                      # the last node has no children: only itself sees it
    for c in t.KV:
        v = c.view(torch.uint8) if kt else c
        x = 0x7f if kt else bad
        v[t.seq[0], :, 712:] = x
        v[t.seq[0], :, :700 - 64] = x              # every row's window starts later
        v[t.seq[0], :, 700 + lone] = x
        v[t.seq[1], :, 133:] = x
    t.run()
    rows = torch.ones(t.T, dtype=torch.bool, device="cuda")
    rows[lone] = False
    assert torch.equal(clean[rows], t.O[rows])
    assert not torch.isfinite(t.O[lone]).any()
    assert depth[lone] >= 1


def test_score_ranges(lib):
    for qs in (0.0, 1e-3, 30.0, 300.0):
        t = Trees(lib, 128, 4, 1, [(500, 9)], 520, qs=qs)
        t.run()
        t.check()


def test_trees_that_do_not_fit(lib):
    t = Trees(lib, 64, 4, 2, [(10, 4), (20, 5), (30, 3), (0, 2), (8, 4)], 60)
    t.BASE.copy_(ints([10, 56, -1, 0, 8]))         # 56 + 5 > 60; a negative base
    t.SEQ.copy_(ints([t.seq[0], t.seq[1], t.seq[2], t.n_seq, t.seq[4]]))
    t.run()
    assert int(t.E) == 2
    t.E.zero_()
    got = t.O.clone()
    assert torch.all(got[4:14] == 0)               # the three trees that do not fit
    assert torch.all(got[:4] != 9) and torch.all(got[14:] != 9)
    t.trees = [t.trees[0], (20, 0), (30, 0), (0, 0), t.trees[4]]
    t.check()
    t.ROW0.copy_(ints([0, 4, 40, 12, 14, 18]))     # rows past T, then descending
    t.BASE.copy_(ints([10, 0, 0, 0, 8]))
    t.O.fill_(9.0)
    t.run()
    assert int(t.E) == 2 and torch.equal(got[:4], t.O[:4])


def test_streams_graphs_and_scratch(lib):
    """Two captured graphs with a scratch each beside an eager call, replayed with other lengths; one scratch for two shapes."""
    a = Trees(lib, 128, 8, 2, [(3000, 16), (100, 9)], 3100, seed=1)
    b = Trees(lib, 64, 8, 2, [(500, 30)], 600, seed=2)
    a.run(), b.run()
    graphs = []
    for t in (a, b):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                t.run()
        graphs.append((s, g))
    torch.cuda.synchronize()
    for t in (a, b):
        t.O.fill_(9.0)
    for _ in range(5):
        for s, g in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    a.check(), b.check()
    # the same graph with other lengths
    a.trees = [(1700, 16), (5, 9)]
    for i, (base, n) in enumerate(a.trees):
        a.pos[a.row0[i]:a.row0[i] + n] = base + U.depths(a.par[i])
    a.BASE.copy_(ints([1700, 5]))
    torch.cuda.synchronize()
    with torch.cuda.stream(graphs[0][0]):
        graphs[0][1].replay()
    torch.cuda.synchronize()
    a.check()
    big = torch.zeros(max(a.size, b.size), dtype=torch.uint8, device="cuda")
    for t in (a, b, a):
        t.O.fill_(9.0)
        t.run(scratch=big)
        t.check()


FIRST_IN_CAPTURE = """
import sys
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import torch
import test_gpu_tree as t
import llama_decoder_forward_02_gb300 as lib
a = t.Trees(lib, {hd}, 8, 2, [(900, 12), (30, 4)], 1000, {kt})
r = lib.rope(10000.0, 64)
tab = torch.zeros((100, 32, 2), device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a.run()
    lib.check(lib.llm_op_rope_table(r, 0, 100, tab.data_ptr(), t.stream()))
g.replay()
a.check()
assert torch.all(tab[0, :, 0] == 1) and torch.all(tab[1:, 0, 1] != 0)
"""


@pytest.mark.parametrize("hd,kt", [(128, 0), (64, 1)])
def test_first_calls_of_a_process_captured(lib, hd, kt):
    """The calls' set-up of the device does not disturb a capture that runs before any other call."""
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_IN_CAPTURE.format(root=os.path.dirname(tests), tests=tests, hd=hd, kt=kt)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_calls_of_two_threads(lib):
    """Two threads that call at once, on a stream and with a scratch each."""
    parts = [Trees(lib, 128, 8, 2, [(1500, 16), (77, 3)], 1600, seed=1), Trees(lib, 64, 12, 4, [(600, 40)], 700, 1, seed=2)]
    torch.cuda.synchronize()
    failed = []

    def work(t):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    t.run()
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            failed.append(e)
    threads = [threading.Thread(target=work, args=(t,)) for t in parts]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not failed
    for t in parts:
        t.check()


def test_windows_of_any_size(lib):
    """Positions and windows at the ends of their type: what pos - window would be passes 32 bits."""
    t = Trees(lib, 64, 4, 2, [(300, 6), (200, 3)], 400, window=2 ** 31 - 1)
    t.run()
    t.check()
    whole = t.O.clone()
    t.POS[:] = -2 ** 31
    t.run()
    assert torch.equal(whole, t.O)                 # every earlier cell is inside
    t.POS[:] = 2 ** 31 - 1
    t.window = 1
    t.run()
    t.pos[:] = 2 ** 31 - 1                         # none is
    t.check()


@pytest.mark.parametrize("hd,kt", [(128, 0), (64, 1)])
def test_values_that_are_not_finite(lib, hd, kt):
    """In a query: its row and head alone; in a key or value that some rows see: theirs, of the heads of its kv head."""
    t = Trees(lib, hd, 8, 2, [(400, 10)], 500, kt)
    clean = t.run().view(t.T, 8, hd).clone()
    q = t.Q.clone()
    t.Q[3, 5, 7] = float("inf")
    t.Q[4, 0, 0] = float("nan")
    t.run()
    got = t.O.view(t.T, 8, hd)
    hit = torch.zeros((t.T, 8), dtype=torch.bool, device="cuda")
    hit[3, 5] = hit[4, 0] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert not torch.isfinite(got[hit]).any()
    t.Q.copy_(q)
    node = 4
    sees = torch.from_numpy(t.seen[0][:, node]).cuda()
    assert sees.any() and not sees.all()
    for c in t.KV:
        keep = c.clone()
        (c.view(torch.uint8) if kt else c)[t.seq[0], 1, 400 + node, 3] = 0x7f if kt else float("nan")
        t.run()
        got = t.O.view(t.T, 8, hd)
        assert torch.equal(got[:, :4], clean[:, :4]) and torch.equal(got[~sees], clean[~sees])
        bad = ~torch.isfinite(got[sees][:, 4:])
        assert bad.any(-1).all()
        c.copy_(keep)


def test_captured_step_replayed(lib):
    """Rotation, attention and acceptance as one graph, replayed on other inputs in the same memory: each replay as eager calls."""
    H, Hkv, hd, n_ctx, n, base = 8, 2, 64, 200, 9, 100
    rng = np.random.default_rng(5)
    par = U.parents(rng, n)
    tab = torch.empty((n_ctx, hd // 2, 2), device="cuda")
    lib.check(lib.llm_op_rope_table(lib.rope(10000.0, hd), 0, n_ctx, tab.data_ptr(), stream()))
    R, S, B, C = ints([0, n]), ints([0]), ints([base]), ints(base + np.arange(n))
    P, M, pr = ints(base + U.depths(par)), dev(U.pack_mask(U.ancestors(par), n).view(np.int32)), ints(par)
    x, tok, tgt = torch.empty((n, (H + 2 * Hkv) * hd), device="cuda"), ints([0] * n), ints([0] * n)
    kv = [torch.empty((1, Hkv, n_ctx, hd), dtype=torch.float16, device="cuda") for _ in range(2)]
    q, o = (torch.empty((n, H * hd), dtype=torch.float16, device="cuda") for _ in range(2))
    path, count, nxt = torch.empty((1, n), dtype=torch.int32, device="cuda"), ints([0]), ints([0])
    sc = torch.zeros(lib.llm_op_attn_tree_scratch_bytes(1, n, H, Hkv, hd, n_ctx), dtype=torch.uint8, device="cuda")

    def step():
        lib.check(lib.llm_op_rope_kv(x.data_ptr(), x.shape[1], None, None, 0.0, tab.data_ptr(), n_ctx, hd, 1, P.data_ptr(),
                                     C.data_ptr(), zeros.data_ptr(), q.data_ptr(), 1, kv[0].data_ptr(), kv[1].data_ptr(), 0, n,
                                     H, Hkv, hd, n_ctx, 1, None, stream()))
        lib.check(lib.llm_op_attn_tree(q.data_ptr(), kv[0].data_ptr(), kv[1].data_ptr(), R.data_ptr(), S.data_ptr(), B.data_ptr(),
                                       M.data_ptr(), None, o.data_ptr(), n, 1, n, H, Hkv, hd, n_ctx, 1, 0, 0, sc.data_ptr(),
                                       sc.numel(), None, stream()))
        lib.check(lib.llm_op_tree_accept(tok.data_ptr(), pr.data_ptr(), tgt.data_ptr(), R.data_ptr(), S.data_ptr(), B.data_ptr(),
                                         kv[0].data_ptr(), kv[1].data_ptr(), 0, path.data_ptr(), count.data_ptr(), nxt.data_ptr(),
                                         n, 1, n, 1, Hkv, hd, n_ctx, 1, None, stream()))
    zeros = ints([0] * n)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(dev(rng.standard_normal(x.shape).astype(np.float32)))
        tok.copy_(ints(rng.integers(0, 3, n)))
        tgt.copy_(ints(rng.integers(0, 3, n)))
        past = [torch.randn_like(c) for c in kv]
        outs = []
        for call in (step, g.replay):
            for c, p in zip(kv, past):
                c.copy_(p)
            o.fill_(9.0)
            call()
            outs.append([t.clone() for t in (*kv, o, path, count, nxt)])
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        want, nx = U.accept(tok.cpu().numpy(), par, tgt.cpu().numpy())
        assert path[0, :len(want)].tolist() == want and int(nxt) == nx


def test_cells_past_32_bits(lib):
    """A cache whose elements pass 2^31: rotation and append, attention and acceptance in its last sequence, and none elsewhere."""
    H, Hkv, hd, n_ctx, n_seq, n, base = 4, 1, 128, 1048576 + 77, 17, 6, 1048576 + 60
    at = n_seq - 1
    assert at * n_ctx * hd > 2 ** 31
    kv = [torch.zeros((n_seq, Hkv, n_ctx, hd), dtype=torch.float16, device="cuda") for _ in range(2)]
    gen = torch.Generator(device="cuda").manual_seed(0)
    for c in kv:
        c[at, 0, :base] = torch.randn((base, hd), generator=gen, device="cuda")
    rng = np.random.default_rng(2)
    par = np.array([-1, 0, 0, 2, 3, 1])
    pos = base + U.depths(par)
    tab = torch.empty((100, hd // 2, 2), device="cuda")
    lib.check(lib.llm_op_rope_table(lib.rope(500000.0, hd), base, 100, tab.data_ptr(), stream()))
    x = dev(rng.standard_normal((n, (H + 2 * Hkv) * hd)).astype(np.float32))
    q, o = (torch.zeros((n, H * hd), dtype=torch.float16, device="cuda") for _ in range(2))
    P, C, S = ints(U.depths(par)), ints(base + np.arange(n)), ints([at] * n)
    E = err_word()
    lib.check(lib.llm_op_rope_kv(x.data_ptr(), x.shape[1], None, None, 0.0, tab.data_ptr(), 100, hd, 0, P.data_ptr(), C.data_ptr(),
                                 S.data_ptr(), q.data_ptr(), 1, kv[0].data_ptr(), kv[1].data_ptr(), 0, n, H, Hkv, hd, n_ctx, n_seq,
                                 E.data_ptr(), stream()))
    # the angles themselves are held against 64 bits above; here the rows have to stand in their cells
    xs = x.cpu().double().numpy().reshape(n, H + 2 * Hkv, hd)
    cs = tab.cpu().double().numpy()[U.depths(par)]
    k_ref, v_ref = U.rotate(xs[:, H:H + 1], cs, hd, 0)[:, 0], xs[:, H + 1]
    for c, ref in zip(kv, (k_ref, v_ref)):
        got = c[at, 0, base:base + n].cpu().double().numpy()
        assert np.all(np.abs(got - ref) <= U16 * np.abs(ref) + TINY16 + 12 * 2.0 ** -24 * 2 * np.abs(ref).max())
    R, Q, B, M = ints([0, n]), ints([at]), ints([base]), dev(U.pack_mask(U.ancestors(par), n).view(np.int32))
    sc = torch.zeros(lib.llm_op_attn_tree_scratch_bytes(1, n, H, Hkv, hd, n_ctx), dtype=torch.uint8, device="cuda")
    lib.check(lib.llm_op_attn_tree(q.data_ptr(), kv[0].data_ptr(), kv[1].data_ptr(), R.data_ptr(), Q.data_ptr(), B.data_ptr(),
                                   M.data_ptr(), None, o.data_ptr(), n, 1, n, H, Hkv, hd, n_ctx, n_seq, 0, 0, sc.data_ptr(),
                                   sc.numel(), E.data_ptr(), stream()))
    k, v = (c[at, 0, :base + n].double() for c in kv)
    s = torch.einsum("nhd,cd->nhc", q.view(n, H, hd).double(), k) / hd ** 0.5
    s[..., base:].masked_fill_(~torch.from_numpy(U.ancestors(par)).cuda()[:, None], float("-inf"))
    w = torch.softmax(s, -1)
    ref, mag = torch.einsum("nhc,cd->nhd", w, v), torch.einsum("nhc,cd->nhd", w, v.abs())
    size = torch.sqrt(torch.einsum("nhd,cd->nhc", q.view(n, H, hd).double() ** 2, k ** 2)).amax(-1)
    tol = U16 * ref.abs() + TINY16 + (2.0 ** -20 * size[..., None] + 2.0 ** -19) * mag
    # more for a million cells: on 2^3 CTAs or more a sum of weights takes below 2^11 additions, off by 2^-24 each like a
    # random walk, and a sum of products 2^4 steps a tile, 2^14 in all, off by 2^-23 each: 2^-18 and 2^-16
    tol += (2.0 ** -18 + 2.0 ** -16) * mag
    assert torch.all((o.view(n, H, hd).double() - ref).abs() <= tol)
    token, target = ints([1, 2, 3, 4, 5, 6]), ints([3, 0, 4, 5, 9, 0])
    rows = [c[at, 0, base:base + n].clone() for c in kv]
    pr, path, count, nxt = ints(par), torch.empty((1, n), dtype=torch.int32, device="cuda"), ints([0]), ints([0])
    lib.check(lib.llm_op_tree_accept(token.data_ptr(), pr.data_ptr(), target.data_ptr(), R.data_ptr(), Q.data_ptr(), B.data_ptr(),
                                     kv[0].data_ptr(), kv[1].data_ptr(), 0, path.data_ptr(), count.data_ptr(), nxt.data_ptr(), n, 1,
                                     n, 1, Hkv, hd, n_ctx, n_seq, E.data_ptr(), stream()))
    assert path[0, :4].tolist() == [0, 2, 3, 4] and int(nxt) == 9 and int(E) == 0
    for c, r in zip(kv, rows):
        assert torch.equal(c[at, 0, base:base + 4], r[[0, 2, 3, 4]]) and torch.equal(c[at, 0, base + 4:base + n], r[4:])
        assert not c[:at].any() and not c[at, 0, base + n:].any()


# ---------------------------------------------------------------- acceptance

def make_accept(rng, sizes, kind="random", agree=0.6, vocab=50):
    token, parent, target = [], [], []
    for n in sizes:
        p = U.parents(rng, n, kind) if n else np.zeros(0, int)
        tok, tgt = rng.integers(0, vocab, n), rng.integers(0, vocab, n)
        for i in range(1, n):                       # most parents pick one of their children
            if rng.random() < agree:
                tgt[p[i]] = tok[i]
        token.append(tok), parent.append(p), target.append(tgt)
    return token, parent, target


@pytest.mark.parametrize("kt", [0, 1, 2])
@pytest.mark.parametrize("hd,Hkv,L,sizes,kind", [
    (128, 2, 3, [16], "random"),
    (128, 1, 2, [256, 1, 0, 40], "chain"),
    (64, 2, 2, [64, 33, 2], "random"),
    (32, 3, 1, [100, 7], "star"),
    (128, 2, 1, [200] * 5, "random"),
])
def test_accept(lib, hd, Hkv, L, sizes, kind, kt):
    rng = np.random.default_rng(hd + L + kt)
    n_tree, n_seq, T = len(sizes), len(sizes) + 1, sum(sizes)
    most = max(sizes)
    n_ctx = most + 30
    token, parent, target = make_accept(rng, sizes, kind, 0.97 if kind == "chain" else 0.6)
    base = rng.integers(0, 30, n_tree)
    seq = rng.permutation(n_seq)[:n_tree]
    row0 = np.concatenate(([0], np.cumsum(sizes)))
    rows = n_seq * L * Hkv * n_ctx
    per = {0: 2 * hd, 1: hd, 2: hd // 2}[kt]
    planes = [rng.integers(0, 256, (n_seq, L * Hkv, n_ctx, per), dtype=np.uint8) for _ in range(2)]
    scales = [rng.integers(0, 256, (n_seq, L * Hkv, n_ctx, hd // 16), dtype=np.uint8) for _ in range(2)]
    KV = [dev(np.concatenate([p.reshape(-1)] + ([s.reshape(-1)] if kt == 2 else []) + [np.zeros(64, np.uint8)]))
          for p, s in zip(planes, scales)]
    path = torch.full((n_tree, most), 77, dtype=torch.int32, device="cuda")
    count, nxt, E = ints([77] * n_tree), ints([77] * n_tree), err_word()
    tk, pr, tg = (ints(np.concatenate(x)) for x in (token, parent, target))
    R, S, B = ints(row0), ints(seq), ints(base)
    assert lib.llm_op_tree_accept(tk.data_ptr(), pr.data_ptr(), tg.data_ptr(), R.data_ptr(), S.data_ptr(), B.data_ptr(),
                                  KV[0].data_ptr(), KV[1].data_ptr(), kt, path.data_ptr(), count.data_ptr(), nxt.data_ptr(),
                                  T, n_tree, most, L, Hkv, hd, n_ctx, n_seq, E.data_ptr(), stream()) == 0
    assert int(E) == 0
    for i, n in enumerate(sizes):
        p, nx = U.accept(token[i], parent[i], target[i]) if n else ([], -1)
        assert path[i].tolist() == p + [-1] * (most - len(p)) and int(count[i]) == len(p) and int(nxt[i]) == nx
        for arrs in (planes, scales):
            for c in arrs:
                held = c[seq[i]]
                held[:, base[i]:base[i] + len(p)] = held[:, [base[i] + j for j in p]]
    for g, p, s in zip(KV, planes, scales):
        want = np.concatenate([p.reshape(-1)] + ([s.reshape(-1)] if kt == 2 else []) + [np.zeros(64, np.uint8)])
        assert np.array_equal(g.cpu().numpy(), want)
    assert rows * per == planes[0].size


def test_accept_refuses_broken_trees(lib):
    """A parent that is not a lower node, a root with a parent, a tree outside the cache: nothing accepted, nothing moved."""
    T, n_ctx, hd = 12, 20, 32
    parent = ints([-1, 0, 1, -1, 2, 0, 0, 0, 0, -1, 0, 1])     # tree 1: node 1 under node 2; tree 2: a root with a parent
    token, target = ints([5] * T), ints([5] * T)
    row0, seq, base = ints([0, 3, 6, 9, 12]), ints([0, 1, 2, 3]), ints([0, 0, 0, 18])
    k = torch.arange(4 * n_ctx * hd, device="cuda").to(torch.float16).view(4, 1, n_ctx, hd)
    v = k.clone()
    keep = k.clone()
    path, count, nxt, E = torch.zeros((4, 3), dtype=torch.int32, device="cuda"), ints([7] * 4), ints([7] * 4), err_word()
    assert lib.llm_op_tree_accept(token.data_ptr(), parent.data_ptr(), target.data_ptr(), row0.data_ptr(), seq.data_ptr(),
                                  base.data_ptr(), k.data_ptr(), v.data_ptr(), 0, path.data_ptr(), count.data_ptr(),
                                  nxt.data_ptr(), T, 4, 3, 1, 1, hd, n_ctx, 4, E.data_ptr(), stream()) == 0
    assert int(E) == 2
    assert count.tolist() == [3, 0, 0, 0] and nxt.tolist() == [5, -1, -1, -1] and path.tolist() == [[0, 1, 2]] + [[-1] * 3] * 3
    assert torch.equal(k, keep) and torch.equal(v, keep)


# ---------------------------------------------------------------- together

def test_step_of_a_tree(lib):
    """Rotate and append, attend, accept and move, attend a chain behind the accepted path: as if it had been decoded alone."""
    rng = np.random.default_rng(9)
    H, Hkv, hd, n_ctx, base, n = 8, 2, 64, 300, 131, 14
    r = lib.rope(10000.0, 32, layout=lib.LLM_ROPE_HALVES, scaling=lib.LLM_ROPE_RAMP, factor=4.0, n_ctx_orig=64)
    tab = torch.empty((n_ctx, 16, 2), device="cuda")
    lib.check(lib.llm_op_rope_table(r, 0, n_ctx, tab.data_ptr(), stream()))
    kc, vc = (torch.zeros((1, Hkv, n_ctx, hd), dtype=torch.float16, device="cuda") for _ in range(2))
    par = U.parents(rng, n)
    depth = U.depths(par)
    deepest = [int(depth.argmax())]
    while deepest[0]:
        deepest.insert(0, int(par[deepest[0]]))

    def append(x, pos, cell):
        T = len(x)
        q = torch.empty((T, H * hd), dtype=torch.float16, device="cuda")
        X, P, C, S = dev(x), ints(pos), ints(cell), ints([0] * T)
        lib.check(lib.llm_op_rope_kv(X.data_ptr(), x.shape[1], None, None, 0.0, tab.data_ptr(), n_ctx, 32, 1, P.data_ptr(),
                                     C.data_ptr(), S.data_ptr(), q.data_ptr(), 1, kc.data_ptr(), vc.data_ptr(), 0, T, H, Hkv, hd,
                                     n_ctx, 1, None, stream()))
        return q

    def attend(q, at, seen):
        T = len(q)
        R, S, B, M = ints([0, T]), ints([0]), ints([at]), dev(U.pack_mask(seen, T).view(np.int32))
        o = torch.empty_like(q)
        sc = torch.zeros(lib.llm_op_attn_tree_scratch_bytes(1, T, H, Hkv, hd, n_ctx), dtype=torch.uint8, device="cuda")
        lib.check(lib.llm_op_attn_tree(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), R.data_ptr(), S.data_ptr(), B.data_ptr(),
                                       M.data_ptr(), None, o.data_ptr(), T, 1, T, H, Hkv, hd, n_ctx, 1, 0, 0, sc.data_ptr(),
                                       sc.numel(), None, stream()))
        return o
    width = (H + 2 * Hkv) * hd
    past, drafts, later = (rng.standard_normal((m, width)).astype(np.float32) for m in (base, n, 3))
    append(past, range(base), range(base))
    o_tree = attend(append(drafts, base + depth, base + np.arange(n)), base, U.ancestors(par))
    token = np.arange(100, 100 + n)
    target = np.full(n, 7)
    for a, b in zip(deepest, deepest[1:]):
        target[a] = token[b]
    path, count, nxt = torch.empty((1, n), dtype=torch.int32, device="cuda"), ints([0]), ints([0])
    tk, pr, tg, R, S, B = ints(token), ints(par), ints(target), ints([0, n]), ints([0]), ints([base])
    lib.check(lib.llm_op_tree_accept(tk.data_ptr(), pr.data_ptr(), tg.data_ptr(), R.data_ptr(), S.data_ptr(), B.data_ptr(),
                                     kc.data_ptr(), vc.data_ptr(), 0, path.data_ptr(), count.data_ptr(), nxt.data_ptr(), n, 1, n,
                                     1, Hkv, hd, n_ctx, 1, None, stream()))
    m = len(deepest)
    assert path[0, :m].tolist() == deepest and int(count) == m and int(nxt) == 7
    at = base + m
    o_later = attend(append(later, at + np.arange(3), at + np.arange(3)), at, U.ancestors(np.arange(-1, 2)))
    # the same without a tree: the path's tokens one behind the other
    kept = [c[0, :, :at + 3].clone() for c in (kc, vc)]
    kc.zero_(), vc.zero_()
    append(past, range(base), range(base))
    o_path = attend(append(drafts[deepest], base + np.arange(m), base + np.arange(m)), base, U.ancestors(np.arange(-1, m - 1)))
    append(later, at + np.arange(3), at + np.arange(3))
    assert all(torch.equal(a, c[0, :, :at + 3]) for a, c in zip(kept, (kc, vc)))
    # sums of other cells beside them: the same up to the rounding of fp16 and of the sums
    assert torch.allclose(o_tree[deepest].float(), o_path.float(), rtol=2 * U16, atol=2.0 ** -17)
    again = attend(append(later, at + np.arange(3), at + np.arange(3)), at, U.ancestors(np.arange(-1, 2)))
    assert torch.equal(o_later, again)
