"""Prefill attention over a Q4_0 cache, held to the precision of its definition:
q as it comes, K and V exact, softmax weights of 22 bits, fp32 sums, one rounding
of o.

Tolerances.  A score is 2 hd / 16 sums of 16 exact products, each truncated at
2^-23 of the largest partial sum, at most sum |q k| / sqrt(hd): relative errors of
a weight are (2 hd / 16 + 4) 2^-23 max sum |q k| / sqrt(hd), with 2^-21 for the
weight itself (exponential and its two fp16 parts).  O takes 24 such sums a tile
of 128 keys.  Both enter numerators and denominator: twice, times sum p |v|.  A
weight's two fp16 parts are kept 2^7 times as large as the weight, the row's largest
being 1 or more; among fp16's subnormals each part is off by half their step,
2^-25: 2 * 2^-25 * 2^-7 = 2^-31 a weight, times sum |v|.  Then o's rounding, half a
step."""
import numpy as np
import pytest
import torch

from oracle import llama as O
from q4_util import pack_cache
from test_gpu_q4 import dev, make_cache, reference, stream, visible_cells

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -11, 2.0 ** -23


@pytest.fixture(scope="module")
def lib():
    import llama_decoder_forward_02_gb300 as L
    return L


def rows_of(runs):
    """pos and seq of runs [(seq, first position, rows)]."""
    pos = np.concatenate([np.arange(a, a + n) for _, a, n in runs]).astype(np.int32)
    seq = np.concatenate([np.full(n, s) for s, _, n in runs]).astype(np.int32)
    return pos, seq


def half_step(x):
    """Half the distance of fp16 numbers next to x."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -14)))
    return 2.0 ** (e - 11)


def tolerance(ref, q, k, v, pos, seq, Hkv, window):
    """The bound of the head of this file, [T][H][hd]; q [T][H][hd]."""
    T, H, hd = q.shape
    vis = visible_cells(pos, seq, k.shape[0], k.shape[2], window)
    ka, va = (np.where(vis[:, None, :, None], np.abs(u), 0) for u in (k, v))
    mag = 0.0
    for s in np.unique(seq):
        a = np.abs(q[seq == s]).reshape(-1, Hkv, H // Hkv, hd)
        mag = max(mag, np.einsum("tjgd,jcd->tjgc", a, ka[s]).max() / np.sqrt(hd))
    tiles = -(-min(int(pos.max()) + 1, window + 128 if window else 1 << 30) // 128) + 1
    w = (2 * hd / 16 + 4) * U32 * mag + 2.0 ** -21 + 24 * tiles * U32
    mean = reference(q, k, va, pos, seq, Hkv, window)
    whole = reference(np.zeros_like(q), k, va, pos, seq, Hkv, window)      # equal weights: the mean of |v|
    seen = np.minimum(pos + 1, window) if window else pos + 1
    off = 2 * w * mean + 2.0 ** -31 * whole * seen[:, None, None]
    return half_step(np.abs(ref) + off) + off


class Prefill:
    def __init__(self, lib, hd, H, Hkv, n_ctx, n_seq, runs, window=0, qs=1.5, vs=1.0, seed=0):
        rng = np.random.default_rng(seed + hd + H + n_ctx)
        self.lib, self.shape, self.window = lib, (H, Hkv, hd, n_ctx, n_seq), window
        self.pos, self.seq = rows_of(runs)
        self.T = len(self.pos)
        vis = visible_cells(self.pos, self.seq, n_seq, n_ctx, window)
        self.kc, self.kd = make_cache(rng, n_seq, Hkv, n_ctx, hd, vis)
        self.vc, self.vd = make_cache(rng, n_seq, Hkv, n_ctx, hd, vis)
        self.vd = (self.vd.astype(np.float32) * np.float32(vs)).astype(np.float16)
        self.q = (rng.standard_normal((self.T, H, hd)) * qs).astype(np.float16)
        k, v = O.dequantize_q4_0(self.kc, self.kd), O.dequantize_q4_0(self.vc, self.vd)
        q = self.q.astype(np.float64)
        self.ref = reference(q, k, v, self.pos, self.seq, Hkv, window)
        self.tol = tolerance(self.ref, q, k, v, self.pos, self.seq, Hkv, window)
        self.o = torch.full((self.T + 3, H * hd), 9.0, dtype=torch.float16, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        n = lib.llm_op_attn_prefill_q4_0_scratch_bytes(self.T, H, Hkv, hd, n_ctx, n_seq)
        self.scratch = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        self.upload()

    def upload(self):
        self.qd, self.kcd, self.vcd = dev(self.q), dev(pack_cache(self.kc, self.kd)), dev(pack_cache(self.vc, self.vd))

    def call(self):
        H, Hkv, hd, n_ctx, n_seq = self.shape
        return self.lib.llm_op_attn_prefill_q4_0(
            self.qd.data_ptr(), self.kcd.data_ptr(), self.vcd.data_ptr(), self.pos.ctypes.data, self.seq.ctypes.data,
            self.o.data_ptr(), self.T, H, Hkv, hd, n_ctx, n_seq, self.window, self.scratch.data_ptr(), self.scratch.numel(),
            self.err.data_ptr(), stream())

    def got(self):
        torch.cuda.synchronize()
        o = self.o.cpu().double().numpy()
        assert np.all(o[self.T:] == 9.0)
        return o[:self.T].reshape(self.ref.shape)

    def check(self, rows=slice(None)):
        off = np.abs(self.got()[rows] - self.ref[rows])
        assert np.all(off <= self.tol[rows]), (off / self.tol[rows]).max()


CASES = [
    (128, 8, 2, 700, [(0, 0, 512)], 0, 1.5, 1.0), (128, 32, 8, 1300, [(0, 1000, 300)], 0, 1.5, 1.0),
    (128, 4, 1, 300, [(0, 37, 100), (2, 0, 9), (1, 250, 1)], 0, 1.5, 1e-2), (64, 6, 2, 400, [(1, 100, 300), (0, 0, 77)], 0, 1.5, 1.0),
    (32, 4, 2, 200, [(0, 0, 150), (1, 33, 65)], 0, 1.5, 1.0), (128, 4, 2, 600, [(0, 300, 200)], 64, 1.5, 1.0),
    (64, 4, 4, 513, [(0, 500, 13), (1, 64, 128)], 1, 1.5, 1.0), (32, 2, 1, 300, [(0, 128, 140)], 70, 1.5, 1e-2),
    (128, 5, 1, 130, [(0, 0, 130)], 0, 0.0, 1.0), (64, 2, 1, 1, [(0, 0, 1)], 0, 1.5, 1.0),
    (128, 4, 2, 640, [(0, 128, 512)], 0, 8.0, 1.0), (64, 4, 2, 640, [(0, 128, 500)], 0, 8.0, 1e-2),
    (32, 4, 2, 640, [(0, 128, 400)], 0, 8.0, 1e-2), (64, 8, 8, 2000, [(0, 1871, 129)], 0, 1.5, 1.0),
    (32, 3, 1, 2000, [(0, 1871, 129)], 1500, 1.5, 1.0), (128, 4, 2, 1000, [(0, 600, 400)], 300, 8.0, 1e-3),
]


@pytest.mark.parametrize("hd,H,Hkv,n_ctx,runs,window,qs,vs", CASES)
def test_precision(lib, hd, H, Hkv, n_ctx, runs, window, qs, vs):
    """Every element within its own rounding and the fp32 sums, whatever the sizes of q and V; the whole within the
    rounding alone: half steps are 2^-10 / sqrt(12) = 2.8e-4 of a value at most, in the mean square."""
    c = Prefill(lib, hd, H, Hkv, n_ctx, max(s for s, _, _ in runs) + 1, runs, window, qs, vs)
    for _ in range(2):
        assert c.call() == 0, lib.llm_last_error(None)
        c.check()
    if vs == 1.0 and len(c.ref) > 64:                             # V of 1e-2 and less: o among the subnormals
        assert np.linalg.norm(c.got() - c.ref) <= 3.2e-4 * np.linalg.norm(c.ref)
    assert int(c.err) == 0


def test_masked_cells_may_hold_anything(lib):
    """Cells without a finite value, or beyond fp16's range, in the middle of the rows' own: rows before them are as if
    they were not there, heads that see them are NaN, in K as in V, whichever block they are in."""
    for hd, H, Hkv, odd, in_k in ((128, 4, 2, np.inf, False), (128, 4, 2, np.nan, True), (64, 6, 2, 9000.0, False),
                                  (64, 6, 2, -np.inf, True), (32, 4, 2, np.nan, False), (32, 4, 2, np.inf, True)):
        c = Prefill(lib, hd, H, Hkv, 400, 1, [(0, 20, 300)])
        cell = 150
        (c.kd if in_k else c.vd)[0, 1, cell, -1] = odd            # kv head 1, last block
        c.upload()
        assert c.call() == 0
        got = c.got()
        before, G = c.pos < cell, H // Hkv
        c.check(before)
        assert np.all(np.isnan(got[~before][:, G:])) and int(c.err) == 0
        assert np.all(np.abs(got[:, :G] - c.ref[:, :G]) <= c.tol[:, :G])


def test_scratch_is_not_needed(lib):
    c = Prefill(lib, 64, 4, 2, 200, 2, [(1, 30, 100), (0, 0, 7)])
    H, Hkv, hd, n_ctx, n_seq = c.shape
    assert lib.llm_op_attn_prefill_q4_0(c.qd.data_ptr(), c.kcd.data_ptr(), c.vcd.data_ptr(), c.pos.ctypes.data,
                                        c.seq.ctypes.data, c.o.data_ptr(), c.T, H, Hkv, hd, n_ctx, n_seq, 0, None, 0, None,
                                        stream()) == 0, lib.llm_last_error(None)
    c.check()


@pytest.mark.parametrize("hd,n_seq", [(64, 150), (32, 65)])
def test_many_sequences_captured(lib, hd, n_seq):
    """Rows of more sequences than one launch takes, captured and replayed after the call's host arrays are gone and q
    and the caches have moved."""
    runs = [(s, s % 50, 1 + s % 3) for s in range(n_seq)]
    a, b = (Prefill(lib, hd, 4, 2, 60, n_seq, runs, seed=i) for i in (1, 2))
    assert a.call() == 0
    a.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert a.call() == 0
    a.pos[:], a.seq[:] = 1 << 20, 1 << 20
    for n in ("qd", "kcd", "vcd"):
        getattr(a, n).copy_(getattr(b, n))
    a.o.fill_(9.0)
    g.replay()
    a.ref, a.tol = b.ref, b.tol
    a.check()


def test_same_bits_again(lib):
    """Two streams at once and a call after another: the same bits."""
    a = Prefill(lib, 128, 8, 2, 700, 2, [(0, 100, 300), (1, 5, 200)])
    assert a.call() == 0
    torch.cuda.synchronize()
    want = a.o.clone()
    b = Prefill(lib, 64, 8, 2, 700, 1, [(0, 100, 300)])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(s1):
            assert a.call() == 0
        with torch.cuda.stream(s2):
            assert b.call() == 0
    torch.cuda.synchronize()
    assert torch.equal(a.o, want)
    b.check()
