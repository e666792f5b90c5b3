"""Decode attention over a Q4_0 cache, held to the precision of its definition
whatever the sizes of q, K and V.

Tolerances.  A score sums a block's codes and its offset 8 sum(q) in six steps of
2^-23 of magnitudes up to (15 + 8) sum |q|, times d, and the blocks in as many
steps; q enters with 22 bits, or two parts of half a subnormal step each, 2^-39 of
its head's largest element.  A weight takes
2^-21 (two parts and the exponential) and the rounding of its exponent, 2^-22 of
the largest score in base 2, twice.  Its products with V's scale are held to 2^-38
of the largest scale, times |c - 8| <= 8 and the number of cells.  O sums 16 keys
in a step of 2^-23, joined over warps and splits.  All of it enters numerators and
denominator: twice, times sum p |v|.  Then o's rounding, half a step."""
import numpy as np
import pytest
import torch

from oracle import llama as O
from q4_util import pack_cache
from test_gpu_q4 import dev, ints, make_cache, reference, stream, visible_cells
from test_gpu_q4_prefill import half_step

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -23


@pytest.fixture(scope="module")
def lib():
    import llama_decoder_forward_02_gb300 as L
    return L


class Decode:
    """n_ctx cells of which a row sees those up to pos (window: the last of them); q of size qs, K of size ks, V of size
    vs; dominant: every head has a cell that takes nearly all of its weight; mixed: V's cells differ in size by 1e4."""

    def __init__(self, lib, hd, H, Hkv, n_ctx, pos, seq, window=0, qs=1.5, ks=1.0, vs=1.0, dominant=False, mixed=False, seed=0):
        rng = np.random.default_rng(seed + hd + H + n_ctx)
        n_seq, T, G = max(seq) + 1, len(pos), H // Hkv
        self.lib, self.shape, self.window = lib, (T, H, Hkv, hd, n_ctx, n_seq), window
        vis = visible_cells(pos, seq, n_seq, n_ctx, window)
        (kc, kd), (vc, vd) = (make_cache(rng, n_seq, Hkv, n_ctx, hd, vis) for _ in range(2))
        size = np.exp(rng.uniform(-9, 0, (n_seq, Hkv, n_ctx, 1))) if mixed else 1.0
        kd, vd = (kd * np.float64(ks)).astype(np.float16), (vd * (size * vs)).astype(np.float16)
        k, v = O.dequantize_q4_0(kc, kd), O.dequantize_q4_0(vc, vd)
        q = rng.standard_normal((T, H, hd)) * qs
        if dominant:
            for t in range(T):
                for h in range(H):
                    c = k[seq[t], h // G, rng.integers(max(0, pos[t] + 1 - window) if window else 0, pos[t] + 1)]
                    q[t, h] = c * (16.0 * np.sqrt(hd) / (c * c).sum()) + 0.3 / ks * rng.standard_normal(hd) / np.sqrt(hd)
        q32 = q.astype(np.float32)
        q = q32.astype(np.float64)
        self.ref = reference(q, k, v, pos, seq, Hkv, window)
        kz, vz, kdz, vdz = (np.where(vis[:, None, :, None], np.abs(u.astype(np.float64)), 0) for u in (k, v, kd, vd))
        mag = top = qk = 0.0
        for t in range(T):
            qb = np.abs(q[t]).reshape(Hkv, G, hd // 32, 32).sum(-1)
            mag = max(mag, 23 * np.einsum("jgb,jcb->jgc", qb, kdz[seq[t]]).max() / np.sqrt(hd))
            qk = max(qk, np.einsum("jgd,jcd->jgc", np.abs(q[t]).reshape(Hkv, G, hd), kz[seq[t]]).max() / np.sqrt(hd))
        top = qk * 1.4426950408889634
        low = 2.0 ** -38 * np.abs(q).max(-1, keepdims=True) * np.ones(hd)
        for t in range(T):
            qk = max(qk, 2.0 ** 21 * np.einsum("jgd,jcd->jgc", low[t].reshape(Hkv, G, hd), kz[seq[t]]).max() / np.sqrt(hd))
        w = (6 + hd // 32) * U32 * mag + 2.0 ** -21 * qk + 2.0 ** -21 + 2.0 ** -21 * top + (n_ctx / 128 + 160) * U32
        mean = reference(q, k, vz, pos, seq, Hkv, window)
        seen = np.minimum(np.array(pos) + 1, window) if window else np.array(pos) + 1
        off = 2 * w * mean + 2.0 ** -35 * vdz.max() * seen[:, None, None]
        self.tol = half_step(np.abs(self.ref) + off) + off
        self.qd, self.kc, self.vc = dev(q32), dev(pack_cache(kc, kd)), dev(pack_cache(vc, vd))
        self.posd, self.seqd = ints(pos), ints(seq)
        self.o = torch.full((T, H * hd), 9.0, dtype=torch.float16, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        n = lib.llm_op_attn_decode_q4_0_scratch_bytes(T, H, Hkv, hd, n_ctx, n_seq)
        self.scratch = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def check(self):
        T, H, Hkv, hd, n_ctx, n_seq = self.shape
        assert self.lib.llm_op_attn_decode_q4_0(
            self.qd.data_ptr(), self.kc.data_ptr(), self.vc.data_ptr(), self.posd.data_ptr(), self.seqd.data_ptr(),
            self.o.data_ptr(), T, H, Hkv, hd, n_ctx, n_seq, self.window, self.scratch.data_ptr(), self.scratch.numel(),
            self.err.data_ptr(), stream()) == 0, self.lib.llm_last_error(None)
        torch.cuda.synchronize()
        off = np.abs(self.o.cpu().double().numpy().reshape(self.ref.shape) - self.ref)
        assert np.all(off <= self.tol), (off / self.tol).max()
        assert int(self.err) == 0


LONG = dict(n_ctx=30000, pos=[29999], seq=[0])
SHORT = dict(n_ctx=2100, pos=[2099, 700], seq=[0, 1])


@pytest.mark.parametrize("hd,H,Hkv", [(128, 8, 2), (64, 8, 1), (32, 4, 2)])
@pytest.mark.parametrize("where", [LONG, SHORT])
@pytest.mark.parametrize("vs", [1.0, 1e-2, 1e-3, 200.0])
@pytest.mark.parametrize("dominant", [False, True])
def test_sizes_of_v(lib, hd, H, Hkv, where, vs, dominant):
    """The weights keep their bits whatever V's size and however they are spread."""
    Decode(lib, hd, H, Hkv, vs=vs, dominant=dominant, **where).check()


@pytest.mark.parametrize("hd,H,Hkv", [(128, 4, 1), (64, 12, 2), (32, 4, 2)])
def test_cells_of_unlike_sizes(lib, hd, H, Hkv):
    """V's scales grow and shrink along the cache, a factor of 1e4 apart."""
    Decode(lib, hd, H, Hkv, mixed=True, **LONG).check()
    Decode(lib, hd, H, Hkv, mixed=True, dominant=True, window=900, **SHORT).check()


@pytest.mark.parametrize("hd,H,Hkv", [(128, 8, 2), (64, 12, 1), (32, 4, 2)])
@pytest.mark.parametrize("qs,ks", [(1e5, 1e-5), (4e4, 4e-5), (1e-6, 2000.0), (1e-30, 1.0), (1e30, 0.0)])
def test_sizes_of_q(lib, hd, H, Hkv, qs, ks):
    """Queries far beyond fp16's range, and far below it, over keys that make their scores ordinary ones."""
    for where in (LONG, SHORT):
        Decode(lib, hd, H, Hkv, qs=qs, ks=ks, **where).check()


def test_heads_of_unlike_queries(lib):
    """Each head's queries are held by their own largest: a head of zeros, tiny ones, huge ones, and one whose largest
    element meets keys of zero."""
    hd, H, Hkv = 64, 8, 2
    c = Decode(lib, hd, H, Hkv, qs=0.0, **SHORT)
    rng = np.random.default_rng(5)
    n_seq, n_ctx = 2, SHORT["n_ctx"]
    (kc, kd), (vc, vd) = (make_cache(rng, n_seq, Hkv, n_ctx, hd, np.ones((n_seq, n_ctx), bool)) for _ in range(2))
    kc[..., 7] = 8                                              # keys' element 7: 0
    kd = (kd * 1e-2).astype(np.float16)
    q = rng.standard_normal((2, H, hd)) * np.array([0.0, 1e-20, 1e2, 3e3, 1.0, 1e2, 1e-3, 1e2])[None, :, None]
    q[:, 5, 7] = 1e6
    q = q.astype(np.float32)
    k, v = O.dequantize_q4_0(kc, kd), O.dequantize_q4_0(vc, vd)
    q64 = q.astype(np.float64)
    ref = reference(q64, k, v, SHORT["pos"], SHORT["seq"], Hkv, 0)
    qb = np.abs(q64).reshape(2, Hkv, 4, 2, 32).sum(-1)
    # by head: the bound of the head of this file
    mag = 23 * np.stack([np.einsum("jgb,jcb->jgc", qb[t], np.abs(kd[t].astype(np.float64))).max(-1).reshape(-1) for t in range(2)]) / 8
    qk = np.stack([np.einsum("jgd,jcd->jgc", (np.abs(q64[t]) + 2.0 ** -17 * np.abs(q64[t]).max(-1, keepdims=True)).reshape(
        Hkv, 4, hd), np.abs(k[t])).max(-1).reshape(-1) for t in range(2)]) / 8
    w = 8 * U32 * mag + 2.0 ** -20 * qk * 1.5 + 2.0 ** -21 + (n_ctx / 128 + 160) * U32
    off = 2 * w[..., None] * reference(q64, k, np.abs(v), SHORT["pos"], SHORT["seq"], Hkv, 0)
    off = off + 2.0 ** -35 * np.abs(vd.astype(np.float64)).max() * (np.array(SHORT["pos"]) + 1)[:, None, None]
    c.ref, c.tol = ref, half_step(np.abs(ref) + off) + off
    c.qd, c.kc, c.vc = dev(q.reshape(2, -1)), dev(pack_cache(kc, kd)), dev(pack_cache(vc, vd))
    c.check()


@pytest.mark.parametrize("odd", [2.0 ** 118, np.inf, np.nan])
def test_queries_out_of_range_stay_in_their_head(lib, odd):
    c = Decode(lib, 128, 8, 2, **SHORT)
    q = c.qd.cpu().numpy()
    q[0, 3, 40] = odd
    c.qd.copy_(torch.from_numpy(q))
    want = c.ref.copy()
    c.ref[0, 3] = 0.0
    c.tol[0, 3] = np.inf
    T, H, Hkv, hd, n_ctx, n_seq = c.shape
    assert lib.llm_op_attn_decode_q4_0(c.qd.data_ptr(), c.kc.data_ptr(), c.vc.data_ptr(), c.posd.data_ptr(), c.seqd.data_ptr(),
                                       c.o.data_ptr(), T, H, Hkv, hd, n_ctx, n_seq, 0, c.scratch.data_ptr(), c.scratch.numel(),
                                       c.err.data_ptr(), stream()) == 0
    got = c.o.cpu().double().numpy().reshape(want.shape)
    assert np.all(np.isnan(got[0, 3]))
    got[0, 3] = 0.0
    assert np.all(np.abs(got - c.ref) <= c.tol)
