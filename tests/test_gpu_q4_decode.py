"""Decode attention over a Q4_0 cache, held to the precision of its definition
whatever the sizes of q, K and V.

Tolerances.  A score sums a block's codes and its offset 8 sum(q) in six steps of
2^-23 of magnitudes up to (15 + 8) sum |q|, times d, and the blocks in as many
steps; q enters with 22 bits, each of two parts half a step off.  A weight takes
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
