"""The 4-bit operators on the GPU against their definitions in float64: Q4_0
weights and their GEMV, the per-head query/key norm with rotation and cache
append, and attention over a Q4_0 cache.

Tolerances are worst-case bounds of the arithmetic: half a step of the output
type, and for the fp32 sums 2^-23 a step (tensor cores add by truncation) of
the sum of magnitudes."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import llama as O
from q4_util import pack_cache, pack_weights, unpack_cache

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -11, 2.0 ** -23


@pytest.fixture(scope="module")
def lib():
    import llama_decoder_forward_02_gb300 as L
    return L


def stream():
    return torch.cuda.current_stream().cuda_stream


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- weights

@pytest.mark.parametrize("N,K", [(1, 256), (5, 512), (67, 2816), (300, 4096)])
def test_quantize_bit_exact(lib, N, K):
    rng = np.random.default_rng(N + K)
    w = (rng.standard_normal((N, K)) * np.exp(rng.uniform(-9, 3, (N, 1)))).astype(np.float16)
    w[0, 32:64] = 0                                            # a block of zeros
    w[0, 64:96] = np.float16(0.25)                             # equals: all at the first's code
    w[-1, :32] = np.arange(-16, 16) / 2                        # ties of the rounding
    w[-1, 96] = np.float16(6e-8)                               # a scale below fp16's steps
    w[-1, 97:128] = 0
    c, d = O.quantize_q4_0(w)
    W, out = dev(w), torch.full((N * K // 16 * 9 + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    assert lib.llm_op_quantize_q4_0(W.data_ptr(), N, K, out.data_ptr(), stream()) == 0
    got = out.cpu().numpy()
    assert np.array_equal(got[:-64], pack_weights(c, d).reshape(-1)) and np.all(got[-64:] == 0xAB)
    assert torch.equal(W.cpu(), torch.from_numpy(w))


def gemv_case(N, K, T, seed, xs=1.0):
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 16, (N, K)).astype(np.uint8)
    d = (rng.standard_normal((N, K // 32)) * 0.01).astype(np.float16)
    d[:, 0] = 0
    x = (rng.standard_normal((T, K)) * xs).astype(np.float16)
    ref = x.astype(np.float64) @ O.dequantize_q4_0(c, d).T
    # codes and the offset 8 are summed apart: |c| + 8 <= 23 a product; 2 + K / 32 steps of the sums
    mag = np.abs(x).astype(np.float64) @ np.repeat(np.abs(d).astype(np.float64), 32, 1).T * 23
    return c, d, x, ref, mag * U32 * (8 + K // 32)


@pytest.mark.parametrize("N,K,T,pad", [
    (1, 256, 1, 0), (7, 256, 8, 8), (33, 512, 3, 0), (64, 2048, 2, 0), (1000, 2816, 5, 16), (4096, 4096, 1, 0),
    (2049, 4096, 8, 0), (513, 14336, 8, 0), (96, 16384, 1, 8), (31, 6400, 4, 0), (10007, 1024, 7, 0), (20000, 768, 6, 0),
])
def test_gemv(lib, N, K, T, pad):
    c, d, x, ref, tol = gemv_case(N, K, T, N + K + T)
    ldx, ldy = K + pad, N + pad // 8
    xp = np.full((T, ldx), np.float16(np.nan))
    xp[:, :K] = x
    W, xd = dev(pack_weights(c, d)), dev(xp)
    y = torch.full((T, ldy), 7.0, device="cuda")
    for _ in range(2):
        assert lib.llm_op_gemv_q4_0(W.data_ptr(), xd.data_ptr(), y.data_ptr(), N, K, T, ldx, ldy, stream()) == 0
        got = y.cpu().double().numpy()
        assert np.all(np.abs(got[:, :N] - ref) <= tol), np.abs(got[:, :N] - ref).max()
        assert np.all(got[:, N:] == 7.0)


@pytest.mark.parametrize("xs", [1e-5, 3e-3, 8000.0])
def test_gemv_magnitudes(lib, xs):
    """x among fp16's subnormals and near its top: the sums keep fp32 precision."""
    N, K, T = 77, 1024, 3
    c, d, x, ref, tol = gemv_case(N, K, T, 5, xs)
    x = np.clip(x, -65504, 65504)
    W, xd, y = dev(pack_weights(c, d)), dev(x), torch.zeros((T, N), device="cuda")
    assert lib.llm_op_gemv_q4_0(W.data_ptr(), xd.data_ptr(), y.data_ptr(), N, K, T, K, N, stream()) == 0
    assert np.all(np.abs(y.cpu().double().numpy() - ref) <= tol)


def test_gemv_nan_stays_in_its_row(lib):
    """A NaN in one row of x reaches that row's outputs only."""
    N, K, T = 40, 512, 4
    c, d, x, ref, tol = gemv_case(N, K, T, 6)
    x[2, 100] = np.nan
    W, xd, y = dev(pack_weights(c, d)), dev(x), torch.zeros((T, N), device="cuda")
    assert lib.llm_op_gemv_q4_0(W.data_ptr(), xd.data_ptr(), y.data_ptr(), N, K, T, K, N, stream()) == 0
    got = y.cpu().double().numpy()
    rows = [0, 1, 3]
    assert np.all(np.isnan(got[2])) and np.all(np.abs(got[rows] - ref[rows]) <= tol[rows])


# ---------------------------------------------------------------- norm, rotation, append

def qk_reference(x, gq, gk, eps, table, pos, H, Hkv, hd):
    """q, k, v rows [T][heads][hd] in float64."""
    x = x.astype(np.float64)[:, :(H + 2 * Hkv) * hd].reshape(len(pos), -1, hd)
    parts = [x[:, :H], x[:, H:H + Hkv]]
    cs = table.astype(np.float64)[pos][:, None]
    out = []
    for p, g in zip(parts, (gq, gk)):
        if g is not None:
            p = p / np.sqrt((p * p).mean(-1, keepdims=True) + eps) * g.astype(np.float64)
        a, b = p[..., 0::2], p[..., 1::2]
        r = np.empty_like(p)
        r[..., 0::2], r[..., 1::2] = a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]
        out.append(r)
    return out[0], out[1], x[:, H + Hkv:]


def rope_table(n_ctx, hd, theta=10000.0):
    a = np.arange(n_ctx)[:, None] * theta ** (-np.arange(0, hd, 2) / hd)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def run_qk(lib, x, ld, gq, gk, eps, table, pos, seq, qt, kc, vc, kt, H, Hkv, hd, n_ctx, n_seq, err):
    T = len(pos)
    q = torch.full((T, H * hd), 3.0, dtype=torch.float16 if qt else torch.float32, device="cuda")
    xd, td = dev(x), dev(table)
    g = [None if v is None else dev(v) for v in (gq, gk)]
    posd, seqd = ints(pos), ints(seq)
    rc = lib.llm_op_qk_norm_rope(xd.data_ptr(), ld, *[0 if v is None else v.data_ptr() for v in g], eps, td.data_ptr(),
                                 posd.data_ptr(), seqd.data_ptr(), q.data_ptr(), qt, kc.data_ptr(), vc.data_ptr(),
                                 kt, T, H, Hkv, hd, n_ctx, n_seq, err.data_ptr() if err is not None else 0, stream())
    assert rc == 0, lib.llm_last_error(None)
    torch.cuda.synchronize()
    return q.cpu().double().numpy().reshape(T, H, hd)


@pytest.mark.parametrize("hd,H,Hkv,T,pad,norm,qt,kt", [
    (128, 32, 8, 3, 0, "qk", 0, 0), (128, 8, 1, 40, 12, "qk", 1, 2), (64, 6, 2, 17, 0, "qk", 0, 2),
    (32, 4, 2, 33, 4, "qk", 1, 2), (32, 5, 5, 1, 0, None, 0, 2), (64, 3, 1, 9, 0, "q", 0, 1), (32, 2, 1, 2, 0, "k", 1, 0),
    (128, 40, 8, 300, 0, "qk", 1, 2), (64, 8, 8, 64, 0, None, 1, 1),
])
def test_qk_norm_rope(lib, hd, H, Hkv, T, pad, norm, qt, kt):
    rng = np.random.default_rng(hd + H + T)
    n_ctx, n_seq, eps = T + 20, 3, 1e-5
    ld = (H + 2 * Hkv) * hd + pad
    x = (rng.standard_normal((T, ld)) * np.exp(rng.uniform(-2, 2, (T, 1)))).astype(np.float32)
    gq, gk = [(1 + 0.2 * rng.standard_normal(hd)).astype(np.float32) if norm and n in norm else None for n in "qk"]
    seq = np.sort(rng.integers(0, n_seq, T))
    pos = np.array([5 + int((seq[:t] == seq[t]).sum()) for t in range(T)])
    table = rope_table(n_ctx, hd)
    rq, rk, rv = qk_reference(x, gq, gk, eps, table, pos, H, Hkv, hd)
    size = n_seq * Hkv * n_ctx * hd * 2 if kt == 0 else n_seq * Hkv * n_ctx * hd if kt == 1 else \
        lib.llm_op_kv_q4_0_bytes(Hkv, hd, n_ctx, n_seq)
    kc, vc = (torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = run_qk(lib, x[:, :], ld, gq, gk, eps, table, pos, seq, qt, kc, vc, kt, H, Hkv, hd, n_ctx, n_seq, err)
    assert int(err) == 0
    # fp32: a sum of hd squares, a root, a division, two products and a rotation: 16 half steps of the pair's length
    pair = lambda r: np.repeat(np.hypot(r[..., 0::2], r[..., 1::2]), 2, -1)  # noqa: E731
    f32 = lambda r: 16 * 2.0 ** -24 * pair(r)  # noqa: E731
    assert np.all(np.abs(q - rq) <= f32(rq) + (U16 * np.abs(rq) + 2.0 ** -25 if qt else 0))
    for cache, ref, tol in ((kc, rk, f32(rk)), (vc, rv, 0 * rv)):
        raw = cache.cpu().numpy()
        touched = np.zeros((n_seq, Hkv, n_ctx), bool)
        touched[seq, :, pos] = True
        if kt == 2:
            c, d = unpack_cache(raw, n_seq, Hkv, n_ctx, hd)
            rc, rd = O.quantize_q4_0(ref)
            assert np.array_equal(c[seq, :, pos], rc)
            assert np.all(np.abs(d[seq, :, pos].astype(float) - rd.astype(float)) <= np.abs(rd.astype(float)) * 2.0 ** -10 + 2.0 ** -24)
            assert np.all(pack_cache(c, d) == raw)
            junk_c, junk_d = unpack_cache(np.full_like(raw, 0x5A), n_seq, Hkv, n_ctx, hd)
            assert np.array_equal(c[~touched], junk_c[~touched]) and np.array_equal(d[~touched].view(np.int16),
                                                                                  junk_d[~touched].view(np.int16))
        else:
            el = 2 if kt == 0 else 1
            got = raw.reshape(n_seq, Hkv, n_ctx, hd * el)
            assert np.all(got[~touched] == 0x5A)
            t = torch.from_numpy(np.ascontiguousarray(got[seq, :, pos])).view(
                torch.float16 if kt == 0 else torch.float8_e4m3fn).float().double().numpy()
            # half a step: 2^-11 of fp16, 2^-4 of E4M3 (2^-10 absolute among its subnormals)
            rel, low = (U16, 2.0 ** -25) if kt == 0 else (2.0 ** -4, 2.0 ** -10)
            assert np.all(np.abs(t - np.clip(ref, -448, 448) if kt else t - ref) <= tol * (1 + rel) + rel * np.abs(ref) + low)


def test_append_codes_at_borders(lib):
    """Values on a border between two codes (ties) and a ulp beside it, equal magnitudes of both signs, zeros."""
    hd, Hkv, T, n_ctx = 64, 1, 6, 8
    x = np.zeros((T, 3 * hd), np.float32)
    v = x[:, 2 * hd:]
    steps = np.arange(-7.5, 8.0, 1.0, dtype=np.float32)         # 16 borders of d = -1 (m = 8)
    for t, f in enumerate((1.0, 1 + 2.0 ** -23, 1 - 2.0 ** -24)):
        v[t, :16] = steps * np.float32(f)
        v[t, 16] = 8.0
        v[t, 32:48] = -steps * np.float32(f)
        v[t, 40] = -8.0
    v[3, :2] = [-3.0, 3.0]
    v[3, 32:34] = [3.0, -3.0]
    v[4, 5] = 1e-30                                              # a scale that fp16 holds as zero
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(lib.llm_op_kv_q4_0_bytes(Hkv, hd, n_ctx, 1), dtype=torch.uint8, device="cuda") for _ in range(2))
    run_qk(lib, x, 3 * hd, None, None, 1e-5, rope_table(n_ctx, hd), list(range(T)), [0] * T, 0, kc, vc, 2, 1, 1, hd, n_ctx, 1, err)
    c, d = unpack_cache(vc.cpu().numpy(), 1, 1, n_ctx, hd)
    rc, rd = O.quantize_q4_0(v)
    assert np.array_equal(c[0, 0, :T], rc) and np.array_equal(d[0, 0, :T], rd) and int(err) == 0


@pytest.mark.parametrize("hd,scale", [(128, 1.0), (64, 3e-32), (32, 700.0), (64, 2e-36)])
def test_append_rotated_codes_at_borders(lib, hd, scale):
    """Keys whose rotated values lie within float32's rounding of a code border: the exact value's side counts."""
    rng = np.random.default_rng(hd)
    Hkv, T, n_ctx = 2, 96, 128
    table = rope_table(n_ctx, hd)
    pos = np.arange(T)
    cs = table.astype(np.float64)[pos][:, None].repeat(Hkv, 1)                      # [T][Hkv][hd / 2][2]
    x = (rng.uniform(-1, 1, (T, Hkv, hd)) * scale).astype(np.float32)
    x[..., 0::32] *= 40                                                             # a block's largest
    c, s = cs[..., 0], cs[..., 1]
    rot = lambda v: (v[..., 0::2] * c - v[..., 1::2] * s, v[..., 0::2] * s + v[..., 1::2] * c)  # noqa: E731
    for _ in range(2):
        even, odd = rot(x.astype(np.float64))
        full = np.stack([even, odd], -1).reshape(T, Hkv, hd // 32, 32)
        top = np.take_along_axis(full, np.abs(full).argmax(-1)[..., None], -1)
        d = np.repeat((top / -8).reshape(T, Hkv, -1), 16, -1)
        border = (rng.integers(-8, 7, d.shape) + 0.5) * d
        a = ((border + x[..., 1::2].astype(np.float64) * s) / c).astype(np.float32)
        keep = (np.arange(hd // 2) % 16 == 0) | (np.abs(c) < 0.3) | (np.abs(a) > 30 * scale)
        x[..., 0::2] = np.where(keep, x[..., 0::2], a)
    H = 2
    qkv = np.zeros((T, (H + 2 * Hkv) * hd), np.float32)
    qkv[:, H * hd:(H + Hkv) * hd] = x.reshape(T, -1)
    kc, vc = (torch.zeros(lib.llm_op_kv_q4_0_bytes(Hkv, hd, n_ctx, 1), dtype=torch.uint8, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_qk(lib, qkv, qkv.shape[1], None, None, 1e-5, table, pos, [0] * T, 0, kc, vc, 2, H, Hkv, hd, n_ctx, 1, err)
    ref = qk_reference(qkv, None, None, 1e-5, table, pos, H, Hkv, hd)[1]
    rc, rd = O.quantize_q4_0(ref)
    exact = np.abs(ref.reshape(T, Hkv, -1, 32) / np.repeat(np.abs(ref.reshape(T, Hkv, -1, 32)).max(-1, keepdims=True), 32, -1) * 8)
    assert (np.abs(exact % 1 - 0.5) < 1e-6).mean() > 0.2                            # the borders are met
    got, gd = unpack_cache(kc.cpu().numpy(), 1, Hkv, n_ctx, hd)
    assert np.array_equal(got[0, :, :T], rc.swapaxes(0, 1)) and int(err) == 0
    assert np.all(np.abs(gd[0, :, :T].astype(float) - rd.swapaxes(0, 1).astype(float)) <= np.abs(rd.swapaxes(0, 1)) * 2.0 ** -10 + 2.0 ** -24)


@pytest.mark.parametrize("kt", [0, 2])
def test_rows_outside_the_cache_and_range(lib, kt):
    """Rows whose cell does not exist are reported and append nothing; so is a value beyond fp16; other rows are as usual."""
    hd, H, Hkv, n_ctx, n_seq = 64, 4, 2, 16, 2
    rng = np.random.default_rng(1)
    pos, seq = [3, 16, -1, 4, 5], [0, 0, 1, 2, 1]
    x = rng.standard_normal((5, (H + 2 * Hkv) * hd)).astype(np.float32)
    size = n_seq * Hkv * n_ctx * hd * 2 if kt == 0 else lib.llm_op_kv_q4_0_bytes(Hkv, hd, n_ctx, n_seq)
    kc, vc = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = rope_table(n_ctx, hd)
    q = run_qk(lib, x, x.shape[1], None, None, 1e-5, table, pos, seq, 0, kc, vc, kt, H, Hkv, hd, n_ctx, n_seq, err)
    assert int(err) == 2
    safe = np.clip(pos, 0, n_ctx - 1)
    rq, _, _ = qk_reference(x, None, None, 1e-5, table, safe, H, Hkv, hd)
    for t in (1, 2, 3):
        assert np.all(q[t] == 0)
    for t in (0, 4):
        assert np.abs(q[t] - rq[t]).max() <= 16 * 2.0 ** -24 * np.abs(rq[t]).max() * 2
    if kt == 2:
        c, d = unpack_cache(vc.cpu().numpy(), n_seq, Hkv, n_ctx, hd)
        used = (d != 0).any(-1)
    else:
        used = (vc.view(torch.float16).view(n_seq, Hkv, n_ctx, hd) != 0).any(-1).cpu().numpy()
    assert used[0, :, 3].all() and used[1, :, 5].all() and used.sum() == 2 * Hkv
    err.zero_()
    x[4, -1] = 7e4
    run_qk(lib, x[4:], x.shape[1], None, None, 1e-5, table, [6], [1], 0, kc, vc, kt, H, Hkv, hd, n_ctx, n_seq, err)
    assert int(err) == 8


# ---------------------------------------------------------------- attention

def make_cache(rng, n_seq, Hkv, n_ctx, hd, visible):
    """A Q4_0 cache; cells outside `visible` ([n_seq][n_ctx] bool) hold NaN and infinite scales."""
    c, d = O.quantize_q4_0(rng.standard_normal((n_seq, Hkv, n_ctx, hd)))
    junk = np.where(rng.random(d.shape) < 0.5, np.float16(np.nan), np.float16(np.inf))
    d = np.where(visible[:, None, :, None], d, junk).astype(np.float16)
    return c, d


def reference(q, kc, vc, pos, seq, Hkv, window):
    """q [T][H][hd]; each row over its own visible cells, float64."""
    out = np.zeros_like(q)
    for t in range(len(pos)):
        lo = max(0, pos[t] + 1 - window) if window else 0
        cells = np.arange(lo, pos[t] + 1)
        k, v = (u[seq[t]][:, cells].transpose(1, 0, 2) for u in (kc, vc))
        out[t:t + 1] = O.attention_one_seq(q[t:t + 1], k, v, np.array([pos[t]]), cells, Hkv)
    return out


def score_tol(q, k, hd, bits):
    """Worst error of a softmax weight, relative: exp of the score's error, whose products carry 2^-bits and
    whose sum hd + 16 steps of 2^-23."""
    mag = np.abs(q).sum(-1).max() * np.abs(k[np.isfinite(k)]).max() / np.sqrt(hd)
    return 2 * mag * (2.0 ** -bits + (hd + 16) * U32)


def visible_cells(pos, seq, n_seq, n_ctx, window):
    vis = np.zeros((n_seq, n_ctx), bool)
    for p, s in zip(pos, seq):
        vis[s, (max(0, p + 1 - window) if window else 0):p + 1] = True
    return vis


class Decode:
    def __init__(self, lib, hd, H, Hkv, n_ctx, n_seq, pos, seq, window=0, seed=0, scale=1.5):
        rng = np.random.default_rng(seed + hd + H + n_ctx)
        self.lib, self.hd, self.H, self.Hkv, self.n_ctx, self.n_seq, self.window = lib, hd, H, Hkv, n_ctx, n_seq, window
        self.pos, self.seq, self.T = pos, seq, len(pos)
        vis = visible_cells(pos, seq, n_seq, n_ctx, window)
        (kc, kd), (vc, vd) = (make_cache(rng, n_seq, Hkv, n_ctx, hd, vis) for _ in range(2))
        self.q = (rng.standard_normal((self.T, H * hd)) * scale).astype(np.float32)
        k, v = O.dequantize_q4_0(kc, kd), O.dequantize_q4_0(vc, vd)
        q = self.q.astype(np.float64).reshape(self.T, H, hd)
        self.ref = reference(q, k, v, pos, seq, Hkv, window).reshape(self.T, -1)
        vmax = np.abs(v[np.isfinite(v)]).max()
        # fp16 output; weights and values held to 22 bits
        self.tol = U16 * np.abs(self.ref) + 2.0 ** -25 + 2 * (score_tol(q, k, hd, 21) + 2.0 ** -20) * vmax
        self.qd, self.kc, self.vc = dev(self.q), dev(pack_cache(kc, kd)), dev(pack_cache(vc, vd))
        self.posd, self.seqd = ints(pos), ints(seq)
        self.o = torch.full((self.T, H * hd), 9.0, dtype=torch.float16, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scratch = torch.zeros(lib.llm_op_attn_decode_q4_0_scratch_bytes(self.T, H, Hkv, hd, n_ctx, n_seq),
                                   dtype=torch.uint8, device="cuda")

    def call(self, st=None):
        rc = self.lib.llm_op_attn_decode_q4_0(
            self.qd.data_ptr(), self.kc.data_ptr(), self.vc.data_ptr(), self.posd.data_ptr(), self.seqd.data_ptr(),
            self.o.data_ptr(), self.T, self.H, self.Hkv, self.hd, self.n_ctx, self.n_seq, self.window,
            self.scratch.data_ptr(), self.scratch.numel(), self.err.data_ptr(), stream() if st is None else st)
        assert rc == 0, self.lib.llm_last_error(None)

    def check(self):
        torch.cuda.synchronize()
        got = self.o.cpu().double().numpy()
        assert np.all(np.abs(got - self.ref) <= self.tol), np.nanmax(np.abs(got - self.ref) - self.tol)


@pytest.mark.parametrize("hd,H,Hkv,n_ctx,pos,seq,window", [
    (128, 32, 8, 1, [0], [0], 0),                                         # one cell
    (128, 32, 8, 2304, [2047], [0], 0),
    (128, 8, 2, 300, [0, 299, 150, 16], [0, 1, 1, 0], 0),
    (64, 32, 8, 640, [511, 600, 3, 64, 65, 127, 128, 639], [0, 1, 2, 3, 0, 1, 2, 3], 0),
    (32, 4, 2, 64, [15], [0], 0), (32, 4, 4, 96, [95, 40], [0, 0], 0),
    (128, 8, 1, 200, [199], [0], 0),                                      # eight heads a kv head
    (64, 6, 2, 333, [332, 7], [0, 1], 0), (128, 5, 1, 129, [128], [0], 0),  # odd groups
    (64, 12, 1, 257, [256, 100], [0, 0], 0),                              # more than eight heads a kv head
    (128, 32, 2, 100, [99, 31], [0, 1], 0),
    (128, 16, 4, 700, [699, 50], [0, 1], 33), (64, 8, 2, 700, [699, 350], [0, 1], 1), (32, 4, 1, 500, [499], [0], 128),
    (128, 4, 2, 5000, [4999], [0], 0),
    (64, 4, 2, 90, list(range(70, 90)), [i % 3 for i in range(20)], 0),   # more than eight rows
    # splits merged through memory: 32 of them, more, and fewer than were launched
    (64, 32, 8, 10000, [9999], [0], 0), (128, 8, 2, 9000, [8999], [0], 0), (128, 5, 1, 9000, [8000, 130], [0, 0], 0),
    (32, 8, 2, 8300, [8299, 20, 4000], [0, 0, 0], 5000),
])
def test_attn_decode(lib, hd, H, Hkv, n_ctx, pos, seq, window):
    c = Decode(lib, hd, H, Hkv, n_ctx, max(seq) + 1, pos, seq, window)
    for _ in range(2):                                                     # the scratch is left ready
        c.call()
        c.check()
    assert int(c.err) == 0


@pytest.mark.parametrize("scale", [0.0, 1e-4, 60.0])
def test_attn_decode_score_ranges(lib, scale):
    """Flat weights, and weights that a few cells take whole."""
    c = Decode(lib, 128, 8, 2, 900, 1, [899], [0], scale=scale)
    c.call()
    c.check()


def test_attn_decode_rows_outside(lib):
    pos, seq = [100, 256, 50, -1, 9], [0, 0, 2, 1, 1]
    ok = [0, 4]
    c = Decode(lib, 64, 8, 2, 256, 2, [100, 9], [0, 1])
    o = torch.full((5, 8 * 64), 9.0, dtype=torch.float16, device="cuda")
    q = dev(np.concatenate([c.q[:1], np.zeros((3, 512), np.float32), c.q[1:]]))
    p, s = ints(pos), ints(seq)
    scratch = torch.zeros(lib.llm_op_attn_decode_q4_0_scratch_bytes(5, 8, 2, 64, 256, 2), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        c.err.zero_()
        assert lib.llm_op_attn_decode_q4_0(q.data_ptr(), c.kc.data_ptr(), c.vc.data_ptr(), p.data_ptr(), s.data_ptr(),
                                           o.data_ptr(), 5, 8, 2, 64, 256, 2, 0, scratch.data_ptr(), scratch.numel(),
                                           c.err.data_ptr(), stream()) == 0
        got = o.cpu().double().numpy()
        assert int(c.err) == 2 and np.all(got[1:4] == 0)
        assert np.all(np.abs(got[ok] - c.ref) <= c.tol)


def shared(n, n_ctx, seed):
    """Positions of n rows, among them the first, the last and short ones."""
    pos = np.random.default_rng(seed).integers(0, n_ctx, n)
    pos[0], pos[-1], pos[n // 2] = n_ctx - 1, 0, 15
    return [int(p) for p in pos]


@pytest.mark.parametrize("hd,H,Hkv,n_ctx,T,window", [
    (128, 8, 2, 8300, 3, 0), (128, 8, 8, 8200, 2, 0), (64, 8, 2, 8200, 33, 0), (32, 2, 1, 8200, 128, 0),
    (32, 2, 1, 8200, 129, 0), (64, 16, 2, 8300, 5, 0), (32, 40, 2, 8200, 9, 3000), (128, 4, 1, 40000, 2, 0),
])
def test_attn_decode_rows_share_splits(lib, hd, H, Hkv, n_ctx, T, window):
    """Rows of unlike lengths over a long cache: each takes its share of the launch."""
    c = Decode(lib, hd, H, Hkv, n_ctx, 2, shared(T, n_ctx, T), [i % 2 for i in range(T)], window)
    for _ in range(2):
        c.call()
        c.check()
    # equal rows, and one long row among empty ones
    for pos in ([n_ctx - 1] * T, [1] * (T - 1) + [n_ctx - 1]):
        c.posd.copy_(ints(pos))
        got = []
        for _ in range(2):
            c.call()
            got.append(c.o.cpu().double().numpy())
        assert np.array_equal(*got, equal_nan=True)            # cells hidden in the first call may hold NaN
        if pos[0] == n_ctx - 1:                                # row 0 sees what it saw before
            assert np.all(np.abs(got[0][:1] - c.ref[:1]) <= c.tol[:1])
    assert int(c.err) == 0


def test_attn_decode_rows_outside_share_splits(lib):
    pos, seq, n_ctx = [8300, 8000, -1, 20, 5, 8199], [0, 0, 1, 1, 2, -1], 8300
    c = Decode(lib, 64, 8, 2, n_ctx, 2, [8000, 20], [0, 1])
    q = dev(np.concatenate([np.full((1, 512), np.nan, np.float32), c.q[:1], np.zeros((1, 512), np.float32), c.q[1:],
                            np.ones((2, 512), np.float32)]))
    o = torch.full((6, 512), 9.0, dtype=torch.float16, device="cuda")
    p, s = ints(pos), ints(seq)
    scratch = torch.zeros(lib.llm_op_attn_decode_q4_0_scratch_bytes(6, 8, 2, 64, n_ctx, 2), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        c.err.zero_()
        assert lib.llm_op_attn_decode_q4_0(q.data_ptr(), c.kc.data_ptr(), c.vc.data_ptr(), p.data_ptr(), s.data_ptr(),
                                           o.data_ptr(), 6, 8, 2, 64, n_ctx, 2, 0, scratch.data_ptr(), scratch.numel(),
                                           c.err.data_ptr(), stream()) == 0
        got = o.cpu().double().numpy()
        assert int(c.err) == 2 and np.all(got[[0, 2, 4, 5]] == 0)
        assert np.all(np.abs(got[[1, 3]] - c.ref) <= c.tol)


def test_attn_decode_replayed_with_other_lengths(lib):
    """A captured call takes its splits from the lengths it finds at the replay."""
    a, b = (Decode(lib, 64, 8, 2, 8300, 2, shared(5, 8300, i), [0, 1, 0, 1, 0], seed=i) for i in (3, 4))
    g = torch.cuda.CUDAGraph()
    a.call()
    with torch.cuda.graph(g):
        a.call()
    for x in (a, b):
        for n in ("qd", "kc", "vc", "posd", "seqd"):
            getattr(a, n).copy_(getattr(x, n))
        a.o.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert np.all(np.abs(a.o.cpu().double().numpy() - x.ref) <= x.tol)


FIRST_IN_CAPTURE = """
import sys
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import torch
import test_gpu_q4 as t
import llama_decoder_forward_02_gb300 as lib
d = t.Decode(lib, 64, 8, 2, {n_ctx}, 1, [40], [0])
w = torch.zeros(64, 512, dtype=torch.float16, device="cuda")
q, y = torch.zeros(64 * 288, dtype=torch.uint8, device="cuda"), torch.full((1, 64), 9.0, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    d.call()
    assert lib.llm_op_quantize_q4_0(w.data_ptr(), 64, 512, q.data_ptr(), t.stream()) == 0
    assert lib.llm_op_gemv_q4_0(q.data_ptr(), w.data_ptr(), y.data_ptr(), 64, 512, 1, 512, 64, t.stream()) == 0
g.replay()
d.check()
assert not y.any()
"""


@pytest.mark.parametrize("n_ctx", [64, 9000])
def test_first_calls_of_a_process_captured(lib, n_ctx):
    """The calls' set-up of the device does not disturb a capture that runs before any other call."""
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_IN_CAPTURE.format(root=os.path.dirname(tests), tests=tests, n_ctx=n_ctx)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_attn_decode_scratch_of_any_shape(lib):
    """One scratch, zeroed once, for calls of different shapes in turn."""
    a = Decode(lib, 128, 32, 8, 9000, 1, [8999], [0])
    b = Decode(lib, 64, 8, 2, 8300, 2, shared(9, 8300, 1), [i % 2 for i in range(9)])
    d = Decode(lib, 32, 4, 2, 100, 1, [99, 3], [0, 0])
    size = max(x.scratch.numel() for x in (a, b, d))
    scratch = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for x in (a, b, d):
        x.scratch = scratch
    for x in (a, b, a, d, b, d, a):
        x.o.fill_(9.0)
        x.call()
        x.check()


def test_attn_decode_streams_and_graphs(lib):
    """Two calls at once on two streams, each with its own scratch, and a captured call replayed after its inputs moved."""
    a, b = Decode(lib, 128, 32, 8, 3000, 1, [2999], [0]), Decode(lib, 64, 8, 2, 800, 2, [799, 3], [0, 1], seed=4)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        a.call(s1.cuda_stream)
        b.call(s2.cuda_stream)
    a.check()
    b.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call()
    b.o.fill_(5.0)
    g.replay()
    b.check()
    other = Decode(lib, 64, 8, 2, 800, 2, [500, 640], [1, 0], seed=4)
    for n in ("qd", "kc", "vc", "posd", "seqd"):
        getattr(b, n).copy_(getattr(other, n))
    g.replay()
    torch.cuda.synchronize()
    assert np.all(np.abs(b.o.cpu().double().numpy() - other.ref) <= other.tol)


@pytest.mark.parametrize("hd,H,Hkv,n_ctx,runs,window", [
    (128, 8, 2, 700, [(0, 512)], 0), (128, 4, 1, 300, [(37, 100), (0, 9), (250, 1)], 0), (64, 6, 2, 400, [(100, 300), (0, 77)], 0),
    (32, 4, 2, 200, [(0, 150), (33, 65)], 0), (128, 4, 2, 600, [(300, 200)], 64), (64, 4, 4, 513, [(500, 13), (64, 128)], 1),
    (32, 2, 1, 300, [(128, 140)], 70), (128, 5, 1, 130, [(0, 130)], 0), (64, 2, 1, 1, [(0, 1)], 0),
])
def test_attn_prefill(lib, hd, H, Hkv, n_ctx, runs, window):
    rng = np.random.default_rng(hd + n_ctx)
    n_seq = len(runs) + 1                                       # a sequence without rows between
    order = [0, n_seq - 1] + list(range(1, n_seq - 1)) if len(runs) > 1 else [1]
    pos = np.concatenate([np.arange(a, a + n) for a, n in runs]).astype(np.int32)
    seq = np.concatenate([np.full(n, s) for (a, n), s in zip(runs, order)]).astype(np.int32)
    T = len(pos)
    vis = visible_cells(pos, seq, n_seq, n_ctx, window)
    (kc, kd), (vc, vd) = (make_cache(rng, n_seq, Hkv, n_ctx, hd, vis) for _ in range(2))
    k, v = O.dequantize_q4_0(kc, kd), O.dequantize_q4_0(vc, vd)
    q = (rng.standard_normal((T, H * hd)) * 1.5).astype(np.float16)
    q64 = q.astype(np.float64).reshape(T, H, hd)
    ref = reference(q64, k, v, pos, seq, Hkv, window).reshape(T, -1)
    qd, kcd, vcd = dev(q), dev(pack_cache(kc, kd)), dev(pack_cache(vc, vd))
    o = torch.full((T + 3, H * hd), 9.0, dtype=torch.float16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    scratch = torch.full((lib.llm_op_attn_prefill_q4_0_scratch_bytes(T, H, Hkv, hd, n_ctx, n_seq),), 0xFF,
                         dtype=torch.uint8, device="cuda")      # NaN in every fp16 of it
    for _ in range(2):
        assert lib.llm_op_attn_prefill_q4_0(qd.data_ptr(), kcd.data_ptr(), vcd.data_ptr(), pos.ctypes.data, seq.ctypes.data,
                                            o.data_ptr(), T, H, Hkv, hd, n_ctx, n_seq, window, scratch.data_ptr(),
                                            scratch.numel(), err.data_ptr(), stream()) == 0, lib.llm_last_error(None)
        torch.cuda.synchronize()
        got = o.cpu().double().numpy()
        # the fp16 prefill kernels' own bound, 1e-2 at values of this size
        assert np.abs(got[:T] - ref).max() <= 1e-2, np.abs(got[:T] - ref).max()
        assert np.all(got[T:] == 9.0) and int(err) == 0


def test_long_cache_offsets(lib):
    """Cells past 2^32 bytes of codes: append, read back and attention through a window at the end of a long cache."""
    hd, H, Hkv, n_ctx, W = 128, 4, 2, 36_000_000, 100
    rng = np.random.default_rng(9)
    n = lib.llm_op_kv_q4_0_bytes(Hkv, hd, n_ctx, 1)
    kc, vc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    T = 130
    pos, seq = np.arange(n_ctx - T, n_ctx), np.zeros(T, np.int64)
    x = rng.standard_normal((T, (H + 2 * Hkv) * hd)).astype(np.float32)
    q = torch.empty((T, H * hd), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    xd, p, s = dev(x), ints(pos), ints(seq)
    # a table of zeros but for the angles of the rows used (cos 1, sin 0): n_ctx rows of 512 bytes
    table = torch.zeros((n_ctx, hd // 2, 2), device="cuda")
    table[-T:, :, 0] = 1
    assert lib.llm_op_qk_norm_rope(xd.data_ptr(), x.shape[1], 0, 0, 0.0, table.data_ptr(), p.data_ptr(), s.data_ptr(),
                                   q.data_ptr(), 0, kc.data_ptr(), vc.data_ptr(), 2, T, H, Hkv, hd, n_ctx, 1,
                                   err.data_ptr(), stream()) == 0
    k, v = (O.dequantize_q4_0(*O.quantize_q4_0(x.reshape(T, -1, hd)[:, i:i + Hkv])) for i in (H, H + Hkv))
    rows = torch.empty((T, Hkv, hd), dtype=torch.float16, device="cuda")
    for cache, ref in ((kc, k), (vc, v)):
        assert lib.llm_op_kv_rows_q4_0(cache.data_ptr(), p.data_ptr(), s.data_ptr(), rows.data_ptr(), T, Hkv, hd, n_ctx, 1,
                                       err.data_ptr(), stream()) == 0
        assert np.array_equal(rows.cpu().numpy(), ref.astype(np.float16))
    scratch = torch.zeros(lib.llm_op_attn_decode_q4_0_scratch_bytes(1, H, Hkv, hd, n_ctx, 1), dtype=torch.uint8, device="cuda")
    o = torch.empty((1, H * hd), dtype=torch.float16, device="cuda")
    last = p[-1:].clone()
    assert lib.llm_op_attn_decode_q4_0(q[-1:].data_ptr(), kc.data_ptr(), vc.data_ptr(), last.data_ptr(),
                                       s[:1].data_ptr(), o.data_ptr(), 1, H, Hkv, hd, n_ctx, 1, W, scratch.data_ptr(),
                                       scratch.numel(), err.data_ptr(), stream()) == 0
    ref = O.attention_one_seq(x[-1:].astype(np.float64)[:, :H * hd].reshape(1, H, hd), k[-W:], v[-W:], np.array([T - 1]),
                              np.arange(T - W, T), Hkv).reshape(-1)
    q64 = x[-1:, :H * hd].astype(np.float64).reshape(1, H, hd)
    tol = U16 * np.abs(ref) + 2.0 ** -25 + 2 * (score_tol(q64, k, hd, 21) + 2.0 ** -20) * np.abs(v).max()
    assert np.all(np.abs(o.cpu().double().numpy()[0] - ref) <= tol) and int(err) == 0


# ---------------------------------------------------------------- one after the other

@pytest.mark.parametrize("hd,H,Hkv,d,T", [(128, 8, 2, 512, 1), (64, 4, 4, 256, 5)])
def test_decode_step_block(lib, hd, H, Hkv, d, T):
    """Steps of an attention block out of 4-bit memory, each row its own sequence: the QKV projection of Q4_0 weights,
    queries and keys normed and rotated, K and V appended to a Q4_0 cache, attention over it, the output projection."""
    rng = np.random.default_rng(hd + T)
    n_ctx, steps, n_qkv = 40, 6, (H + 2 * Hkv) * hd
    (cw, dw), (co, do) = (O.quantize_q4_0(rng.standard_normal(s) * 0.05) for s in ((n_qkv, d), (d, H * hd)))
    Wq, Wo = dev(pack_weights(cw, dw)), dev(pack_weights(co, do))
    gq, gk = ((1 + 0.1 * rng.standard_normal(hd)).astype(np.float32) for _ in range(2))
    table = rope_table(n_ctx, hd)
    td, gqd, gkd = dev(table), dev(gq), dev(gk)
    kc, vc = (torch.zeros(lib.llm_op_kv_q4_0_bytes(Hkv, hd, n_ctx, T), dtype=torch.uint8, device="cuda") for _ in range(2))
    scratch = torch.zeros(lib.llm_op_attn_decode_q4_0_scratch_bytes(T, H, Hkv, hd, n_ctx, T), dtype=torch.uint8, device="cuda")
    qkv, q = torch.empty((T, n_qkv), device="cuda"), torch.empty((T, H * hd), device="cuda")
    o, y = torch.empty((T, H * hd), dtype=torch.float16, device="cuda"), torch.empty((T, d), device="cuda")
    err, posd, seqd = torch.zeros(1, dtype=torch.int32, device="cuda"), ints([0] * T), ints(list(range(T)))
    xd = torch.empty((T, d), dtype=torch.float16, device="cuda")

    def step(st):
        check = lib.check
        check(lib.llm_op_gemv_q4_0(Wq.data_ptr(), xd.data_ptr(), qkv.data_ptr(), n_qkv, d, T, d, n_qkv, st))
        check(lib.llm_op_qk_norm_rope(qkv.data_ptr(), n_qkv, gqd.data_ptr(), gkd.data_ptr(), 1e-5, td.data_ptr(),
                                      posd.data_ptr(), seqd.data_ptr(), q.data_ptr(), 0, kc.data_ptr(), vc.data_ptr(), 2, T, H,
                                      Hkv, hd, n_ctx, T, err.data_ptr(), st))
        check(lib.llm_op_attn_decode_q4_0(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), posd.data_ptr(), seqd.data_ptr(),
                                          o.data_ptr(), T, H, Hkv, hd, n_ctx, T, 0, scratch.data_ptr(), scratch.numel(),
                                          err.data_ptr(), st))
        check(lib.llm_op_gemv_q4_0(Wo.data_ptr(), o.data_ptr(), y.data_ptr(), d, H * hd, T, H * hd, d, st))

    W, Wo64 = O.dequantize_q4_0(cw, dw), O.dequantize_q4_0(co, do)
    ks, vs = np.zeros((T, Hkv, n_ctx, hd)), np.zeros((T, Hkv, n_ctx, hd))
    xd.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    step(stream())                                              # sizes and attributes settled before the capture
    with torch.cuda.graph(g):
        step(stream())
    for p in range(steps):
        x = rng.standard_normal((T, d)).astype(np.float16)
        xd.copy_(torch.from_numpy(x))
        posd.fill_(p)
        g.replay()
        torch.cuda.synchronize()
        rq, rk, rv = qk_reference((x.astype(np.float64) @ W.T), gq, gk, 1e-5, table, np.full(T, p), H, Hkv, hd)
        # a code may lie one off where the fp32 projection leaves a value next to a border: take the library's cells,
        # which must be within a step (and nearly all equal)
        for cache, mine, ref in ((kc, ks, rk), (vc, vs, rv)):
            c, dd = unpack_cache(cache.cpu().numpy(), T, Hkv, n_ctx, hd)
            rc, rd = O.quantize_q4_0(ref)
            off = np.abs(c[:, :, p].astype(int) - rc.astype(int))
            assert off.max() <= 1 and (off > 0).mean() < 0.01
            mine[:, :, p] = O.dequantize_q4_0(c[:, :, p], dd[:, :, p])
        ref = reference(rq, ks, vs, [p] * T, list(range(T)), Hkv, 0).reshape(T, -1)
        got = o.cpu().double().numpy()
        vmax = np.abs(vs).max()
        assert np.all(np.abs(got - ref) <= U16 * np.abs(ref) + 2.0 ** -25 + 2 * (score_tol(rq, ks, hd, 18) + 2.0 ** -18) * vmax)
        ref_y = got @ Wo64.T
        mag = np.abs(got) @ np.repeat(np.abs(do.astype(np.float64)), 32, 1).T * 23
        assert np.all(np.abs(y.cpu().double().numpy() - ref_y) <= mag * U32 * (8 + H * hd // 32))
    assert int(err) == 0


def test_attn_prefill_many_sequences_and_capture(lib):
    """Rows of more sequences than a launch carries by value, and a captured call replayed after q and the cache moved."""
    hd, H, Hkv, n_ctx, n_seq = 64, 4, 2, 70, 80
    rng = np.random.default_rng(17)

    def case(runs):
        pos = np.concatenate([np.arange(a, a + n) for _, a, n in runs]).astype(np.int32)
        seq = np.concatenate([np.full(n, s) for s, _, n in runs]).astype(np.int32)
        vis = visible_cells(pos, seq, n_seq, n_ctx, 0)
        (kc, kd), (vc, vd) = (make_cache(rng, n_seq, Hkv, n_ctx, hd, vis) for _ in range(2))
        q = (rng.standard_normal((len(pos), H * hd)) * 1.5).astype(np.float16)
        ref = reference(q.astype(np.float64).reshape(-1, H, hd), O.dequantize_q4_0(kc, kd), O.dequantize_q4_0(vc, vd), pos, seq,
                        Hkv, 0).reshape(len(pos), -1)
        return pos, seq, dev(q), dev(pack_cache(kc, kd)), dev(pack_cache(vc, vd)), ref

    def call(pos, seq, q, kc, vc, o, scratch):
        assert lib.llm_op_attn_prefill_q4_0(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), pos.ctypes.data, seq.ctypes.data,
                                            o.data_ptr(), len(pos), H, Hkv, hd, n_ctx, n_seq, 0, scratch.data_ptr(),
                                            scratch.numel(), 0, stream()) == 0, lib.llm_last_error(None)

    def buffers(T):
        n = lib.llm_op_attn_prefill_q4_0_scratch_bytes(T, H, Hkv, hd, n_ctx, n_seq)
        return torch.zeros((T, H * hd), dtype=torch.float16, device="cuda"), torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    many = [(s, s % 60, 1 + s % 3) for s in range(n_seq)]
    pos, seq, q, kc, vc, ref = case(many)
    o, scratch = buffers(len(pos))
    call(pos, seq, q, kc, vc, o, scratch)
    assert np.abs(o.cpu().double().numpy() - ref).max() <= 1e-2
    few = [(3, 10, 40), (79, 0, 17)]
    pos, seq, q, kc, vc, ref = case(few)
    o, scratch = buffers(len(pos))
    call(pos, seq, q, kc, vc, o, scratch)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(pos, seq, q, kc, vc, o, scratch)
    _, _, q2, kc2, vc2, ref = case(few)
    for a, b in ((q, q2), (kc, kc2), (vc, vc2)):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    assert np.abs(o.cpu().double().numpy() - ref).max() <= 1e-2
