"""Attention of trees of drafted tokens at scores far beyond the usual ones: large finite scores of either sign,
whose softmax is all but a choice, against the definition in 64 bits.

Tolerance.  Every key holds one value hd times, of at most 11 bits, and every query one, so that the scores and their
partial sums are fp32 numbers and the products exact.  What is left: with d the distance of a score to the row's largest
as an exponent of two, log2(e) / sqrt(hd) is good to 2^-23 and the exponent's rounding to 2^-24 of at most d + 16, so a
weight with d <= 40 is off by 0.7 (40 2^-23 + 56 2^-24) + 2^-21 (its two parts and the exponential) < 2^-17 of it; the
others are below 2^-40 of the largest.  2^-16 of the weighted sum of |V| for the sums above and below the line; then
o's rounding."""
import numpy as np
import pytest
import torch

import tree_util as U
from test_gpu_tree import TINY16, U16, Trees, dev, lib  # noqa: F401  (lib: the fixture)

pytestmark = pytest.mark.gpu


def put_keys(t, rng, climb):
    """Keys of one value each, of rising size and then sign where they climb, and queries of one value each from tiny
    to the largest."""
    kt, hd = t.kt, t.hd
    n_seq, Hkv, n_ctx = t.k.shape[:3]
    bits, most = (3, 8) if kt else (10, 15)
    low = -6 if kt else -10
    shape = (n_seq, Hkv, n_ctx)
    e = rng.integers(low, most + 1, shape) if climb else np.full(shape, most - 1)
    v = np.ldexp(1 + rng.integers(0, 1 << bits, shape) / (1 << bits), e)
    if kt:
        v = np.minimum(v, 448)
    if climb:
        v = np.sort(v * rng.choice([-1.0, 1.0], shape), -1)
    else:
        v *= rng.choice([-1.0, 1.0], (n_seq, Hkv, 1))
    t.k = np.repeat(v[..., None], hd, -1)
    k = torch.from_numpy(t.k.astype(np.float32)).to(t.KV[0].dtype)
    assert np.array_equal(k.double().numpy(), t.k)
    t.KV[0].copy_(k)
    q = np.ldexp(rng.choice([-1.0, 1.0], (t.T, t.H, 1)), 15 - rng.integers(0, 25, (t.T, t.H, 1)))
    q[rng.random((t.T, t.H)) < 0.3] = 65504.0
    t.q = np.repeat(q, hd, -1).astype(np.float16)
    t.Q.copy_(dev(t.q).view(t.Q.shape))


def check(t):
    got = t.O.cpu().double().numpy().reshape(t.T, t.H, t.hd)
    assert int(t.E) == 0
    far = 0
    for i, ((b, n), r) in enumerate(zip(t.trees, t.row0)):
        s = t.seq[i]
        ref, mag, _ = U.attention(t.q[r:r + n].astype(np.float64), t.k[s], t.v[s], b, t.seen[i], t.pos[r:r + n], t.window)
        d, tol = np.abs(got[r:r + n] - ref), U16 * np.abs(ref) + TINY16 + 2.0 ** -16 * mag
        assert np.all(d <= tol), (i, float((d / tol).max()))
        far = max(far, float(np.abs(t.q[r:r + n].astype(np.float64)).max() * np.abs(t.k[s]).max() * t.hd ** 0.5 * 1.44))
    assert far > 2.0 ** 26


@pytest.mark.parametrize("kt", [0, 1])
@pytest.mark.parametrize("climb", [False, True])
@pytest.mark.parametrize("hd,H,Hkv,trees,n_ctx,window", [
    (128, 4, 1, [(100, 9)], 128, 0),                    # one CTA
    (64, 8, 2, [(700, 20), (3, 5)], 900, 0),            # joined inside a cluster
    (128, 8, 2, [(3000, 16)], 3100, 0),
    (128, 8, 2, [(9000, 20), (40, 3)], 9100, 0),        # and through memory
    (64, 8, 2, [(9000, 12)], 9100, 0),
    (32, 4, 2, [(500, 9)], 600, 300),
])
def test_large_scores(lib, hd, H, Hkv, trees, n_ctx, window, climb, kt):      # noqa: F811
    t = Trees(lib, hd, H, Hkv, trees, n_ctx, kt, window)
    for seed in range(3):
        put_keys(t, np.random.default_rng(seed), climb)
        t.O.fill_(9.0)
        t.run()
        check(t)


def test_scores_of_near_size(lib):      # noqa: F811
    """Scores of 2^22 to 2^27 that differ by an exponent of 0.1 to 4, so that several cells share a row."""
    hd, base = 128, 900
    t = Trees(lib, hd, 8, 2, [(base, 12)], 1000)
    rng = np.random.default_rng(4)
    # q = (2^a, 1, .., 1), K = (2^12, 2^(a - 10) j, 0, .., 0): 2^(a + 12) + 2^(a - 10) j, of 23 bits
    for a in (10, 12, 14, 15):
        t.q = np.ones((t.T, t.H, hd), np.float16)
        t.q[..., 0] = 2.0 ** a * rng.choice([-1.0, 1.0], (t.T, t.H))
        t.k = np.zeros_like(t.k)
        t.k[..., 0] = 4096
        t.k[..., 1] = rng.integers(0, 32, t.k.shape[:3]) * 2.0 ** (a - 10)
        t.Q.copy_(dev(t.q).view(t.Q.shape))
        t.KV[0].copy_(torch.from_numpy(t.k))
        t.run()
        got = t.O.cpu().double().numpy().reshape(t.T, t.H, hd)
        s = t.seq[0]
        ref, mag, _ = U.attention(t.q.astype(np.float64), t.k[s], t.v[s], base, t.seen[0], t.pos, 0)
        assert np.all(np.abs(got - ref) <= U16 * np.abs(ref) + TINY16 + 2.0 ** -16 * mag)
