"""How exact a softmax weight of the attention of trees is: 22 bits down to 2^-9 of the row's largest, below that 2^-30 of
the largest."""
import numpy as np
import pytest
import torch

from test_gpu_tree import TINY16, U16, Trees, dev, lib  # noqa: F401  (lib: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [128, 64])
@pytest.mark.parametrize("sign", [1, -1])
def test_small_weights(lib, hd, sign):      # noqa: F811
    """Two cells a row, of the scores 0 and -x, or x and 0, whose lower one has V = 60000 and the other none, so that o is the
    lower one's weight."""
    n, H = 200, 8
    t = Trees(lib, hd, H, 2, [(2, n)], 300, seen=[np.zeros((n, n), bool)])
    rng = np.random.default_rng(hd + sign)
    t.q[:] = 0
    t.q[..., 0] = rng.uniform(0, 22 * hd ** 0.5, (n, H)) * sign
    t.k[:] = 0
    t.k[:, :, 0 if sign < 0 else 1, 0] = -1
    t.v[:] = 0
    t.v[:, :, 1] = 60000
    t.Q.copy_(dev(t.q).view(t.Q.shape))
    for c, a in zip(t.KV, (t.k, t.v)):
        c.copy_(torch.from_numpy(a))
    t.run()
    got = t.O.cpu().double().numpy().reshape(n, H, hd)
    x = np.abs(t.q[..., 0].astype(np.float64)) / np.sqrt(hd)
    p = np.exp(-x)                                 # of the largest weight
    w = p / (1 + p)
    assert p.min() < 2.0 ** -30 and p.max() > 0.5
    # the weight's two parts, 2^-22 of it or 2^-30 of the largest; its exponent, up to 32, through log2(e) / sqrt(hd) and
    # the rounding, 2^-23 and 2^-24 of at most 32 + 7, times ln 2, and the exponential 2^-22: below 2^-17 of it; then o's rounding
    tol = U16 * 60000 * w + TINY16 + 60000 * (2.0 ** -17 * w + 2.0 ** -30)
    assert np.all(np.abs(got - 60000 * w[..., None]) <= tol[..., None])
    assert int(t.E) == 0
