"""Attention of trees of drafted tokens with infinities in the cells that a row sees, held against the definition: a
score of -inf has weight 0, a row of which nothing else is seen is NaN as softmax has it, a score of +inf or NaN makes
its row NaN, and a row that sees nothing is zero."""
import numpy as np
import pytest
import torch

import tree_util as U
from test_gpu_tree import TINY16, U16, Trees, lib  # noqa: F401  (lib: the fixture)

pytestmark = pytest.mark.gpu
INF = float("inf")


def check(t):
    """Where the definition is finite, within the bounds of usual scores; elsewhere nothing finite."""
    got = t.O.cpu().double().numpy().reshape(t.T, t.H, t.hd)
    counts = np.zeros(3, int)
    for i, ((b, n), r) in enumerate(zip(t.trees, t.row0)):
        s = t.seq[i]
        q = t.q[r:r + n].astype(np.float64)
        with np.errstate(invalid="ignore"):
            ref, _, _ = U.attention(q, t.k[s], t.v[s], b, t.seen[i], t.pos[r:r + n], t.window)
        # magnitudes of the finite part: at most the largest |V| and the largest root of a finite key's products
        v, k = (np.where(np.isfinite(c[s]), c[s], 0) for c in (t.v, t.k))
        mag = np.abs(v).max()
        size = np.sqrt((k ** 2).max(1).sum(-1).max() * (q ** 2).max())
        tol = U16 * np.abs(ref) + TINY16 + (2.0 ** -20 * size + 2.0 ** -19) * mag
        g, fine = got[r:r + n], np.isfinite(ref)
        assert not np.isfinite(g[~fine]).any()
        assert np.all(np.abs(g[fine] - ref[fine]) <= tol[fine])
        assert np.all(g[(ref == 0).all(-1)] == 0)
        counts += [fine.sum(), (~fine).sum(), (ref == 0).all(-1).sum()]
    assert int(t.E) == 0
    return counts


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("hd,trees,n_ctx", [(128, [(400, 10), (0, 4)], 500), (64, [(700, 12), (0, 3)], 800),
                                            (128, [(9000, 6), (20, 3)], 9100), (32, [(100, 9)], 128)])
def test_infinite_keys(lib, hd, trees, n_ctx, sign):      # noqa: F811
    def cells(t, which):
        for i, (b, n) in enumerate(t.trees):
            at = {"one": [b // 3], "past": range(b), "node": [b], "all": range(b + n)}[which]
            yield t.seq[i], np.asarray(list(at), int)
    for which in ("one", "past", "node", "all"):
        t = Trees(lib, hd, 8, 2, trees, n_ctx)
        for s, at in cells(t, which):
            t.k[s, 1, at, 3] = sign * INF
        t.KV[0].copy_(torch.from_numpy(t.k))
        t.run()
        fine, odd, _ = check(t)
        assert fine and odd


def test_nothing_seen_beside_infinite_scores(lib):      # noqa: F811
    """Rows without a cell are zero, rows whose only cells have a score of -inf are not."""
    for hd in (128, 64):
        seen = [np.zeros((40, 40), bool), np.zeros((3, 3), bool)]
        seen[0][::2, ::3] = True                            # every other row; no row of the second tree
        t = Trees(lib, hd, 8, 2, [(0, 40), (0, 3)], 300, seen=seen, max_nodes=45)
        t.k[t.seq[0], 0, :40, 3] = -INF
        t.KV[0].copy_(torch.from_numpy(t.k))
        t.run()
        fine, odd, zero = check(t)
        assert fine and odd and zero >= (20 + 3) * 8


@pytest.mark.parametrize("hd,base", [(128, 384), (64, 8960)])
def test_infinite_values_of_infinite_scores(lib, hd, base):      # noqa: F811
    """Weight 0 times an infinity: not finite, also where all cells of a CTA are such."""
    t = Trees(lib, hd, 8, 2, [(base, 10)], base + 100)
    t.k[t.seq[0], 1, :base, 3] = INF
    t.v[t.seq[0], 1, :base, 5] = INF
    for c, a in zip(t.KV, (t.k, t.v)):
        c.copy_(torch.from_numpy(a))
    t.run()
    got = t.O.view(t.T, 8, hd)
    low = torch.from_numpy(t.q[:, 4:, 3] < 0).cuda()
    assert low.any() and not torch.isfinite(got[:, 4:, 5][low]).any()
    assert torch.isfinite(got[:, :4]).all() and int(t.E) == 0
