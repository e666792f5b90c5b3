"""Calls of the operators of drafted decoding that their documentation allows, beside those of test_gpu_tree.py: rows
before the first tree, more query heads of a kv head than a tile has rows, no error word, tables past 2^31 elements,
cells that one leaf alone sees, and the bytes around the caches."""
import numpy as np
import pytest
import torch

import tree_util as U
from test_gpu_tree import Trees, err_word, ints, lib, make_accept, stream  # noqa: F401  (lib: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kt", [0, 1])
def test_rows_before_the_first_tree(lib, kt):      # noqa: F811
    """Rows that belong to no tree are left as they are, those in front too."""
    t = Trees(lib, 64, 8, 2, [(0, 0), (300, 7), (40, 12)], 400, kt, spare=4)
    t.run()
    want = t.O.clone()
    lead = 5
    q, o = (torch.full((t.T + lead, 8 * 64), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    q[lead:] = t.Q.view(t.T, -1)
    mask = torch.cat((t.MASK[:1].expand(lead, -1), t.MASK)).contiguous()
    args, row0 = t.args(o=o), ints(t.row0 + lead)
    args[0], args[3], args[6], args[9] = q.data_ptr(), row0.data_ptr(), mask.data_ptr(), t.T + lead
    lib.check(lib.llm_op_attn_tree(*args))
    assert torch.all(o[:lead] == 9) and torch.equal(o[lead:], want) and int(t.E) == 0


@pytest.mark.parametrize("hd,H,Hkv,trees", [
    (32, 320, 1, [(150, 5), (20, 2)]),            # a node of two and a half tiles of rows
    (64, 260, 2, [(300, 3)]),
    (128, 144, 1, [(130, 2)]),
])
@pytest.mark.parametrize("kt", [0, 1])
def test_many_query_heads(lib, hd, H, Hkv, trees, kt):      # noqa: F811
    t = Trees(lib, hd, H, Hkv, trees, 400, kt)
    t.run()
    t.check()


def test_no_error_word(lib):      # noqa: F811
    t = Trees(lib, 64, 4, 2, [(10, 4), (20, 5)], 60)
    t.BASE.copy_(ints([10, 56]))                   # 56 + 5 > 60
    args = t.args()
    args[-2] = None
    lib.check(lib.llm_op_attn_tree(*args))
    torch.cuda.synchronize()
    assert torch.all(t.O[4:] == 0)
    t.trees = [t.trees[0], (20, 0)]
    t.check()


def test_table_past_32_bits(lib):      # noqa: F811
    """The last rows of a table of more than 2^31 floats, as a call of their own gives them."""
    n, last = (1 << 24) + 1111, 1500
    r = lib.rope(500000.0, 128, scaling=lib.LLM_ROPE_RAMP, factor=4.0, n_ctx_orig=8192)
    big, small = torch.empty((n, 64, 2), device="cuda"), torch.empty((last, 64, 2), device="cuda")
    assert big.numel() > 2 ** 31
    lib.check(lib.llm_op_rope_table(r, 0, n, big.data_ptr(), stream()))
    for at in (n - last, (1 << 24) - last // 2):
        lib.check(lib.llm_op_rope_table(r, at, last, small.data_ptr(), stream()))
        assert torch.equal(big[at:at + last], small)


@pytest.mark.parametrize("kt", [0, 1])
def test_cells_that_a_leaf_alone_sees(lib, kt):      # noqa: F811
    """NaN in the cells of a node without children changes the row of that node and no other."""
    t = Trees(lib, 128, 8, 2, [(700, 12), (128, 5)], 900, kt)
    clean = t.run().clone()
    for i in range(2):
        n = t.trees[i][1]
        leaves = [j for j in range(n) if j not in t.par[i]]
        for j in leaves:
            assert t.seen[i][:, j].sum() == 1 and t.seen[i][j, j]
            for c in t.KV:
                at = (c.view(torch.uint8) if kt else c)[t.seq[i], :, t.trees[i][0] + j]
                held = at.clone()
                at.fill_(0x7f if kt else float("nan"))
                t.O.fill_(9.0)
                t.run()
                row = int(t.row0[i]) + j
                rest = torch.arange(t.T, device="cuda") != row
                assert torch.equal(clean[rest], t.O[rest]) and not torch.isfinite(t.O[row]).any()
                at.copy_(held)
        assert leaves


@pytest.mark.parametrize("kt", [0, 1, 2])
def test_bytes_around_the_caches(lib, kt):      # noqa: F811
    """Caches of exactly the documented size, [n_seq][n_layer][Hkv][n_ctx][hd], with other bytes right before and behind."""
    L, Hkv, hd, n_seq, sizes, guard = 2, 3, 64, 2, [40, 9], 256
    n_ctx, rng = 40, np.random.default_rng(kt)     # the first tree's cells fill its sequence
    size = n_seq * L * Hkv * n_ctx * hd
    size = {0: 2 * size, 1: size, 2: size // 2 + size // 32 * 2}[kt]
    token, parent, target = make_accept(rng, sizes, "chain", 1.0)
    parent[0][1:] = 0                              # only one child of the root is taken, the last one
    token[0][:] = np.arange(40)
    target[0][0] = 39
    hold = [torch.randint(0, 256, (size + 2 * guard,), dtype=torch.uint8, device="cuda") for _ in range(2)]
    keep = [h.clone() for h in hold]
    tk, pr, tg = (ints(np.concatenate(x)) for x in (token, parent, target))
    R, S, B = ints([0, 40, 49]), ints([1, 0]), ints([0, 31])
    path, count, nxt, E = torch.zeros((2, 40), dtype=torch.int32, device="cuda"), ints([0, 0]), ints([0, 0]), err_word()
    lib.check(lib.llm_op_tree_accept(tk.data_ptr(), pr.data_ptr(), tg.data_ptr(), R.data_ptr(), S.data_ptr(), B.data_ptr(),
                                     hold[0].data_ptr() + guard, hold[1].data_ptr() + guard, kt, path.data_ptr(), count.data_ptr(),
                                     nxt.data_ptr(), 49, 2, 40, L, Hkv, hd, n_ctx, n_seq, E.data_ptr(), stream()))
    assert int(E) == 0 and path[0, :3].tolist() == [0, 39, -1]
    rows = n_seq * L * Hkv * n_ctx
    for h, k in zip(hold, keep):
        assert torch.equal(h[:guard], k[:guard]) and torch.equal(h[-guard:], k[-guard:])
        parts, at = ((2 * hd,), (hd,), (hd // 2, hd // 16))[kt], guard
        for per in parts:
            new, old = (x[at:at + rows * per].view(n_seq, L * Hkv, n_ctx, per) for x in (h, k))
            want = old.clone()
            want[1, :, 1] = old[1, :, 39]
            path1, _ = U.accept(token[1], parent[1], target[1])
            want[0, :, 31:31 + len(path1)] = old[0][:, [31 + j for j in path1]]
            assert torch.equal(new, want)
            at += rows * per
        assert at == size + guard
