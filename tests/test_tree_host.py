"""CPU checks of the entry points of drafted decoding: their refusals, which
come before any device work (no pointer here is ever dereferenced), and their sizes."""
import ctypes

import numpy as np
import pytest

import tree_util as U

lib = pytest.importorskip("llama_decoder_forward_02_gb300")
P, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4100)
BAD = lib.LLM_ERR_INVALID


def reason():
    return lib.llm_last_error(None).decode()


@pytest.mark.parametrize("change,why", [
    (dict(n_rot=4), "n_rot"), (dict(n_rot=136), "n_rot"), (dict(n_rot=20), "n_rot"), (dict(layout=2), "layout"),
    (dict(scaling=4), "scaling"), (dict(scaling=-1), "scaling"), (dict(theta=1.0), "theta"), (dict(theta=float("nan")), "theta"),
    (dict(scaling=1, factor=0.5), "factor"), (dict(scaling=2, n_ctx_orig=0), "n_ctx_orig"),
    (dict(scaling=2, slow=4.0, fast=4.0), "slow"), (dict(scaling=3, slow=0.0), "slow"),
    (dict(scaling=3, factor=float("inf")), "factor"), (dict(attn_factor=-1.0), "attn_factor"),
])
def test_rotations_refused(change, why):
    ok = dict(theta=10000.0, n_rot=64, factor=2.0, n_ctx_orig=2048)
    assert lib.llm_op_rope_table(lib.rope(**{**ok, **change}), 0, 8, P, None) == BAD and why in reason()


def test_table_arguments_refused():
    r = lib.rope(10000.0, 64)
    for args, why in (((r, -1, 8, P), "positions"), ((r, 0, 0, P), "positions"), ((r, (1 << 30) - 3, 4, P), "positions"),
                      ((r, 0, 8, None), "NULL"), ((r, 0, 8, ODD), "aligned"), ((None, 0, 8, P), "NULL")):
        assert lib.llm_op_rope_table(*args, None) == BAD and why in reason()


ROPE = dict(qkv=P, ld=(8 + 4) * 64, q_gain=None, k_gain=None, eps=1e-5, rope=P, n_pos=100, n_rot=64, layout=0, pos=P, cell=None,
            seq=P, q=P, q_type=1, k=P, v=P, kv_type=0, T=4, H=8, Hkv=2, hd=64, n_ctx=100, n_seq=1, err=None, stream=None)


@pytest.mark.parametrize("change,why", [
    (dict(qkv=None), "NULL"), (dict(rope=None), "NULL"), (dict(pos=None), "NULL"), (dict(seq=None), "NULL"), (dict(q=None), "NULL"),
    (dict(k=None), "NULL"), (dict(T=0), "T must"), (dict(hd=48), "head_dim"), (dict(H=7), "multiple"), (dict(n_ctx=0), "positive"),
    (dict(ld=767), "ld"), (dict(ld=764), "ld"), (dict(n_pos=0), "n_pos"), (dict(n_rot=72), "n_rot"), (dict(n_rot=12), "n_rot"),
    (dict(layout=2), "layout"), (dict(q_type=2), "q_type"), (dict(kv_type=3), "kv_type"), (dict(eps=-1.0), "eps"),
    (dict(rope=ODD), "aligned"), (dict(k_gain=ODD), "aligned"), (dict(v=ODD), "aligned"),
])
def test_rotation_and_append_refused(change, why):
    assert lib.llm_op_rope_kv(*{**ROPE, **change}.values()) == BAD and why in reason()


TREE = dict(q=P, k=P, v=P, row0=P, seq=P, base=P, mask=P, pos=None, o=P, T=20, n_tree=2, max_nodes=16, H=8, Hkv=2, hd=64,
            n_ctx=500, n_seq=2, kv_type=0, window=0, scratch=P, size=1 << 40, err=None, stream=None)


@pytest.mark.parametrize("change,why", [
    (dict(q=None), "NULL"), (dict(row0=None), "NULL"), (dict(mask=None), "NULL"), (dict(o=None), "NULL"), (dict(T=0), "T must"),
    (dict(hd=96), "head_dim"), (dict(H=9), "multiple"), (dict(n_tree=0), "n_tree"), (dict(n_tree=5000), "n_tree"),
    (dict(max_nodes=0), "max_nodes"), (dict(max_nodes=257), "max_nodes"), (dict(kv_type=2), "kv_type"),
    (dict(window=-1), "window"), (dict(window=8), "pos"), (dict(scratch=None), "scratch"), (dict(size=0), "scratch"),
    (dict(k=ODD), "aligned"), (dict(scratch=ODD), "aligned"), (dict(n_ctx=1 << 29, n_seq=4), "rows"),
    (dict(n_tree=4096, max_nodes=256, H=64), "groups"),
])
def test_attention_refused(change, why):
    assert lib.llm_op_attn_tree(*{**TREE, **change}.values()) == BAD and why in reason()


def test_sizes():
    assert lib.llm_op_attn_tree_scratch_bytes(1, 16, 32, 8, 128, 4096) > 0
    for args in ((0, 16, 32, 8, 128, 4096), (1, 300, 32, 8, 128, 4096), (1, 16, 30, 8, 128, 4096), (1, 16, 32, 8, 100, 4096),
                 (1, 16, 32, 8, 128, 0)):
        assert lib.llm_op_attn_tree_scratch_bytes(*args) == BAD


ACCEPT = dict(token=P, parent=P, target=P, row0=P, seq=P, base=P, k=P, v=P, kv_type=0, path=P, n=P, next=P, T=20, n_tree=2,
              max_nodes=16, n_layer=2, Hkv=2, hd=64, n_ctx=100, n_seq=2, err=None, stream=None)


@pytest.mark.parametrize("change,why", [
    (dict(token=None), "NULL"), (dict(path=None), "NULL"), (dict(next=None), "NULL"), (dict(T=0), "T must"),
    (dict(max_nodes=257), "max_nodes"), (dict(n_tree=0), "n_tree"), (dict(n_layer=0), "n_layer"), (dict(n_layer=40000), "n_layer"),
    (dict(kv_type=5), "kv_type"), (dict(hd=16), "head_dim"), (dict(k=ODD), "aligned"), (dict(n_ctx=1 << 30, n_seq=1 << 10), "2^46"),
])
def test_acceptance_refused(change, why):
    assert lib.llm_op_tree_accept(*{**ACCEPT, **change}.values()) == BAD and why in reason()


def test_definitions():
    """The definitions that the GPU tests compare with, by hand."""
    par = np.array([-1, 0, 0, 1, 3])
    assert U.depths(par).tolist() == [0, 1, 1, 2, 3]
    assert U.ancestors(par)[4].tolist() == [True, True, False, True, True]
    assert U.pack_mask(U.ancestors(par), 40)[4].tolist() == [0b11011, 0]
    assert U.accept([9, 5, 6, 5, 8], par, [5, 5, 0, 8, 1]) == ([0, 1, 3, 4], 1)
    assert U.accept([9, 5, 5, 1, 1], [-1, 0, 0, 2, 1], [5, 7, 1, 0, 0]) == ([0, 1], 7)      # the lowest of two equal children
    f, m = U.frequencies(10000.0, 64, 3, 4.0, 1.0, 32.0, 2048)
    f0 = 10000.0 ** (-np.arange(32) / 32)
    turns = 2048 * f0 / (2 * np.pi)
    assert np.allclose(f[turns > 40], f0[turns > 40]) and np.allclose(f[turns < 0.7], f0[turns < 0.7] / 4)
    assert m == pytest.approx(1.1386294)
    f, _ = U.frequencies(10000.0, 64, 2, 8.0, 1.0, 4.0, 2048)
    assert np.allclose(f[turns > 4], f0[turns > 4]) and np.allclose(f[turns < 1], f0[turns < 1] / 8)
    x = np.arange(8.0).reshape(1, 1, 8)
    quarter = np.array([[[0.0, 1.0]] * 2])
    assert U.rotate(x, quarter, 4, 0)[0, 0].tolist() == [-1, 0, -3, 2, 4, 5, 6, 7]
    assert U.rotate(x, quarter, 4, 1)[0, 0].tolist() == [-2, -3, 0, 1, 4, 5, 6, 7]


def check_tree(n_nodes, token, parent, seq_id=None, pos_max=(9, -1, 4), n_vocab=50, n_ctx=40, n_ubatch=32):
    b, keep = lib.tree_batch(n_nodes, token, parent, seq_id)
    n = max(len(token), 1)
    pos, cell = (ctypes.c_int32 * n)(), (ctypes.c_int32 * n)()
    ends = (ctypes.c_int32 * len(pos_max))(*pos_max)
    rc = lib.llm_tree_check(n_vocab, n_ctx, len(pos_max), n_ubatch, ends, ctypes.byref(b), pos, cell)
    return rc, list(pos), list(cell)


def test_tree_batches():
    rc, pos, cell = check_tree([4, 2], [1, 2, 3, 4, 5, 6], [-1, 0, 0, 2, -1, 0], [2, 1])
    assert rc == 0 and pos == [5, 6, 6, 7, 0, 1] and cell == [5, 6, 7, 8, 0, 1]
    rc, pos, _ = check_tree([1, 1, 1], [0, 0, 0], [-1, -1, -1])
    assert rc == 0 and pos == [10, 0, 5]
    assert check_tree([30], [0] * 30, [-1] + [0] * 29)[0] == 0          # cells 10 .. 39
    assert check_tree([31], [0] * 31, [-1] + [0] * 30)[0] == lib.LLM_NO_KV_ROOM
    for args in (([33], [0] * 33, [-1] + [0] * 32), ([257], [0] * 257, [-1] + [0] * 256), ([0], [], []),
                 ([2], [0, 0], [-1, -1]), ([2], [0, 0], [-1, 1]), ([1], [0], [0]), ([1], [50], [-1]),
                 ([1], [0], [-1], [3]), ([1], [0], [-1], [-1]), ([1, 1], [0, 0], [-1, -1], [2, 2]),
                 ([1] * 4, [0] * 4, [-1] * 4, [0, 1, 2, 0])):
        assert check_tree(*args)[0] == BAD
    assert lib.llm_tree_check(50, 40, 3, 32, None, None, None, None) == BAD
    with pytest.raises(ValueError):
        lib.tree_batch([2], [1], [-1])


def test_context_calls_refuse_null():
    one = (ctypes.c_int32 * 1)(0)
    b, keep = lib.tree_batch([1], [0], [-1])
    assert lib.llm_decode_tree(None, ctypes.byref(b)) == BAD
    assert lib.llm_tree_accept(None, one, None, None, None) == BAD
    r = lib.rope(10000.0, 64)
    assert lib.llm_model_set_rope(None, ctypes.byref(r), None) == BAD
