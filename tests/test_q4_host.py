"""CPU checks of the Q4_0 encoding and of the 4-bit entry points' refusals,
which come before any device work (no pointer here is ever dereferenced)."""
import ctypes

import numpy as np
import pytest

from oracle import llama as O
from q4_util import pack_cache, pack_groups, pack_weights, unpack_cache, unpack_groups

lib = pytest.importorskip("llama_decoder_forward_02_gb300")


def test_q4_0_hand_values():
    w = np.zeros((1, 32))
    w[0, :6] = [8.0, -8.0, 7.0, 0.5, 1.5, -7.6]        # first of equals: m = 8, d = -1
    c, d = O.quantize_q4_0(w)
    assert d[0, 0] == -1.0
    # w / d = -8, 8, -7, -0.5, -1.5, 7.6; ties to even; +8, clamped
    assert list(c[0, :6]) == [0, 15, 1, 8, 6, 15]
    assert list(O.dequantize_q4_0(c, d)[0, :6]) == [8.0, -7.0, 7.0, 0.0, 2.0, -7.0]
    c, d = O.quantize_q4_0(-w)
    assert d[0, 0] == 1.0 and list(c[0, :6]) == [0, 15, 1, 8, 6, 15]


def test_q4_0_error_bound_and_zero_blocks():
    rng = np.random.default_rng(3)
    w = rng.standard_normal((8, 96)) * np.exp(rng.uniform(-6, 6, (8, 1)))
    w[2, 32:64] = 0
    c, d = O.quantize_q4_0(w)
    top = np.abs(w.reshape(8, 3, 32)).max(-1)
    err = np.abs(O.dequantize_q4_0(c, d) - w).reshape(8, 3, 32).max(-1)
    # half a step inside, a whole one where 8 is clamped to 7; the stored scale is half an fp16 step off
    # (or half a subnormal step of fp16, 8 levels of it)
    assert np.all(err <= top / 8 * (1 + 8 * 2.0 ** -11) + 8 * 2.0 ** -25)
    assert d[2, 1] == 0 and np.all(c[2, 32:64] == 8)
    assert np.array_equal(O.round_to(w, "q4_0"), O.dequantize_q4_0(c, d))


@pytest.mark.parametrize("nb", [1, 2, 4])
def test_layout_round_trip(nb):
    rng = np.random.default_rng(nb)
    c = rng.integers(0, 16, (3, 5, 7, 32 * nb)).astype(np.uint8)
    d = rng.standard_normal((3, 5, 7, nb)).astype(np.float16)
    raw = pack_groups(c, nb)
    assert raw.shape[-1] == 16 * nb and np.array_equal(unpack_groups(raw, nb), c)
    c2, d2 = unpack_cache(pack_cache(c, d), 3, 5, 7, 32 * nb)
    assert np.array_equal(c2, c) and np.array_equal(d2, d)
    # element 8 t + 2 i + odd of block b: word t * nb + b, bit 4 i + 16 odd
    one = np.zeros(32 * nb, np.uint8)
    one[32 * (nb - 1) + 8 * 2 + 2 * 3 + 1] = 9
    assert pack_groups(one, nb).view(np.uint32)[2 * nb + nb - 1] == 9 << 28
    w = rng.integers(0, 16, (2, 512)).astype(np.uint8)
    assert pack_weights(w, np.ones((2, 16), np.float16)).shape == (2, 288)


P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4100)
BAD = lib.LLM_ERR_INVALID


def why():
    return lib.llm_last_error(None)


def test_weight_calls_refuse():
    for n, k in ((0, 256), (4, 0), (4, 128), (4, 384)):
        assert lib.llm_op_quantize_q4_0(P, n, k, P, None) == BAD
        assert lib.llm_op_gemv_q4_0(P, P, P, n, k, 1, 1024, 1024, None) == BAD
    assert lib.llm_op_quantize_q4_0(None, 4, 256, P, None) == BAD
    assert lib.llm_op_quantize_q4_0(P, 4, 256, ODD, None) == BAD and b"aligned" in why()
    for T in (0, 9):
        assert lib.llm_op_gemv_q4_0(P, P, P, 4, 256, T, 256, 4, None) == BAD and b"T must" in why()
    for ldx, ldy in ((248, 4), (260, 4), (256, 3)):
        assert lib.llm_op_gemv_q4_0(P, P, P, 4, 256, 1, ldx, ldy, None) == BAD and b"ldx" in why()
    assert lib.llm_op_gemv_q4_0(P, ODD, P, 4, 256, 1, 256, 4, None) == BAD and b"aligned" in why()
    assert lib.llm_op_gemv_q4_0(None, P, P, 4, 256, 1, 256, 4, None) == BAD
    assert lib.llm_model_quantize(None, 7, None) == BAD


SHAPES = [  # T, H, Hkv, hd, n_ctx, n_seq, reason
    (0, 8, 2, 64, 64, 1, b"T must"), (1, 8, 2, 48, 64, 1, b"head_dim"), (1, 8, 2, 256, 64, 1, b"head_dim"),
    (1, 8, 3, 64, 64, 1, b"multiple"), (1, 0, 1, 64, 64, 1, b"multiple"), (1, 8, 0, 64, 64, 1, b"multiple"),
    (1, 8, 2, 64, 0, 1, b"n_ctx"), (1, 8, 2, 64, 64, 0, b"n_seq"), (1, 8192, 2, 64, 64, 1, b"4096"),
    (1, 8, 2, 64, (1 << 30) + 1, 1, b"2^30"),
]


@pytest.mark.parametrize("T,H,Hkv,hd,n_ctx,n_seq,reason", SHAPES)
def test_shapes_refused(T, H, Hkv, hd, n_ctx, n_seq, reason):
    host = (ctypes.c_int32 * 4)()
    big = 1 << 60
    assert lib.llm_op_qk_norm_rope(P, 1 << 24, None, None, 1e-5, P, P, P, P, 0, P, P, 2, T, H, Hkv, hd, n_ctx, n_seq,
                                   None, None) == BAD and reason in why()
    assert lib.llm_op_attn_decode_q4_0(P, P, P, P, P, P, T, H, Hkv, hd, n_ctx, n_seq, 0, P, big, None, None) == BAD
    assert reason in why()
    assert lib.llm_op_attn_prefill_q4_0(P, P, P, host, host, P, T, H, Hkv, hd, n_ctx, n_seq, 0, P, big, None,
                                        None) == BAD and reason in why()
    assert lib.llm_op_attn_decode_q4_0_scratch_bytes(T, H, Hkv, hd, n_ctx, n_seq) == BAD
    assert lib.llm_op_attn_prefill_q4_0_scratch_bytes(T, H, Hkv, hd, n_ctx, n_seq) == BAD
    if H == 8 and Hkv == 2:
        assert lib.llm_op_kv_rows_q4_0(P, P, P, P, T, Hkv, hd, n_ctx, n_seq, None, None) == BAD and reason in why()
        if T:
            assert lib.llm_op_kv_q4_0_bytes(Hkv, hd, n_ctx, n_seq) == BAD


def test_sizes():
    assert lib.llm_op_kv_q4_0_bytes(8, 128, 32768, 2) == 2 * 8 * 32768 * 72
    assert lib.llm_op_kv_q4_0_bytes(1, 32, 1, 1) == 18
    assert 0 < lib.llm_op_attn_decode_q4_0_scratch_bytes(8, 32, 8, 128, 1 << 20, 8) < 1 << 25
    # two fp16 planes padded to 128 positions, and the row lists
    assert 2 * 3 * 2 * 128 * 64 * 2 <= lib.llm_op_attn_prefill_q4_0_scratch_bytes(9, 4, 2, 64, 100, 3) <= 2 * 3 * 2 * 128 * 64 * 2 + 4096


def test_arguments_refused():
    def qk(qkv=P, ld=768, eps=1e-5, rope=P, q=P, qt=0, k=P, kt=0, gain=None):
        return lib.llm_op_qk_norm_rope(qkv, ld, gain, None, eps, rope, P, P, q, qt, k, P, kt, 2, 8, 2, 64, 64, 1, None,
                                       None)
    for kw, reason in (({"qkv": None}, b"NULL"), ({"ld": 764}, b"ld"), ({"ld": 770}, b"ld"), ({"qt": 2}, b"q_type"),
                       ({"kt": 3}, b"kv_type"), ({"kt": -1}, b"kv_type"), ({"eps": -1.0}, b"eps"),
                       ({"eps": float("nan")}, b"eps"), ({"q": ODD}, b"aligned"), ({"k": ODD}, b"aligned"),
                       ({"gain": ODD}, b"aligned")):
        assert qk(**kw) == BAD and reason in why(), (kw, why())
    need = lib.llm_op_attn_decode_q4_0_scratch_bytes(2, 8, 2, 64, 64, 1)
    dec = lambda q=P, w=0, s=P, n=need, T=2: lib.llm_op_attn_decode_q4_0(q, P, P, P, P, P, T, 8, 2, 64, 64, 1, w, s, n,  # noqa: E731
                                                                         None, None)
    for kw, reason in (({"q": None}, b"NULL"), ({"w": -1}, b"window"), ({"s": None}, b"scratch"),
                       ({"n": need - 1}, b"scratch"), ({"q": ODD}, b"aligned"), ({"T": 4097}, b"T must")):
        assert dec(**kw) == BAD and reason in why(), (kw, why())
    assert lib.llm_op_attn_decode_q4_0_scratch_bytes(4097, 8, 2, 64, 64, 1) == BAD


def test_prefill_rows_refused():
    for pos, seq, reason in (([62, 63, 64], [0, 0, 0], b"n_ctx"), ([-1, 0], [0, 0], b"n_ctx"), ([0, 1], [2, 2], b"n_seq"),
                             ([0, 1], [-1, -1], b"n_seq"), ([0, 2], [0, 0], b"consecutive"), ([1, 0], [0, 0], b"consecutive"),
                             ([0, 5, 1], [0, 1, 0], b"consecutive"), ([0, 0], [0, 0], b"consecutive")):
        ph, sh = (ctypes.c_int32 * len(pos))(*pos), (ctypes.c_int32 * len(pos))(*seq)
        assert lib.llm_op_attn_prefill_q4_0(P, P, P, ph, sh, P, len(pos), 8, 2, 64, 64, 2, 0, P, 1 << 40, None,
                                            None) == BAD
        assert reason in why(), (pos, seq, why())


def test_oracle_head_norms_and_q4_model():
    """Normed heads have unit RMS before the gain, and the Q4_0 model's weights lie on their own grid."""
    rng = np.random.default_rng(2)
    hp = O.Hparams(64, 64, 1, 4, 2, 32, 40, 0.0, 1e4, False)
    q, k = rng.standard_normal((3, 4, 32)) * 5, rng.standard_normal((3, 2, 32))
    nq, nk = O.head_norms(hp, {"attn_q_norm": np.full(32, 2.0)}, q, k)
    assert np.allclose((nq * nq).mean(-1), 4.0) and np.array_equal(nk, k)
    w = {n: rng.standard_normal(s) for n, s in (
        ("token_embd", (64, 64)), ("output_norm", 64), ("output", (64, 64)), ("blk.0.attn_norm", 64), ("blk.0.attn_q", (128, 64)),
        ("blk.0.attn_k", (64, 64)), ("blk.0.attn_v", (64, 64)), ("blk.0.attn_output", (64, 128)), ("blk.0.ffn_norm", 64),
        ("blk.0.ffn_gate", (40, 64)), ("blk.0.ffn_up", (40, 64)), ("blk.0.ffn_down", (64, 40)))}
    m = O.Model(hp, w)
    for name in ("blk.0.attn_q", "blk.0.ffn_down", "output"):
        v = m.quantized_q4_0().w[name]
        full = np.pad(v, ((0, 0), (0, -v.shape[1] % 32)))
        assert v.shape == w[name].shape and not np.array_equal(v, w[name])
        # at most 16 levels a block, evenly spaced
        for block in full.reshape(-1, 32):
            levels = np.unique(block[block != 0])
            assert levels.size <= 15
    assert np.array_equal(m.quantized_q4_0().w["token_embd"], w["token_embd"])
    # rounding of the operands changes what a projection reads by half an fp16 step
    h = rng.standard_normal((2, 64))
    a, b = (O.norm_operand(h, w["blk.0.attn_norm"], 1e-5, o) for o in (None, "fp16"))
    assert 0 < np.abs(a - b).max() <= np.abs(a).max() * 2.0 ** -11


def test_cache_sizes_beyond_memory_refused():
    """Sizes whose products pass 64 bits are refused, not wrapped."""
    huge = (4096, 128, 1 << 30, (1 << 31) - 1)
    assert lib.llm_op_kv_q4_0_bytes(*huge) == BAD
    assert lib.llm_op_attn_prefill_q4_0_scratch_bytes(9, 4096, *huge) == BAD
    assert lib.llm_op_attn_decode_q4_0_scratch_bytes(1, 4096, *huge) == BAD
    assert lib.llm_op_kv_q4_0_bytes(1, 32, 1 << 30, 1 << 11) == 18 << 41


def test_prefill_of_many_sequences_needs_no_table():
    """A sequence's rows in two places are found whatever n_seq is (nothing of n_seq's size is kept on the host)."""
    ph, sh = ((ctypes.c_int32 * 3)(*v) for v in ((0, 0, 1), (5, (1 << 31) - 2, 5)))
    assert lib.llm_op_attn_prefill_q4_0(P, P, P, ph, sh, P, 3, 1, 1, 32, 64, (1 << 31) - 1, 0, P, 1 << 60, None,
                                        None) == BAD
    assert b"consecutive" in lib.llm_last_error(None)


def test_cache_type_refused():
    out = ctypes.c_void_p(123)
    assert lib.llm_kv_alloc_typed(None, 64, 1, 16, lib.LLM_KV_Q4_0, None, ctypes.byref(out)) == BAD and out.value is None
    for kv in (-1, 3):
        assert lib.llm_kv_alloc_typed(P, 64, 1, 16, kv, None, ctypes.byref(out)) == BAD and b"cache type" in why()
    assert lib.llm_kv_alloc_typed(P, 64, 1, 16, lib.LLM_KV_Q4_0, None, None) == BAD
