"""Models that answer out of 4 bits, end to end against the oracle: Q4_0 weights,
the Q4_0 cache, normed queries and keys, alone and together."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from gpu_model_util import LOGIT_TOL, MED64, MED128, compare_logits
from oracle import llama as O

pytestmark = pytest.mark.gpu

# head_dim 32 and a group of 3 query heads; the other shapes have groups of 2 and 4
MED32 = synth.Shape(n_vocab=640, n_embd=256, n_layer=2, n_head=8, n_head_kv=2, head_dim=32, n_ff=500, rms_eps=1e-5,
                    rope_theta=10000.0, tied_output=True)
WIDE = synth.Shape(n_vocab=1024, n_embd=512, n_layer=2, n_head=12, n_head_kv=4, head_dim=128, n_ff=1100, rms_eps=1e-5,
                   rope_theta=500000.0, tied_output=False)


@pytest.fixture(scope="module")
def lib():
    import llama_decoder_forward_02_gb300 as L
    return L


def stream():
    return torch.cuda.current_stream().cuda_stream


class Both:
    """The library's model and context and the oracle's, with the same weights."""

    def __init__(self, lib, shape, seed, n_ctx, n_seq=1, n_ubatch=64, weights=None, cache=None, norms="", window=0):
        self.lib, self.shape = lib, shape
        t = synth.make_weights(shape, seed, "cpu")
        g = torch.Generator().manual_seed(seed)
        gains = {n: [(1 + 0.2 * torch.randn(shape.head_dim, generator=g)).to(torch.bfloat16) for _ in range(shape.n_layer)]
                 for n in norms}
        host = synth.host_weights(t)
        for n, ts in gains.items():
            host.update({f"blk.{i}.attn_{n}_norm": v.view(torch.int16).numpy().view(np.uint16) for i, v in enumerate(ts)})
        self.model = lib.Model(shape, {k: v.cuda() for k, v in t.items()}, stream=stream())
        if norms:
            on_gpu = {n: [v.cuda() for v in ts] for n, ts in gains.items()}
            self.model.set_qk_norm(on_gpu.get("q"), on_gpu.get("k"), stream())
        if weights == "q4":
            self.model.quantize(lib.LLM_WTYPE_Q4_0, stream())
        self.ctx = lib.Context(self.model, n_ctx, n_seq, n_ubatch, stream=stream())
        om = O.Model(O.Hparams.of(shape), host)
        self.oc = O.Context(om.quantized_q4_0() if weights == "q4" else om, n_ctx, n_seq, n_ubatch,
                            kv_store="q4_0" if cache == "q4" else None, window=window)
        if cache == "q4":
            # A code is a decision: an element next to a border moves by a whole step, an eighth of its block's largest,
            # on a difference of any size.  The library reads its projections' operands as fp16 (2^-12 off on average,
            # one element in a thousand), so the oracle takes the same roundings and decides on the same values.
            self.oc.cache.operands = "fp16"
            self.ctx.set_option("kv_q4", 1)
        if window:
            self.ctx.set_option("swa_window", window)

    def logits(self):
        self.ctx.synchronize()
        return self.lib.logits_numpy(self.ctx, self.shape.n_vocab)

    def decode(self, tokens, **kw):
        assert self.ctx.decode(tokens, **kw) == 0
        kw = {{"seq_id": "seq"}.get(k, k): v for k, v in kw.items()}
        assert self.oc.decode(tokens, **kw) == 0
        got = self.logits()
        compare_logits(got, self.oc.logits)
        return got

    def free(self):
        self.ctx.free()
        self.model.free()


@pytest.mark.parametrize("shape,weights,cache,norms", [
    (MED64, "q4", None, ""), (MED128, "q4", None, ""), (MED32, "q4", None, "qk"), (MED64, None, "q4", ""),
    (MED128, None, "q4", "qk"), (MED64, None, None, "qk"), (MED128, None, None, "k"), (MED32, None, "q4", ""),
    (MED32, None, None, "q"), (MED64, "q4", "q4", "qk"), (MED128, "q4", "q4", "qk"), (WIDE, "q4", "q4", ""),
    (WIDE, None, "q4", "qk"),
])
def test_model(lib, shape, weights, cache, norms):
    """Prefill over ubatches, steps of one, two and eight rows (captured and replayed), a step with one output row,
    a context shift, and steps after it."""
    p = Both(lib, shape, 31, n_ctx=256, weights=weights, cache=cache, norms=norms)
    prompt = synth.prompt(shape.n_vocab, 31, 150)
    out = np.zeros(150, np.int8)
    out[[0, 63, 64, 149]] = 1
    p.decode(prompt, output=out)
    for tok in (3, 42, 7):
        p.decode([tok])
    p.decode([5, 6], output=[1, 1])
    p.decode([8, 9], output=[0, 1])
    p.decode(list(range(8)), output=[1] * 8)
    p.ctx.seq_shift(0, 20, 40)
    p.oc.seq_discard(0, 20, 40)
    p.decode([7])
    p.decode([11, 12, 13], output=[1] * 3)
    p.decode(synth.prompt(shape.n_vocab, 5, 70), output=[0] * 69 + [1])
    p.free()


@pytest.mark.parametrize("shape,weights,cache", [(MED64, "q4", "q4"), (MED128, None, "q4"), (MED32, "q4", "q4")])
def test_sequences_and_window(lib, shape, weights, cache):
    """Several sequences of different lengths in one batch, then steps of all of them at once, with a sliding window."""
    p = Both(lib, shape, 33, n_ctx=200, n_seq=3, n_ubatch=48, weights=weights, cache=cache, norms="qk", window=50)
    lens = [90, 7, 31]
    toks, seq = [], []
    for s, n in enumerate(lens):
        toks += list(synth.prompt(shape.n_vocab, 40 + s, n))
        seq += [s] * n
    out = np.zeros(len(toks), np.int8)
    out[np.cumsum(lens) - 1] = 1
    p.decode(toks, seq_id=seq, output=out)
    for step in range(4):
        p.decode([step, step + 1, step + 2], seq_id=[0, 1, 2], output=[1, 1, 1])
    p.decode([1, 2, 3, 4], seq_id=[2, 2, 2, 0], output=[1, 1, 1, 1])
    # a sequence begins again over the cells of the old one
    p.ctx.seq_clear(0)
    p.oc.seq_clear(0)
    p.decode(list(synth.prompt(shape.n_vocab, 50, 60)) + [9], seq_id=[0] * 60 + [1], output=[0] * 59 + [1, 1])
    p.decode([4, 5, 6], seq_id=[0, 1, 2], output=[1, 1, 1])
    p.free()


@pytest.mark.parametrize("shape,n_ctx", [(MED64, 8400), (WIDE, 8400)])
def test_long_cache(lib, shape, n_ctx):
    """A context whose rows share the keys' splits: sequences of unlike lengths, steps of one, two and eight rows."""
    p = Both(lib, shape, 36, n_ctx=n_ctx, n_seq=3, n_ubatch=256, weights="q4", cache="q4")
    lens = [400, 5, 130]
    toks, seq = [], []
    for s, n in enumerate(lens):
        toks += list(synth.prompt(shape.n_vocab, 60 + s, n))
        seq += [s] * n
    out = np.zeros(len(toks), np.int8)
    out[np.cumsum(lens) - 1] = 1
    p.decode(toks, seq_id=seq, output=out)
    for step in range(2):
        p.decode([step], seq_id=[step])
        p.decode([step, step + 1], seq_id=[0, 2], output=[1, 1])
        p.decode(list(range(8)), seq_id=[0, 1, 2, 2, 1, 0, 0, 2], output=[1] * 8)
    p.free()


def test_generate_and_options(lib):
    """Greedy steps on the device equal the same steps one call at a time; the fp16 copies of Q4_0 weights give the
    same logits up to one rounding; both caches of the context are refused together and changed while empty only."""
    a, b = (Both(lib, MED64, 35, n_ctx=128, weights="q4", cache="q4", norms="qk") for _ in range(2))
    prompt = synth.prompt(MED64.n_vocab, 35, 40)
    for x in (a, b):
        assert x.ctx.decode(prompt) == 0
    out = torch.zeros(12, dtype=torch.int32, device="cuda")
    a.ctx.generate(0, 12, out.data_ptr())
    last = a.logits()
    want = []
    for _ in range(12):
        want.append(b.ctx.argmax()[-1])
        assert b.ctx.decode([want[-1]]) == 0
    assert out.cpu().tolist() == want and np.array_equal(last, b.logits())
    times = {}
    a.ctx.kernel_timing(True)
    assert a.ctx.decode([1]) == 0
    a.ctx.synchronize()
    times = a.ctx.kernel_times()
    a.ctx.kernel_timing(False)
    assert times["qk_norm_rope_kv"][1] == MED64.n_layer and times["attn_decode"][1] == MED64.n_layer
    assert b.ctx.decode([1]) == 0
    b.ctx.set_option("gemv_q4", 0)
    assert b.ctx.decode([2]) == 0
    assert a.ctx.decode([2]) == 0
    assert np.abs(a.logits() - b.logits()).max() <= LOGIT_TOL
    with pytest.raises(lib.LlmError):
        a.ctx.set_option("kv_q4", 0)
    with pytest.raises(lib.LlmError):
        a.ctx.set_option("kv_q4", 2)
    a.ctx.seq_clear(0)
    with pytest.raises(lib.LlmError):
        a.ctx.set_option("kv_fp8", 1)
    a.ctx.set_option("kv_q4", 0)
    a.ctx.set_option("kv_fp8", 1)
    with pytest.raises(lib.LlmError):
        a.ctx.set_option("kv_q4", 1)
    a.ctx.set_option("kv_fp8", 0)
    a.oc.cache.store = a.oc.cache.operands = None
    a.oc.seq_clear(0)
    a.decode(prompt)
    a.decode([3])
    # a model with contexts takes neither gains nor another weight type
    with pytest.raises(lib.LlmError):
        a.model.quantize(lib.LLM_WTYPE_Q8_0)
    with pytest.raises(lib.LlmError):
        a.model.set_qk_norm([torch.ones(64, dtype=torch.bfloat16, device="cuda")] * 3)
    a.free()
    b.free()


def test_fp8_cache_with_norms(lib):
    """Normed queries and keys with the FP8 cache: the append of the same kernel."""
    p = Both(lib, MED128, 36, n_ctx=128, norms="qk")
    p.ctx.set_option("kv_fp8", 1)
    p.oc.cache.store = "e4m3"
    p.decode(synth.prompt(MED128.n_vocab, 36, 80))
    for tok in (3, 4):
        p.decode([tok])
    p.free()


@pytest.mark.parametrize("shape", [MED32, MED64, MED128])
def test_fp8_cache_of_q4_model(lib, shape):
    """Q4_0 weights with the FP8 cache: the append of the GEMV's own epilogue, for one and several rows and sequences."""
    p = Both(lib, shape, 37, n_ctx=128, n_seq=2, weights="q4")
    p.ctx.set_option("kv_fp8", 1)
    p.oc.cache.store = "e4m3"
    p.decode(synth.prompt(shape.n_vocab, 37, 60))
    for tok in (3, 4):
        p.decode([tok])
    p.decode([5, 6, 7], seq_id=[1, 1, 0], output=[1, 1, 1])
    p.decode(list(range(8)), seq_id=[0, 1] * 4, output=[1] * 8)
    p.decode([9], seq_id=[1])
    p.free()


@pytest.mark.parametrize("weights,n_ctx", [("q4", 600), (None, 600), ("q4", 8300)])
def test_overlapped_launches_change_nothing(lib, weights, n_ctx):
    """The norm's and the attention's launches overlap the kernels before them and read what stands since before those:
    the same bits as without the overlap, over steps of one and several rows, replayed and not."""
    a, b = (Both(lib, MED128, 38, n_ctx=n_ctx, n_seq=3, weights=weights, cache="q4", norms="qk") for _ in range(2))
    b.ctx.set_option("pdl_attn", 0)
    b.ctx.set_option("graphs", 0)
    toks = synth.prompt(MED128.n_vocab, 38, 300)
    for x in (a, b):
        assert x.ctx.decode(toks, seq_id=[0] * 200 + [1] * 90 + [2] * 10, output=[0] * 299 + [1]) == 0
    for step in range(30):
        for rows in ([step % 3], [0, 1, 1], [0, 1, 2, 2, 2, 1, 0, 0]):
            for x in (a, b):
                assert x.ctx.decode([(7 * step + i) % 500 for i in range(len(rows))], seq_id=rows, output=[1] * len(rows)) == 0
            assert np.array_equal(a.logits(), b.logits()), (step, rows)
    a.free()
    b.free()


def test_qk_norm_arguments(lib):
    t = synth.make_weights(MED64, 1, "cpu")
    m = lib.Model(MED64, {k: v.cuda() for k, v in t.items()}, stream=stream())
    one = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    ptrs = (ctypes.c_void_p * 3)(one.data_ptr(), None, one.data_ptr())
    assert lib.llm_model_set_qk_norm(None, ptrs, None, None) == lib.LLM_ERR_INVALID
    assert lib.llm_model_set_qk_norm(m.handle, None, None, None) == lib.LLM_ERR_INVALID
    assert lib.llm_model_set_qk_norm(m.handle, ptrs, None, None) == lib.LLM_ERR_INVALID
    with pytest.raises(ValueError):
        m.set_qk_norm([one])
    m.set_qk_norm([one] * 3, [one] * 3)
    m.set_qk_norm(None, [one * 2] * 3)                # replaces both
    m.free()
