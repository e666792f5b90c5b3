"""Paths of the Q4_0 cache and of normed queries and keys that meet other weights
and other shapes: Q8_0 weights (streamed GEMVs that let their successor start before
their own dependency wait), and launches that read ahead of the kernel before them
at head_dim 64, with windows and with cell counts that no line of scales ends on."""
import numpy as np
import pytest
import torch

import synth
from gpu_model_util import MED64, MED128, compare_logits
from oracle import llama as O
from test_gpu_q4_model import MED32, WIDE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import llama_decoder_forward_02_gb300 as L
    return L


def stream():
    return torch.cuda.current_stream().cuda_stream


def make(lib, shape, seed, weights, norms="", rounded=False):
    """The library's model and the oracle's; weights None, "q8" or "q4".  rounded: the oracle's encoded weights as the
    library's prefill reads them, rounded to fp16.  Over a Q4_0 cache that decides codes: of the oracle's own logits
    behind 100 tokens of MED128 with Q8_0 weights and norms the rounding moves some by 0.061, and by 0.0012 where the
    cache is not encoded."""
    t = synth.make_weights(shape, seed, "cpu")
    g = torch.Generator().manual_seed(seed)
    gains = {n: [(1 + 0.2 * torch.randn(shape.head_dim, generator=g)).to(torch.bfloat16) for _ in range(shape.n_layer)]
             for n in norms}
    host = synth.host_weights(t)
    for n, ts in gains.items():
        host.update({f"blk.{i}.attn_{n}_norm": v.view(torch.int16).numpy().view(np.uint16) for i, v in enumerate(ts)})
    m = lib.Model(shape, {k: v.cuda() for k, v in t.items()}, stream=stream())
    if norms:
        on_gpu = {n: [v.cuda() for v in ts] for n, ts in gains.items()}
        m.set_qk_norm(on_gpu.get("q"), on_gpu.get("k"), stream())
    om = O.Model(O.Hparams.of(shape), host)
    if weights:
        m.quantize(lib.LLM_WTYPE_Q8_0 if weights == "q8" else lib.LLM_WTYPE_Q4_0, stream())
        om = om.quantized_q8_0() if weights == "q8" else om.quantized_q4_0()
        if rounded:
            om.w = {k: v.astype(np.float16).astype(v.dtype) if v.dtype.kind == "f" else v for k, v in om.w.items()}
    return m, om


@pytest.mark.parametrize("shape,cache,norms", [
    (MED64, "q4", ""), (MED128, "q4", "qk"), (MED128, None, "qk"), (MED32, "q4", "k"), (MED64, None, "q"), (WIDE, "q4", "qk"),
])
def test_q8_weights(lib, shape, cache, norms):
    """Q8_0 weights with the Q4_0 cache and with normed heads: prefill, one-row steps (streamed Q8_0 rows), steps of
    several rows, a context shift, and greedy steps on the device."""
    m, om = make(lib, shape, 61, "q8", norms, rounded=cache is not None)
    ctx = lib.Context(m, 200, 1, 64, stream=stream(), kv_type=lib.LLM_KV_Q4_0 if cache else lib.LLM_KV_F16)
    oc = O.Context(om, 200, 1, 64, kv_store="q4_0" if cache else None)
    if cache:
        oc.cache.operands = "fp16"                              # the oracle decides codes on the values the library reads

    def step(tokens, **kw):
        assert ctx.decode(tokens, **kw) == 0 and oc.decode(tokens, **kw) == 0
        ctx.synchronize()
        compare_logits(lib.logits_numpy(ctx, shape.n_vocab), oc.logits)

    step(synth.prompt(shape.n_vocab, 61, 100))
    for tok in (3, 42, 7):
        step([tok])
    step([5, 6], output=[1, 1])
    ctx.seq_shift(0, 20, 40)
    oc.seq_discard(0, 20, 40)
    step([7])
    step(list(range(8)), output=[1] * 8)
    step([9])
    out = torch.zeros(6, dtype=torch.int32, device="cuda")
    first = int(oc.logits[-1].argmax())
    ctx.generate(0, 6, out.data_ptr())
    ctx.synchronize()
    top = np.sort(oc.logits[-1])
    if top[-1] - top[-2] > 0.1:
        assert int(out[0]) == first
    ctx.free()
    m.free()


@pytest.mark.parametrize("shape,weights,cache,norms,n_ctx,window", [
    (MED64, "q4", "q4", "", 611, 0), (MED64, "q4", "q4", "qk", 611, 37), (MED64, None, "q4", "qk", 8301, 0),
    (MED64, "q4", "q4", "", 8301, 53), (MED32, "q4", "q4", "qk", 503, 21), (MED128, "q8", "q4", "qk", 611, 0),
    (MED64, "q8", "q4", "", 611, 37), (MED64, "q8", None, "qk", 400, 0), (MED128, "q4", "q4", "", 605, 50),
])
def test_overlapped_launches_change_nothing(lib, shape, weights, cache, norms, n_ctx, window):
    """The same bits as without the overlap, over steps of one and several rows, replayed and not."""
    m, _ = make(lib, shape, 62, weights, norms)
    a, b = (lib.Context(m, n_ctx, 3, 64, stream=stream(), kv_type=lib.LLM_KV_Q4_0 if cache else lib.LLM_KV_F16) for _ in range(2))
    for c in (a, b):
        c.set_option("swa_window", window)
    b.set_option("pdl_attn", 0)
    b.set_option("pdl_prefill", 0)
    b.set_option("graphs", 0)
    toks = synth.prompt(shape.n_vocab, 62, 300)
    for c in (a, b):
        assert c.decode(toks, seq_id=[0] * 200 + [1] * 90 + [2] * 10, output=[0] * 299 + [1]) == 0
    got = []
    for i in range(25):
        for rows in ([i % 3], [0, 1, 1], [0, 1, 2, 2, 2, 1, 0, 0]):
            got = []
            for c in (a, b):
                assert c.decode([(7 * i + j) % 500 for j in range(len(rows))], seq_id=rows, output=[1] * len(rows)) == 0
                c.synchronize()
                got.append(lib.logits_numpy(c, shape.n_vocab))
            assert np.array_equal(*got), (i, rows)
        if i == 12:                                             # a prompt among the steps, over two ubatches
            more = synth.prompt(shape.n_vocab, 63, 90)
            for c in (a, b):
                assert c.decode(more, seq_id=[1] * 90, output=[0] * 89 + [1]) == 0
    a.free()
    b.free()
    m.free()


@pytest.mark.parametrize("cache,norms", [("q4", ""), (None, "qk")])
def test_output_rows_do_not_change_a_step(lib, cache, norms):
    """A step of several rows gives a row the same bits whichever rows are outputs, leaves the same cache, and hands out
    the hidden rows of the outputs; a step without outputs counts too."""
    shape = MED128
    m, _ = make(lib, shape, 64, "q4", norms)
    a, b = (lib.Context(m, 100, 2, 16, stream=stream(), kv_type=lib.LLM_KV_Q4_0 if cache else lib.LLM_KV_F16) for _ in range(2))
    prompt = synth.prompt(shape.n_vocab, 64, 20)
    for c in (a, b):
        assert c.decode(prompt) == 0
    hidden = [torch.zeros((1, shape.n_layer, 8, shape.n_embd), device="cuda") for _ in range(2)]
    for out in ([0, 1], [1, 0, 1, 1, 0, 0, 0, 1], [0, 0, 1, 0, 0], [0, 0, 0]):
        n = len(out)
        toks, seq = list(range(7, 7 + n)), [0, 1, 1, 0, 0, 0, 1, 0][:n]
        for c, o, h in ((a, [1] * n, hidden[0]), (b, out, hidden[1])):
            if n in (8, 3):
                lib.check(lib.llm_debug_hidden(c.handle, h.data_ptr(), 8, 1), c.handle)
            assert c.decode(toks, seq_id=seq, output=o) == 0
            c.synchronize()
            if n in (8, 3):
                lib.check(lib.llm_debug_hidden(c.handle, None, 0, 0), c.handle)
        rows = [i for i in range(n) if out[i]]
        if rows:
            assert np.array_equal(lib.logits_numpy(a, shape.n_vocab)[rows], lib.logits_numpy(b, shape.n_vocab))
        if n == 8:
            assert torch.equal(hidden[0][:, :-1], hidden[1][:, :-1])
            assert torch.equal(hidden[0][:, -1, rows], hidden[1][:, -1, :len(rows)]) and not hidden[1][:, -1, len(rows):].any()
    for c in (a, b):
        assert c.decode([3]) == 0
        c.synchronize()
    assert np.array_equal(lib.logits_numpy(a, shape.n_vocab), lib.logits_numpy(b, shape.n_vocab))
    for c in (a, b):
        c.free()
    m.free()
