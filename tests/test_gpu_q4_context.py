"""Contexts with a cache of 4 or 8 bits: made so from the start, and changed."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from gpu_model_util import MED64, MED128, compare_logits
from oracle import llama as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import llama_decoder_forward_02_gb300 as L
    return L


def stream():
    return torch.cuda.current_stream().cuda_stream


def make_model(lib, shape, seed, weights=None):
    t = synth.make_weights(shape, seed, "cpu")
    m = lib.Model(shape, {k: v.cuda() for k, v in t.items()}, stream=stream())
    om = O.Model(O.Hparams.of(shape), synth.host_weights(t))
    if weights == "q4":
        m.quantize(lib.LLM_WTYPE_Q4_0, stream())
        om = om.quantized_q4_0()
    return m, om


def logits(lib, ctx, shape):
    ctx.synchronize()
    return lib.logits_numpy(ctx, shape.n_vocab)


@pytest.mark.parametrize("weights", [None, "q4"])
@pytest.mark.parametrize("kind,option", [("LLM_KV_Q4_0", "kv_q4"), ("LLM_KV_E4M3", "kv_fp8"), ("LLM_KV_F16", None)])
def test_type_at_creation(lib, kind, option, weights):
    """A context made with a type equals one changed to it: prefill, steps of one and several rows, and back to fp16."""
    m, _ = make_model(lib, MED128, 51, weights)
    a = lib.Context(m, 300, 2, 64, stream=stream(), kv_type=getattr(lib, kind))
    b = lib.Context(m, 300, 2, 64, stream=stream())
    if option:
        b.set_option(option, 1)
    prompt = synth.prompt(MED128.n_vocab, 51, 200)
    for step in (dict(tokens=prompt), dict(tokens=[3]), dict(tokens=[4, 5, 6], seq_id=[0, 1, 1], output=[1, 1, 1])):
        for c in (a, b):
            assert c.decode(**step) == 0
        assert np.array_equal(logits(lib, a, MED128), logits(lib, b, MED128))
    if option:
        for s in (0, 1):
            a.seq_clear(s)
        a.set_option(option, 0)
        f = lib.Context(m, 300, 2, 64, stream=stream())
        for c in (a, f):
            assert c.decode(prompt) == 0 and c.decode([9]) == 0
        assert np.array_equal(logits(lib, a, MED128), logits(lib, f, MED128))
        f.free()
    a.free()
    b.free()
    m.free()


def test_memory_of_a_q4_context(lib):
    """The fp16 cache never exists: a context whose fp16 cache alone would not fit beside what the test leaves free."""
    m, _ = make_model(lib, MED64, 52)
    n_ctx = 1 << 20
    elems = MED64.n_layer * MED64.n_head_kv * n_ctx * MED64.head_dim
    f16, q4 = 2 * 2 * elems, 2 * (elems // 2 + elems // 16)
    rope = 2 * n_ctx * MED64.head_dim // 2 * 8
    torch.cuda.synchronize()
    before, _ = torch.cuda.mem_get_info()
    c = lib.Context(m, n_ctx, 1, 16, stream=stream(), kv_type=lib.LLM_KV_Q4_0)
    after, _ = torch.cuda.mem_get_info()
    assert before - after <= q4 + rope + (200 << 20) < f16, (before - after, q4, f16)
    # nothing but the caches grows with n_ctx: planes that prefill widens into would be n_ctx * Hkv * hd * 4 bytes
    assert c.decode(synth.prompt(MED64.n_vocab, 52, 70)) == 0
    c.synchronize()
    c.free()
    m.free()


def test_injected_failure_at_creation(lib):
    """Every device allocation of a Q4_0 context failing in turn: an error, no context, nothing held."""
    m, om = make_model(lib, MED64, 53)
    n_failed = 0
    for n in range(64):
        assert lib.llm_debug_fail_alloc(n) == 0
        out = ctypes.c_void_p()
        rc = lib.llm_kv_alloc_typed(m.handle, 64, 1, 16, lib.LLM_KV_Q4_0, ctypes.c_void_p(stream()), ctypes.byref(out))
        if rc == lib.LLM_OK:
            lib.llm_kv_free(out)
            break
        assert rc == lib.LLM_ERR_ALLOC and out.value is None
        n_failed += 1
    assert n_failed >= 12
    m.quantize(lib.LLM_WTYPE_Q4_0, stream())                    # needs a model without contexts
    m.free()


def test_failed_change_changes_nothing(lib):
    """Each device allocation of the change to Q4_0, and of the change back, failing in turn: the context goes on
    decoding with the cache it has, as the oracle does."""
    m, om = make_model(lib, MED64, 54)
    ctx = lib.Context(m, 64, 1, 16, stream=stream())
    prompt = synth.prompt(MED64.n_vocab, 54, 30)

    def check(store):
        oc = O.Context(om, 64, 1, 16, kv_store=store)
        if store:
            oc.cache.operands = "fp16"
        assert ctx.decode(prompt) == 0 and oc.decode(prompt) == 0
        compare_logits(logits(lib, ctx, MED64), oc.logits)
        assert ctx.decode([5]) == 0 and oc.decode([5]) == 0
        compare_logits(logits(lib, ctx, MED64), oc.logits)
        ctx.seq_clear(0)

    for want, allocs, store in ((1, 4, None), (0, 2, "q4_0")):
        for n in range(allocs):
            assert lib.llm_debug_fail_alloc(n) == 0
            with pytest.raises(lib.LlmError):
                ctx.set_option("kv_q4", want)
            check(store)
        ctx.set_option("kv_q4", want)
    check(None)
    ctx.free()
    m.free()


def test_failed_change_to_fp8_leaves_no_cache_to_use(lib):
    """The FP8 change frees the old cache first: where it fails, the calls that would use a cache refuse, and a later
    change brings one back."""
    m, om = make_model(lib, MED64, 55)
    ctx = lib.Context(m, 64, 1, 16, stream=stream())
    prompt = synth.prompt(MED64.n_vocab, 55, 30)
    assert ctx.decode(prompt) == 0 and ctx.decode([5]) == 0      # a captured step over the cache that goes
    ctx.synchronize()
    out = torch.zeros(4, dtype=torch.int32, device="cuda")
    for n in (0, 1):
        ctx.seq_clear(0)
        assert lib.llm_debug_fail_alloc(n) == 0
        with pytest.raises(lib.LlmError):
            ctx.set_option("kv_fp8", 1)
        for call in (lambda: ctx.decode([5]), lambda: ctx.decode(prompt), lambda: ctx.generate(0, 4, out.data_ptr()),
                     lambda: ctx.set_option("kv_q4", 1), lambda: ctx.seq_shift(0, 0, 1)):
            with pytest.raises(lib.LlmError):
                call()
        ctx.set_option("kv_fp8", 0)
        oc = O.Context(om, 64, 1, 16)
        for toks in (prompt, [5]):
            assert ctx.decode(toks) == 0 and oc.decode(toks) == 0
            compare_logits(logits(lib, ctx, MED64), oc.logits)
    ctx.free()
    m.free()
