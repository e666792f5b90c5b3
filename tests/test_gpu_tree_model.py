"""Trees of drafted tokens and rotations in every layout through the model, end to end against the oracle."""
import numpy as np
import pytest
import torch

import synth
import tree_util as U
from gpu_model_util import MED64, MED128, compare_logits
from oracle import llama as O
from test_gpu_q4_model import MED32, Both, stream

pytestmark = pytest.mark.gpu
# logits of one model computed over other kernels: the residual stream's fp16 operands differ by their rounding
FP8_TOL = 5e-2


@pytest.fixture(scope="module")
def lib():
    import llama_decoder_forward_02_gb300 as L
    return L


def path_of(par, node):
    p = [node]
    while par[p[0]] >= 0:
        p.insert(0, int(par[p[0]]))
    return p


def oracle_tree(p, prompts, trees, store=None, window=0):
    """The oracle's logits of each node: its sequence's prompt, then the tokens on the path to it."""
    out = []
    for s, tok, par in trees:
        for node in range(len(tok)):
            oc = O.Context(p.oc.model, p.oc.n_ctx, 1, p.oc.n_ubatch, kv_store=store, window=window)
            assert oc.decode(list(prompts[s]) + [int(tok[i]) for i in path_of(par, node)]) == 0
            out.append(oc.logits[-1])
    return np.array(out)


def draft(rng, shape, n, kind="random"):
    return rng.integers(0, shape.n_vocab, n), U.parents(rng, n, kind)


@pytest.mark.parametrize("shape,weights,norms,fp8,window,sizes,lens", [
    (MED64, None, "", 0, 0, [5], [40]),
    (MED64, None, "", 0, 0, [1], [17]),           # one row: the streamed GEMVs where they apply
    (MED128, None, "", 0, 0, [12], [150]),
    (MED128, None, "qk", 0, 0, [4, 9, 3], [20, 1, 130]),
    (MED32, None, "", 0, 0, [30], [33]),
    (MED64, "q4", "", 0, 0, [6], [50]),           # a step over the Q4_0 rows
    (MED64, "q4", "k", 0, 0, [14], [50]),
    (MED64, None, "", 1, 0, [7, 2], [60, 11]),
    (MED128, None, "", 1, 0, [11], [129]),
    (MED64, None, "", 0, 6, [20], [40]),          # a window
    (synth.TINY, None, "", 0, 2, [9], [10]),      # a window inside the tree
])
def test_tree_step(lib, shape, weights, norms, fp8, window, sizes, lens):
    rng = np.random.default_rng(len(sizes) + sizes[0])
    n_seq = len(sizes) + 1
    p = Both(lib, shape, 7, n_ctx=200, n_seq=n_seq, n_ubatch=64, weights=weights, norms=norms, window=window)
    if fp8:
        p.ctx.set_option("kv_fp8", 1)
    store = "e4m3" if fp8 else None
    prompts = {}
    seqs = [n_seq - 1 - i for i in range(len(sizes))]
    for s, n in zip(seqs, lens):
        prompts[s] = rng.integers(0, shape.n_vocab, n)
        assert p.ctx.decode(list(prompts[s]), seq_id=[s] * n) == 0
    kind = "chain" if window else "random"
    trees = [(s, *draft(rng, shape, n, kind if n < 12 else "random")) for s, n in zip(seqs, sizes)]
    tok = np.concatenate([t for _, t, _ in trees])
    par = np.concatenate([q for _, _, q in trees])
    assert p.ctx.decode_tree(sizes, tok, par, seqs) == 0
    assert [p.ctx.seq_pos_max(s) for s in seqs] == [n - 1 for n in lens]
    ref = oracle_tree(p, prompts, trees, store, window)
    compare_logits(p.logits(), ref)
    # accept the deepest path of each tree, then go on: steps of one row and another tree
    target = np.full(len(tok), -1)
    r, want = 0, []
    for s, t, q in trees:
        path = path_of(q, int(U.depths(q).argmax()))
        for a, b in zip(path, path[1:]):
            target[r + a] = t[b]
        target[r + path[-1]] = 5
        stand, nxt = U.accept(t, q, target[r:r + len(t)])
        want.append((stand, nxt))
        prompts[s] = np.concatenate((prompts[s], t[stand]))
        r += len(t)
    assert p.ctx.tree_accept(target) == want
    assert [p.ctx.seq_pos_max(s) for s in seqs] == [len(prompts[s]) - 1 for s in seqs]
    trees = [(s, np.array([5, 6, 7]), np.array([-1, 0, 0])) for s in seqs]
    assert p.ctx.decode_tree([3] * len(seqs), [5, 6, 7] * len(seqs), [-1, 0, 0] * len(seqs), seqs) == 0
    compare_logits(p.logits(), oracle_tree(p, prompts, trees, store, window))
    assert p.ctx.tree_accept([9] * 3 * len(seqs)) == [([0], 9)] * len(seqs)
    assert p.ctx.decode([9] * len(seqs), seq_id=seqs, output=[1] * len(seqs)) == 0
    ref = []
    for s in seqs:
        oc = O.Context(p.oc.model, 200, 1, 64, kv_store=store, window=window)
        assert oc.decode(list(prompts[s]) + [5, 9]) == 0
        ref.append(oc.logits[-1])
    compare_logits(p.logits(), np.array(ref))
    p.free()


@pytest.mark.parametrize("shape", [MED64, MED128])
def test_drafted_generation_is_greedy_generation(lib, shape):
    """Whatever is drafted, the tokens are those of one-by-one decoding (as far as the two largest logits are apart)."""
    steps = 40
    p = Both(lib, shape, 11, n_ctx=128)
    prompt = synth.prompt(shape.n_vocab, 11, 30)
    oc = p.oc
    ref, logits = O.generate_greedy(oc, prompt, steps)
    top = np.sort(logits, axis=1)
    sure = top[:, -1] - top[:, -2] > 0.1
    assert p.ctx.decode(list(prompt)) == 0
    rng = np.random.default_rng(0)
    toks, nxt = [], p.ctx.argmax()[-1]
    rounds = 0
    while len(toks) < steps:
        at = len(toks)
        if sure[at]:
            assert nxt == ref[at]
        nxt = int(ref[at])                          # keep to the oracle's tokens where the choice is open
        # a root, a guess of its followers (right for some steps), and children that are wrong
        good = [int(t) for t in ref[at + 1:at + 1 + int(rng.integers(0, 4))]]
        tok, par = [nxt] + good, [-1] + list(range(len(good)))
        for i in range(6):
            tok.append(int(rng.integers(0, shape.n_vocab)))
            par.append(int(rng.integers(0, i + 1)))
        assert p.ctx.decode_tree([len(tok)], tok, par) == 0
        target = p.ctx.argmax()
        for j in range(len(good)):                  # likewise
            if at + 1 + j < len(sure) and not sure[at + 1 + j]:
                target[j] = good[j]
        [(path, nxt)] = p.ctx.tree_accept(target)
        toks += [tok[i] for i in path]
        rounds += 1
    assert toks[:steps] == [int(t) for t in ref[:steps]]
    assert rounds < steps
    p.free()


def test_calls_that_drop_a_tree_and_refusals(lib):
    shape = MED64
    p = Both(lib, shape, 3, n_ctx=60, n_seq=2, n_ubatch=16)
    L = lib
    with pytest.raises(L.LlmError, match="no tree"):
        p.ctx.tree_nodes = [1]
        p.ctx.tree_accept([0])
    assert p.ctx.decode(list(range(50))) == 0
    before = p.logits().copy()
    for nodes, tok, par, seq, why in [
            ([0], [], [], None, "nodes"), ([17], [1] * 17, [-1] + [0] * 16, None, "ubatch"), ([2], [1, 2], [-1, 1], None, "parent"),
            ([2], [1, 2], [0, 0], None, "parent"), ([1], [shape.n_vocab], [-1], None, "token"), ([1], [-1], [-1], None, "token"),
            ([1, 1], [1, 2], [-1, -1], [1, 1], "seq_id"), ([1], [1], [-1], [2], "seq_id"),
            ([1] * 3, [1] * 3, [-1] * 3, [0, 1, 0], "more trees")]:
        with pytest.raises(L.LlmError, match=why):
            p.ctx.decode_tree(nodes, tok, par, seq)
    assert p.ctx.decode_tree([11], [1] * 11, [-1] + [0] * 10) == L.LLM_NO_KV_ROOM
    assert np.array_equal(p.logits(), before)
    tokens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for drop in (lambda: p.ctx.decode([1]), lambda: p.ctx.seq_clear(1), lambda: p.ctx.seq_shift(0, 0, 1)):
        assert p.ctx.decode_tree([2], [1, 2], [-1, 0]) == 0
        drop()
        with pytest.raises(L.LlmError, match="no tree"):
            p.ctx.tree_accept([0, 0])
    assert p.ctx.decode_tree([2], [1, 2], [-1, 0]) == 0
    with pytest.raises(L.LlmError, match="tree"):
        p.ctx.generate(0, 1, tokens.data_ptr())
    assert len(p.ctx.argmax()) == 2
    [(path, _)] = p.ctx.tree_accept([2, 3])
    assert path == [0, 1]
    with pytest.raises(L.LlmError, match="no tree"):
        p.ctx.tree_accept([2, 3])
    assert p.ctx.decode([1]) == 0 and p.ctx.generate(0, 2, tokens.data_ptr()) == 0
    p.ctx.synchronize()
    p.free()
    p = Both(lib, shape, 3, n_ctx=60, cache="q4")
    with pytest.raises(L.LlmError, match="fp16 or FP8"):
        p.ctx.decode_tree([1], [1], [-1])
    p.free()


def test_tree_beside_plain_steps(lib):
    """Plain steps after a tree give the bits that they give without one (captured graphs replayed among them)."""
    shape = MED128
    outs = []
    for tree in (False, True):
        p = Both(lib, shape, 5, n_ctx=100)
        assert p.ctx.decode(list(range(20))) == 0
        got = []
        for i in range(3):
            if tree:
                assert p.ctx.decode_tree([7], [3] * 7, [-1, 0, 0, 1, 1, 2, 5]) == 0   # not accepted
            assert p.ctx.decode([30 + i]) == 0
            got.append(p.logits())
        outs.append(got)
        p.free()
    assert all(np.array_equal(a, b) for a, b in zip(*outs))


# ---------------------------------------------------------------- rotations

@pytest.mark.parametrize("shape,layout,n_rot,scaling,weights,norms", [
    (MED64, 1, 64, 0, None, ""), (MED64, 1, 32, 2, None, "qk"), (MED128, 1, 128, 3, None, ""), (MED128, 0, 96, 1, None, ""),
    (MED64, 0, 64, 3, "q4", "q"), (MED32, 1, 24, 3, None, ""), (synth.TINY, 1, 32, 2, None, ""),
])
def test_model_rotation(lib, monkeypatch, shape, layout, n_rot, scaling, weights, norms):
    """Prefill, steps of one and several rows, a context shift and a tree with the model's own rotation."""
    orig, factor, theta = 64, 4.0, 20000.0
    f, m = U.frequencies(theta, n_rot, scaling, factor, 1.0, 4.0 if scaling == 2 else 32.0, orig)

    def rope(x, pos, _theta):
        pos = np.asarray(pos, np.float64)
        a = pos[:, None] * f
        # a shift turns back without the factor
        cs = np.stack((np.cos(a), np.sin(a)), -1) * np.where(pos < 0, 1.0, m)[:, None, None]
        return U.rotate(x, cs, n_rot, layout).astype(x.dtype)
    monkeypatch.setattr(O, "rope", rope)
    t = synth.make_weights(shape, 13, "cpu")
    g = torch.Generator().manual_seed(13)
    gains = {n: [(1 + 0.2 * torch.randn(shape.head_dim, generator=g)).to(torch.bfloat16) for _ in range(shape.n_layer)]
             for n in norms}
    host = synth.host_weights(t)
    for n, ts in gains.items():
        host.update({f"blk.{i}.attn_{n}_norm": v.view(torch.int16).numpy().view(np.uint16) for i, v in enumerate(ts)})
    model = lib.Model(shape, {k: v.cuda() for k, v in t.items()}, stream=stream())
    r = lib.rope(theta, n_rot, layout, scaling, factor, n_ctx_orig=orig)
    model.set_rope(r, stream())
    with pytest.raises(lib.LlmError, match="already"):
        model.set_rope(r, stream())
    if norms:
        on_gpu = {n: [v.cuda() for v in ts] for n, ts in gains.items()}
        model.set_qk_norm(on_gpu.get("q"), on_gpu.get("k"), stream())
    om = O.Model(O.Hparams.of(shape), host)
    if weights:
        model.quantize(lib.LLM_WTYPE_Q4_0, stream())
        om = om.quantized_q4_0()
    ctx = lib.Context(model, 160, 1, 64, stream=stream())
    oc = O.Context(om, 160, 1, 64)

    def both(tokens, output=None):
        assert ctx.decode(list(tokens), output=output) == 0 and oc.decode(tokens, output=output) == 0
        ctx.synchronize()
        compare_logits(lib.logits_numpy(ctx, shape.n_vocab), oc.logits)
    both(synth.prompt(shape.n_vocab, 1, 90))
    both([4])
    both([5, 6], [1, 1])
    ctx.seq_shift(0, 10, 25)
    oc.seq_discard(0, 10, 25)
    both([7])
    assert ctx.decode_tree([3], [8, 9, 10], [-1, 0, 0]) == 0
    assert ctx.tree_accept([10, 0, 0]) == [([0, 2], 0)]
    assert oc.decode([8]) == 0 and oc.decode([10]) == 0
    both([11])
    both(synth.prompt(shape.n_vocab, 2, 30))
    ctx.free()
    model.free()


def test_set_rope_refused(lib):
    shape = MED64
    t = {k: v.cuda() for k, v in synth.make_weights(shape, 0, "cpu").items()}
    r = lib.rope(10000.0, 64)
    for late in ("quantize", "norm", "context"):
        m = lib.Model(shape, t, stream=stream())
        with pytest.raises(lib.LlmError, match="n_rot"):
            m.set_rope(lib.rope(10000.0, 72), stream())
        ctx = None
        if late == "quantize":
            m.quantize(None, stream())
        elif late == "norm":
            m.set_qk_norm([torch.ones(64, dtype=torch.bfloat16, device="cuda")] * shape.n_layer, None, stream())
        else:
            ctx = lib.Context(m, 16, 1, 16, stream=stream())
        with pytest.raises(lib.LlmError, match="comes before|live contexts"):
            m.set_rope(r, stream())
        if ctx:
            ctx.free()
        m.free()
