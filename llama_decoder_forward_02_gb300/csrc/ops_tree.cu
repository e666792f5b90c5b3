// C entry points of drafted decoding, one call at a time: rotary tables and the
// rotation in every layout, attention of trees of drafted tokens, and the
// acceptance of a tree's path.  Argument checks come before any device work;
// nothing here allocates device memory or waits for the stream.
#include <cmath>

#include "kernels.h"
#include "launch.cuh"
#include "ops.h"

using namespace llm;

namespace llm {

// What is wrong with a rotation, or null.
const char *rope_error(const llm_rope *r, int hd) {
    if (!r) return "rope is NULL";
    if (r->n_rot < 8 || r->n_rot > hd || r->n_rot % 8) return "n_rot must be a multiple of 8, at least 8 and at most head_dim";
    if (r->layout != LLM_ROPE_PAIRS && r->layout != LLM_ROPE_HALVES) return "unknown layout";
    if (r->scaling < LLM_ROPE_NONE || r->scaling > LLM_ROPE_RAMP) return "unknown scaling";
    if (!(r->theta > 1.f) || !std::isfinite(r->theta)) return "theta must be above 1";
    if (r->scaling != LLM_ROPE_NONE && (!(r->factor >= 1.f) || !std::isfinite(r->factor))) return "factor must be at least 1";
    if (r->scaling >= LLM_ROPE_BANDS) {
        if (r->n_ctx_orig < 1) return "n_ctx_orig must be positive";
        if (!(r->slow > 0.f) || !(r->fast > r->slow) || !std::isfinite(r->fast)) return "slow must be positive and fast above it";
    }
    if (!(r->attn_factor >= 0.f) || !std::isfinite(r->attn_factor)) return "attn_factor must not be negative";
    return nullptr;
}

RopeSpec rope_spec(const llm_rope &r) {
    return RopeSpec{r.theta, r.n_rot, r.scaling, r.factor, r.slow, r.fast, r.n_ctx_orig, r.attn_factor};
}

}  // namespace llm

namespace {

// One layer's fp16 or FP8 caches as the kernels see them.
KvView layer_view(const void *k, const void *v, int kv_type, int Hkv, int hd, int n_ctx, int n_seq) {
    KvView kv;
    kv.k = kv.v = nullptr;
    kv.seq_stride = (long long)Hkv * n_ctx * hd;
    kv.n_ctx = n_ctx; kv.n_seq = n_seq; kv.head_dim = hd; kv.n_kv_head = Hkv;
    if (kv_type == LLM_KV_F16) { kv.k = (f16 *)k; kv.v = (f16 *)v; }
    if (kv_type == LLM_KV_E4M3) { kv.k8 = (uint8_t *)k; kv.v8 = (uint8_t *)v; }
    if (kv_type == LLM_KV_Q4_0) {
        const size_t codes = (size_t)n_seq * Hkv * n_ctx * (hd / 2);
        kv.k4 = (uint8_t *)k; kv.v4 = (uint8_t *)v;
        kv.kd = (f16 *)(kv.k4 + codes); kv.vd = (f16 *)(kv.v4 + codes);
    }
    return kv;
}

const char *tree_error(int n_tree, int max_nodes) {
    if (n_tree < 1 || n_tree > 4096) return "n_tree must be 1..4096";
    if (max_nodes < 1 || max_nodes > TREE_MAX_NODES) return "max_nodes must be 1..256";
    return nullptr;
}
const char *attn_tree_error(int n_tree, int max_nodes, int H, int Hkv) {
    if (const char *why = tree_error(n_tree, max_nodes)) return why;
    const long long groups = (long long)n_tree * Hkv * (((long long)max_nodes * (H / Hkv) + 127) / 128);
    return groups > 65535 ? "the trees have more than 65535 groups of 128 rows of a kv head" : nullptr;
}

}  // namespace

extern "C" int32_t llm_op_rope_table(const llm_rope *rope, int32_t pos0, int32_t n_pos, float *out, void *stream) {
    const char *who = "llm_op_rope_table";
    if (const char *why = rope_error(rope, 128)) return refuse(who, why);
    if (!out) return refuse(who, "a pointer is NULL");
    if (pos0 < 0 || n_pos < 1 || (long long)pos0 + n_pos > (1 << 30)) return refuse(who, "positions must lie in [0, 2^30)");
    if (!aligned(out, 16)) return refuse(who, "out must be 16-byte aligned");
    return launched(who, launch_rope_table(rope_spec(*rope), pos0, n_pos, rope->n_rot / 2, (float2 *)out, nullptr, overlapped(stream)));
}

extern "C" int32_t llm_op_rope_kv(const float *qkv, int32_t ld, const float *q_gain, const float *k_gain, float eps,
                                  const float *rope, int32_t n_pos, int32_t n_rot, int32_t layout, const int32_t *pos,
                                  const int32_t *cell, const int32_t *seq, void *q, int32_t q_type, void *k_cache,
                                  void *v_cache, int32_t kv_type, int32_t T, int32_t H, int32_t Hkv, int32_t hd,
                                  int32_t n_ctx, int32_t n_seq, uint32_t *err, void *stream) {
    const char *who = "llm_op_rope_kv";
    if (!qkv || !rope || !pos || !seq || !q || !k_cache || !v_cache) return refuse(who, "a pointer is NULL");
    if (const char *why = shape_error(T, H, Hkv, hd, n_ctx, n_seq)) return refuse(who, why);
    if (ld < (H + 2 * Hkv) * hd || ld % 4) return refuse(who, "ld must be a multiple of 4 and hold every head");
    if (n_pos < 1 || n_pos > (1 << 30)) return refuse(who, "n_pos must be 1..2^30");
    if (n_rot < 8 || n_rot > hd || n_rot % 8) return refuse(who, "n_rot must be a multiple of 8, at least 8 and at most head_dim");
    if (layout != LLM_ROPE_PAIRS && layout != LLM_ROPE_HALVES) return refuse(who, "unknown layout");
    if (q_type != LLM_Q_F32 && q_type != LLM_Q_F16) return refuse(who, "unknown q_type");
    if (kv_type < LLM_KV_F16 || kv_type > LLM_KV_Q4_0) return refuse(who, "unknown kv_type");
    if (!(eps >= 0.f)) return refuse(who, "eps must not be negative");
    if (!aligned(qkv, 16) || !aligned(q_gain, 16) || !aligned(k_gain, 16) || !aligned(rope, 16) || !aligned(q, 16) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return refuse(who, "qkv, gains, rope, q and the caches must be 16-byte aligned");
    QkNormArgs a;
    a.qkv = qkv; a.ld = ld; a.q_gain = q_gain; a.k_gain = k_gain; a.eps = eps;
    a.rope = (const float2 *)rope; a.pos = pos; a.seq = seq; a.cell = cell;
    a.n_pos = n_pos; a.n_rot = n_rot; a.halves = layout == LLM_ROPE_HALVES;
    a.q32 = q_type == LLM_Q_F32 ? (float *)q : nullptr;
    a.q16 = q_type == LLM_Q_F16 ? (f16 *)q : nullptr;
    a.kv = layer_view(k_cache, v_cache, kv_type, Hkv, hd, n_ctx, n_seq);
    a.T = T; a.H = H; a.err = err;
    return launched(who, launch_qk_norm_rope(a, overlapped(stream)));
}

extern "C" int64_t llm_op_attn_tree_scratch_bytes(int32_t n_tree, int32_t max_nodes, int32_t H, int32_t Hkv, int32_t hd,
                                                  int32_t n_ctx) {
    if (shape_error(1, H, Hkv, hd, n_ctx, 1) || attn_tree_error(n_tree, max_nodes, H, Hkv)) return LLM_ERR_INVALID;
    return (int64_t)attn_tree_scratch_bytes(n_tree, max_nodes, H, Hkv, hd, n_ctx);
}

extern "C" int32_t llm_op_attn_tree(const void *q, const void *k_cache, const void *v_cache, const int32_t *row0,
                                    const int32_t *seq, const int32_t *base, const uint32_t *mask, const int32_t *pos,
                                    void *o, int32_t T, int32_t n_tree, int32_t max_nodes, int32_t H, int32_t Hkv,
                                    int32_t hd, int32_t n_ctx, int32_t n_seq, int32_t kv_type, int32_t window,
                                    void *scratch, int64_t scratch_bytes, uint32_t *err, void *stream) {
    const char *who = "llm_op_attn_tree";
    if (!q || !k_cache || !v_cache || !row0 || !seq || !base || !mask || !o) return refuse(who, "a pointer is NULL");
    if (const char *why = shape_error(T, H, Hkv, hd, n_ctx, n_seq)) return refuse(who, why);
    if (const char *why = attn_tree_error(n_tree, max_nodes, H, Hkv)) return refuse(who, why);
    if (kv_type != LLM_KV_F16 && kv_type != LLM_KV_E4M3) return refuse(who, "kv_type must be LLM_KV_F16 or LLM_KV_E4M3");
    if (window < 0) return refuse(who, "window must not be negative");
    if (window > 0 && !pos) return refuse(who, "a window needs pos");
    if ((double)n_seq * Hkv * n_ctx > 2147483000.0) return refuse(who, "the cache has more than 2^31 rows");
    if (!scratch || scratch_bytes < llm_op_attn_tree_scratch_bytes(n_tree, max_nodes, H, Hkv, hd, n_ctx))
        return refuse(who, "scratch is NULL or smaller than llm_op_attn_tree_scratch_bytes");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(scratch, 16))
        return refuse(who, "q, the caches, o and scratch must be 16-byte aligned");
    if (cudaError_t e = init_kernel_attributes()) return launched(who, e);
    AttnTreeArgs a;
    a.q = (const f16 *)q;
    a.kv = layer_view(k_cache, v_cache, kv_type, Hkv, hd, n_ctx, n_seq);
    a.row0 = row0; a.seq = seq; a.base = base; a.mask = mask; a.pos = pos; a.o = (f16 *)o;
    a.T = T; a.n_tree = n_tree; a.max_nodes = max_nodes; a.words = (max_nodes + 31) / 32; a.H = H; a.window = window;
    a.scratch = scratch; a.err = err;
    TmaMap mk, mv;
    const long long rows = (long long)n_seq * Hkv * n_ctx;
    const bool made = kv_type == LLM_KV_F16 ? make_cache_map(&mk, a.kv.k, rows, hd) && make_cache_map(&mv, a.kv.v, rows, hd)
                                            : make_cache8_map(&mk, a.kv.k8, rows, hd) && make_cache8_map(&mv, a.kv.v8, rows, hd);
    if (!made) {
        set_global_error("llm_op_attn_tree: TMA descriptor creation failed");
        return LLM_ERR_COMPUTE;
    }
    return launched(who, launch_attn_tree(a, mk, mv, overlapped(stream)));
}

extern "C" int32_t llm_op_tree_accept(const int32_t *token, const int32_t *parent, const int32_t *target,
                                      const int32_t *row0, const int32_t *seq, const int32_t *base, void *k_cache,
                                      void *v_cache, int32_t kv_type, int32_t *path, int32_t *n_accept, int32_t *next,
                                      int32_t T, int32_t n_tree, int32_t max_nodes, int32_t n_layer, int32_t Hkv,
                                      int32_t hd, int32_t n_ctx, int32_t n_seq, uint32_t *err, void *stream) {
    const char *who = "llm_op_tree_accept";
    if (!token || !parent || !target || !row0 || !seq || !base || !k_cache || !v_cache || !path || !n_accept || !next)
        return refuse(who, "a pointer is NULL");
    if (const char *why = shape_error(T, Hkv, Hkv, hd, n_ctx, n_seq)) return refuse(who, why);
    if (const char *why = tree_error(n_tree, max_nodes)) return refuse(who, why);
    if (n_layer < 1 || (long long)n_layer * Hkv > 65535) return refuse(who, "n_layer * n_head_kv must be 1..65535");
    if ((double)n_seq * n_layer * Hkv * n_ctx * hd > 0x1p46) return refuse(who, "the cache has more than 2^46 elements");
    if (kv_type < LLM_KV_F16 || kv_type > LLM_KV_Q4_0) return refuse(who, "unknown kv_type");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return refuse(who, "the caches must be 16-byte aligned");
    TreeAcceptArgs a;
    a.token = token; a.parent = parent; a.target = target; a.row0 = row0; a.seq = seq; a.base = base;
    a.k = k_cache; a.v = v_cache; a.kv_type = kv_type; a.path = path; a.n_accept = n_accept; a.next = next;
    a.T = T; a.n_tree = n_tree; a.max_nodes = max_nodes; a.heads = n_layer * Hkv; a.head_dim = hd;
    a.n_ctx = n_ctx; a.n_seq = n_seq; a.err = err;
    return launched(who, launch_tree_accept(a, overlapped(stream)));
}
