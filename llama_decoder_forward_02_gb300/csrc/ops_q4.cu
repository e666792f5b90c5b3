// C entry points of the 4-bit kernels, one call at a time: Q4_0 weights, the
// per-head query/key norm with rotation and cache append, and attention over
// a Q4_0 cache.  Argument checks come before any device work; nothing here
// allocates device memory or waits for the stream.
#include <algorithm>
#include <new>
#include <string>
#include <vector>

#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "../../include/llm.h"

namespace llm {
void set_global_error(const char *msg);
}

using namespace llm;

namespace {

int32_t refuse(const char *who, const char *why) {
    set_global_error((std::string(who) + ": " + why).c_str());
    return LLM_ERR_INVALID;
}

int32_t launched(const char *who, cudaError_t e) {
    if (!e) return LLM_OK;
    set_global_error((std::string(who) + ": " + cudaGetErrorString(e)).c_str());
    return LLM_ERR_COMPUTE;
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The kernels of these calls wait for the previous one before they touch
// memory, so their launches may overlap its end (programmatic dependent
// launch): calls in a row then follow each other without the gap of a launch,
// 2 to 4 us.
Launch overlapped(void *stream) { return Launch{(cudaStream_t)stream, true, nullptr}; }

int current_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}

// What is wrong with the shape of one layer's heads and cache, or null.
const char *shape_error(int T, int H, int Hkv, int hd, int n_ctx, int n_seq) {
    if (T < 1) return "T must be positive";
    if (hd != 32 && hd != 64 && hd != 128) return "head_dim must be 32, 64 or 128";
    if (Hkv < 1 || H < 1 || H % Hkv) return "n_head must be a positive multiple of n_head_kv";
    if (H > 4096) return "n_head must be at most 4096";
    if (n_ctx < 1 || n_seq < 1) return "n_ctx and n_seq must be positive";
    if (n_ctx > (1 << 30)) return "n_ctx must be at most 2^30";
    if ((double)n_seq * Hkv * n_ctx * hd > 0x1p46) return "the cache has more than 2^46 elements";
    return nullptr;
}

size_t cache_rows(int n_seq, int Hkv, int n_ctx) { return (size_t)n_seq * Hkv * n_ctx; }

// One layer's Q4_0 caches as the kernels see them: codes, then scales.
KvView q4_view(const void *k, const void *v, int Hkv, int hd, int n_ctx, int n_seq) {
    KvView kv;
    kv.k = kv.v = nullptr;
    kv.seq_stride = (long long)Hkv * n_ctx * hd;
    kv.n_ctx = n_ctx; kv.n_seq = n_seq; kv.head_dim = hd; kv.n_kv_head = Hkv;
    const size_t codes = cache_rows(n_seq, Hkv, n_ctx) * (hd / 2);
    kv.k4 = (uint8_t *)k; kv.v4 = (uint8_t *)v;
    kv.kd = (f16 *)(kv.k4 + codes); kv.vd = (f16 *)(kv.v4 + codes);
    return kv;
}

constexpr int DECODE_MAX_T = 4096;

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

int padded_ctx(int n_ctx) { return (n_ctx + 127) / 128 * 128; }

}  // namespace

extern "C" int32_t llm_op_quantize_q4_0(const void *W, int32_t N, int32_t K, void *out, void *stream) {
    const char *who = "llm_op_quantize_q4_0";
    if (!W || !out) return refuse(who, "a pointer is NULL");
    if (N < 1 || K < 256 || K % 256) return refuse(who, "N must be positive and K a positive multiple of 256");
    if (!aligned(W, 16) || !aligned(out, 16)) return refuse(who, "W and out must be 16-byte aligned");
    // write_back is off: W is only read
    return launched(who, launch_quantize_q4_0((f16 *)W, N, K, (uint8_t *)out, false, (cudaStream_t)stream));
}

extern "C" int32_t llm_op_gemv_q4_0(const void *Wq, const void *x, float *y, int32_t N, int32_t K, int32_t T,
                                    int32_t ldx, int32_t ldy, void *stream) {
    const char *who = "llm_op_gemv_q4_0";
    if (!Wq || !x || !y) return refuse(who, "a pointer is NULL");
    if (T < 1 || T > 8) return refuse(who, "T must be 1..8");
    if (N < 1 || K < 256 || K % 256 || K > (1 << 24))
        return refuse(who, "N must be positive and K a positive multiple of 256, at most 2^24");
    if (ldx < K || ldx % 8 || ldy < N) return refuse(who, "ldx must be a multiple of 8 and at least K, ldy at least N");
    if (!aligned(Wq, 16) || !aligned(x, 16) || !aligned(y, 4))
        return refuse(who, "Wq and x must be 16-byte aligned, y 4-byte");
    if (cudaError_t e = init_kernel_attributes()) return launched(who, e);
    GemvQ4Args a = {};
    a.W = (const uint8_t *)Wq; a.N = N; a.K = K; a.T = T;
    a.x = (const f16 *)x; a.ldx = ldx; a.out = y; a.ldo = ldy;
    return launched(who, launch_gemv_q4(EPI_STORE, a, current_sms(), overlapped(stream), false));
}

extern "C" int64_t llm_op_kv_q4_0_bytes(int32_t Hkv, int32_t hd, int32_t n_ctx, int32_t n_seq) {
    if (shape_error(1, Hkv, Hkv, hd, n_ctx, n_seq)) return LLM_ERR_INVALID;
    return (int64_t)(cache_rows(n_seq, Hkv, n_ctx) * (hd / 2 + hd / 16));
}

extern "C" int32_t llm_op_qk_norm_rope(const float *qkv, int32_t ld, const float *q_gain, const float *k_gain, float eps,
                                       const float *rope, const int32_t *pos, const int32_t *seq, void *q,
                                       int32_t q_type, void *k_cache, void *v_cache, int32_t kv_type, int32_t T,
                                       int32_t H, int32_t Hkv, int32_t hd, int32_t n_ctx, int32_t n_seq, uint32_t *err,
                                       void *stream) {
    const char *who = "llm_op_qk_norm_rope";
    if (!qkv || !rope || !pos || !seq || !q || !k_cache || !v_cache) return refuse(who, "a pointer is NULL");
    if (const char *why = shape_error(T, H, Hkv, hd, n_ctx, n_seq)) return refuse(who, why);
    if (ld < (H + 2 * Hkv) * hd || ld % 4) return refuse(who, "ld must be a multiple of 4 and hold every head");
    if (q_type != LLM_Q_F32 && q_type != LLM_Q_F16) return refuse(who, "unknown q_type");
    if (kv_type < LLM_KV_F16 || kv_type > LLM_KV_Q4_0) return refuse(who, "unknown kv_type");
    if (!(eps >= 0.f)) return refuse(who, "eps must not be negative");
    if (!aligned(qkv, 16) || !aligned(q_gain, 16) || !aligned(k_gain, 16) || !aligned(rope, 16) || !aligned(q, 16) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return refuse(who, "qkv, gains, rope, q and the caches must be 16-byte aligned");
    QkNormArgs a;
    a.qkv = qkv; a.ld = ld; a.q_gain = q_gain; a.k_gain = k_gain; a.eps = eps;
    a.rope = (const float2 *)rope; a.pos = pos; a.seq = seq;
    a.q32 = q_type == LLM_Q_F32 ? (float *)q : nullptr;
    a.q16 = q_type == LLM_Q_F16 ? (f16 *)q : nullptr;
    a.kv = q4_view(k_cache, v_cache, Hkv, hd, n_ctx, n_seq);
    if (kv_type != LLM_KV_Q4_0) a.kv.k4 = a.kv.v4 = nullptr;
    if (kv_type == LLM_KV_F16) { a.kv.k = (f16 *)k_cache; a.kv.v = (f16 *)v_cache; }
    if (kv_type == LLM_KV_E4M3) { a.kv.k8 = (uint8_t *)k_cache; a.kv.v8 = (uint8_t *)v_cache; }
    a.T = T; a.H = H; a.err = err;
    return launched(who, launch_qk_norm_rope(a, overlapped(stream)));
}

extern "C" int32_t llm_op_kv_rows_q4_0(const void *cache, const int32_t *pos, const int32_t *seq, void *out, int32_t T,
                                       int32_t Hkv, int32_t hd, int32_t n_ctx, int32_t n_seq, uint32_t *err,
                                       void *stream) {
    const char *who = "llm_op_kv_rows_q4_0";
    if (!cache || !pos || !seq || !out) return refuse(who, "a pointer is NULL");
    if (const char *why = shape_error(T, Hkv, Hkv, hd, n_ctx, n_seq)) return refuse(who, why);
    if (!aligned(cache, 16) || !aligned(out, 16)) return refuse(who, "cache and out must be 16-byte aligned");
    const KvView kv = q4_view(cache, cache, Hkv, hd, n_ctx, n_seq);
    return launched(who, launch_kv_rows_q4(kv.k4, kv.kd, kv, pos, seq, (f16 *)out, T, err, overlapped(stream)));
}

extern "C" int64_t llm_op_attn_decode_q4_0_scratch_bytes(int32_t T, int32_t H, int32_t Hkv, int32_t hd, int32_t n_ctx,
                                                         int32_t n_seq) {
    if (shape_error(T, H, Hkv, hd, n_ctx, n_seq) || T > DECODE_MAX_T) return LLM_ERR_INVALID;
    return (int64_t)attn_q4_scratch_bytes(T, H, Hkv, hd, n_ctx);
}

extern "C" int32_t llm_op_attn_decode_q4_0(const float *q, const void *k_cache, const void *v_cache, const int32_t *pos,
                                           const int32_t *seq, void *o, int32_t T, int32_t H, int32_t Hkv, int32_t hd,
                                           int32_t n_ctx, int32_t n_seq, int32_t window, void *scratch,
                                           int64_t scratch_bytes, uint32_t *err, void *stream) {
    const char *who = "llm_op_attn_decode_q4_0";
    if (!q || !k_cache || !v_cache || !pos || !seq || !o) return refuse(who, "a pointer is NULL");
    if (const char *why = shape_error(T, H, Hkv, hd, n_ctx, n_seq)) return refuse(who, why);
    if (T > DECODE_MAX_T) return refuse(who, "T must be 1..4096");
    if (window < 0) return refuse(who, "window must not be negative");
    if (!scratch || scratch_bytes < llm_op_attn_decode_q4_0_scratch_bytes(T, H, Hkv, hd, n_ctx, n_seq))
        return refuse(who, "scratch is NULL or smaller than llm_op_attn_decode_q4_0_scratch_bytes");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(scratch, 16))
        return refuse(who, "q, the caches, o and scratch must be 16-byte aligned");
    if (cudaError_t e = init_kernel_attributes()) return launched(who, e);
    AttnDecodeArgs at;
    at.q = q;
    at.kv = q4_view(k_cache, v_cache, Hkv, hd, n_ctx, n_seq);
    at.pos = pos; at.seq = seq; at.o = (f16 *)o; at.T = T; at.H = H;
    at.err = err; at.window = window;
    return launched(who, launch_attn_decode_q4(at, scratch, overlapped(stream)));
}

// Not used any more (the kernels widen what they read themselves): two fp16
// planes [n_seq][Hkv][padded n_ctx][hd] and the row lists, as programs written
// for them size it.
extern "C" int64_t llm_op_attn_prefill_q4_0_scratch_bytes(int32_t T, int32_t H, int32_t Hkv, int32_t hd, int32_t n_ctx,
                                                          int32_t n_seq) {
    if (shape_error(T, H, Hkv, hd, n_ctx, n_seq)) return LLM_ERR_INVALID;
    const size_t plane = align256(cache_rows(n_seq, Hkv, padded_ctx(n_ctx)) * hd * sizeof(f16));
    return (int64_t)(256 + 2 * plane + align256((size_t)T * sizeof(AttnTile)));
}

extern "C" int32_t llm_op_attn_prefill_q4_0(const void *q, const void *k_cache, const void *v_cache, const int32_t *pos,
                                            const int32_t *seq, void *o, int32_t T, int32_t H, int32_t Hkv, int32_t hd,
                                            int32_t n_ctx, int32_t n_seq, int32_t window, void *scratch,
                                            int64_t scratch_bytes, uint32_t *err, void *stream) {
    const char *who = "llm_op_attn_prefill_q4_0";
    if (!q || !k_cache || !v_cache || !pos || !seq || !o) return refuse(who, "a pointer is NULL");
    if (const char *why = shape_error(T, H, Hkv, hd, n_ctx, n_seq)) return refuse(who, why);
    if (window < 0) return refuse(who, "window must not be negative");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16))
        return refuse(who, "q, the caches and o must be 16-byte aligned");
    (void)scratch;
    (void)scratch_bytes;
    const bool tc = attn_prefill_q4_tc_ok(hd);
    const int rows_max = attn_prefill_q4_rows(tc);
    std::vector<KvRuns::Run> runs;
    try {
        for (int i = 0; i < T;) {
            if (seq[i] < 0 || seq[i] >= n_seq) return refuse(who, "a sequence id is outside [0, n_seq)");
            int j = i;
            while (j < T && seq[j] == seq[i]) {
                if (pos[j] < 0 || pos[j] >= n_ctx) return refuse(who, "a position is outside [0, n_ctx)");
                if (j > i && pos[j] != pos[j - 1] + 1)
                    return refuse(who, "positions of a sequence's rows must be consecutive");
                ++j;
            }
            runs.push_back(KvRuns::Run{i, j - i, seq[i], pos[i], 0});
            i = j;
        }
        std::vector<int> ids;
        for (const KvRuns::Run &r : runs) ids.push_back(r.seq);
        std::sort(ids.begin(), ids.end());
        if (std::adjacent_find(ids.begin(), ids.end()) != ids.end())
            return refuse(who, "the rows of a sequence must be consecutive");
    } catch (const std::bad_alloc &) {
        set_global_error("llm_op_attn_prefill_q4_0: out of host memory");
        return LLM_ERR_ALLOC;
    }
    if (cudaError_t e = init_kernel_attributes()) return launched(who, e);
    TmaMap mq;
    if (tc && !make_operand_map(&mq, (const f16 *)q, T, H * hd, 128)) {
        set_global_error("llm_op_attn_prefill_q4_0: TMA descriptor creation failed");
        return LLM_ERR_COMPUTE;
    }
    AttnPrefillArgs at;
    at.q = (const f16 *)q;
    at.kv = q4_view(k_cache, v_cache, Hkv, hd, n_ctx, n_seq);
    at.tiles = nullptr; at.o = (f16 *)o; at.H = H; at.err = err; at.window = window;
    // the runs go with the launch, as many as one takes at a time
    for (size_t i = 0; i < runs.size();) {
        KvRuns part;
        int n = 0;
        at.n_tiles = 0;
        for (; n < KvRuns::MAX && i < runs.size(); ++n, ++i) {
            part.run[n] = runs[i];
            part.run[n].tile0 = at.n_tiles;
            at.n_tiles += (runs[i].n_rows + rows_max - 1) / rows_max;
        }
        if (cudaError_t e = launch_attn_prefill_q4(at, &part, n, tc ? &mq : nullptr, overlapped(stream))) return launched(who, e);
    }
    return LLM_OK;
}
