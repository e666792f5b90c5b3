// Attention over a Q4_0 cache ("LLama.cpp — how it works", "KV-cache": a
// quantised cache where memory is short; the attention itself as in
// attn_decode.cu): for each row t and query head h, o = softmax(q K^T /
// sqrt(hd)) V over the visible positions of sequence seq[t], K and V standing
// for d * (c - 8) (q4.cuh).
//
// Decode: one CTA per (split, kv head and chunk of 8 of its query heads, row)
// walks its span of keys, a warp 32 keys at a time with its own online
// softmax; the splits' (max, sum, numerators) are merged in split order by the
// CTA that arrives last.
//
// Prefill: the visible rows of the ubatch's sequences are widened once to fp16
// and the fp16 prefill attention runs on them.
#include "common.cuh"
#include "launch.cuh"
#include "q4.cuh"

namespace llm {

namespace {

constexpr int THREADS = 128, NW = THREADS / 32;
constexpr int GC = 8;                    // query heads of a chunk
constexpr int MAX_SPLIT = ATTN_DECODE_MAX_SPLIT;
constexpr int MIN_KEYS = 64;             // keys of a split
constexpr int SMS = 152;                 // of the one GPU this library is compiled for: scratch sizes follow from it

__device__ __forceinline__ int split_chunk(int S, int n_split) {
    int chunk = (S + n_split - 1) / n_split;
    chunk = (chunk + MIN_KEYS - 1) / MIN_KEYS * MIN_KEYS;
    return chunk < MIN_KEYS ? MIN_KEYS : chunk;
}

template <int HD>
__global__ void __launch_bounds__(THREADS) attn_decode_q4_kernel(const AttnDecodeArgs a, int chunks) {
    constexpr int REC = HD + 2, DPL = HD / 32;
    __shared__ float qs[GC][HD];
    __shared__ float wst[NW][GC][REC];
    __shared__ int s_last;
    const int sp = blockIdx.x, j = blockIdx.y / chunks, ck = blockIdx.y - j * chunks, t = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hkv = a.kv.n_kv_head, G = a.H / Hkv, h0 = j * G + ck * GC, gn = min(GC, G - ck * GC);
    pdl_wait();
    pdl_trigger();
    const int pos = a.pos[t], seq = a.seq[t];
    const bool ok = pos >= 0 && pos < a.kv.n_ctx && seq >= 0 && seq < a.kv.n_seq;
    if (!ok && tid == 0 && sp == 0 && blockIdx.y == 0) raise_error(a.err, ERRF_BAD_INDEX);
    const int lo = (ok && a.window > 0 && pos + 1 > a.window) ? pos + 1 - a.window : 0;
    const int S = ok ? pos + 1 - lo : 0;
    const int chunk = split_chunk(S, a.n_split);
    const int n_eff = S > 0 ? (S + chunk - 1) / chunk : 1;
    if (sp >= n_eff) return;
    const int kb = lo + sp * chunk, ke = min(lo + S, kb + chunk);
    const size_t base = ok ? (size_t)seq * a.kv.seq_stride + (size_t)j * a.kv.n_ctx * HD : 0;
    const float scale = 1.4426950408889634f / sqrtf((float)HD);
    for (int i = tid; i < GC * HD; i += THREADS) {
        const int g = i / HD, d = i - g * HD;
        qs[g][d] = g < gn ? a.q[((size_t)t * a.H + h0 + g) * HD + d] * scale : 0.f;
    }
    __syncthreads();

    float o[GC][DPL], m[GC], l[GC];
#pragma unroll
    for (int g = 0; g < GC; ++g) {
        m[g] = -INFINITY; l[g] = 0.f;
#pragma unroll
        for (int e = 0; e < DPL; ++e) o[g][e] = 0.f;
    }
    for (int k0 = kb + warp * 32; k0 < ke; k0 += THREADS) {
        const int key = k0 + lane;
        float s[GC];
#pragma unroll
        for (int g = 0; g < GC; ++g) s[g] = -INFINITY;
        if (key < ke) {
            const size_t row = base + (size_t)key * HD;
            const uint32_t *w = reinterpret_cast<const uint32_t *>(a.kv.k4 + row / 2);
            const f16 *sc = a.kv.kd + row / 32;
#pragma unroll
            for (int g = 0; g < GC; ++g) s[g] = 0.f;
            for (int i = 0; i < HD / 8; ++i) {
                const uint32_t word = w[i];
                const int b = i % (HD / 32), tt = i / (HD / 32);
                const float d = hf(sc[b]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = (float)((int)((word >> q4::shift_of(e)) & 15u) - 8) * d;
#pragma unroll
                    for (int g = 0; g < GC; ++g) s[g] += qs[g][32 * b + 8 * tt + e] * v;
                }
            }
        }
#pragma unroll
        for (int g = 0; g < GC; ++g) {
            const float mn = fmaxf(m[g], warp_max(s[g]));
            const float f = m[g] == -INFINITY ? 0.f : exp2f(m[g] - mn);
            s[g] = exp2f(s[g] - mn);
            l[g] = l[g] * f + warp_sum(s[g]);
            m[g] = mn;
#pragma unroll
            for (int e = 0; e < DPL; ++e) o[g][e] *= f;
        }
        for (int k = 0; k < 32 && k0 + k < ke; ++k) {
            const size_t row = base + (size_t)(k0 + k) * HD;
            float v[DPL];
#pragma unroll
            for (int e = 0; e < DPL; ++e) {
                const int d = lane * DPL + e, b = d >> 5, r = d & 31;
                const uint32_t word = reinterpret_cast<const uint32_t *>(a.kv.v4 + row / 2)[(r >> 3) * (HD / 32) + b];
                v[e] = (float)((int)((word >> (4 * ((r & 7) >> 1) + 16 * (r & 1))) & 15u) - 8) * hf(a.kv.vd[row / 32 + b]);
            }
#pragma unroll
            for (int g = 0; g < GC; ++g) {
                const float p = __shfl_sync(0xffffffffu, s[g], k);
#pragma unroll
                for (int e = 0; e < DPL; ++e) o[g][e] += p * v[e];
            }
        }
    }
#pragma unroll
    for (int g = 0; g < GC; ++g) {
        if (lane == 0) { wst[warp][g][0] = m[g]; wst[warp][g][1] = l[g]; }
#pragma unroll
        for (int e = 0; e < DPL; ++e) wst[warp][g][2 + lane * DPL + e] = o[g][e];
    }
    __syncthreads();
    float *part = a.part + ((size_t)(t * a.H + h0) * a.n_split + sp) * REC;
    for (int i = tid; i < gn * HD; i += THREADS) {
        const int g = i / HD, d = i - g * HD;
        float M = -INFINITY, num = 0.f, den = 0.f;
        for (int w = 0; w < NW; ++w) M = fmaxf(M, wst[w][g][0]);
        if (M != -INFINITY)
            for (int w = 0; w < NW; ++w) {
                const float f = exp2f(wst[w][g][0] - M);
                num += f * wst[w][g][2 + d];
                den += f * wst[w][g][1];
            }
        float *rp = part + (size_t)g * a.n_split * REC;
        rp[2 + d] = num;
        if (d == 0) { rp[0] = M; rp[1] = den; }
    }
    __threadfence();
    __syncthreads();
    unsigned *cnt = a.counters + (size_t)t * gridDim.y + blockIdx.y;
    if (tid == 0) s_last = atomicAdd(cnt, 1u) == (unsigned)(n_eff - 1);
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int i = tid; i < gn * HD; i += THREADS) {
        const int g = i / HD, d = i - g * HD;
        const float *rp = a.part + ((size_t)(t * a.H + h0 + g) * a.n_split) * REC;
        float M = -INFINITY, num = 0.f, den = 0.f;
        for (int p = 0; p < n_eff; ++p) {
            const float pm = __ldcg(rp + (size_t)p * REC);
            if (pm == -INFINITY) continue;
            const float mn = fmaxf(M, pm), fo = M == -INFINITY ? 0.f : exp2f(M - mn), fn = exp2f(pm - mn);
            num = num * fo + __ldcg(rp + (size_t)p * REC + 2 + d) * fn;
            den = den * fo + __ldcg(rp + (size_t)p * REC + 1) * fn;
            M = mn;
        }
        a.o[((size_t)t * a.H + h0 + g) * HD + d] = f2h(den > 0.f ? num / den : 0.f);
    }
    if (tid == 0) *cnt = 0u;
}

// One thread a word: eight neighbouring elements out of a row's word w.
__device__ __forceinline__ uint4 widen_word(uint32_t word, float d) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = pack_h2((float)((int)((word >> (4 * i)) & 15u) - 8) * d, (float)((int)((word >> (16 + 4 * i)) & 15u) - 8) * d);
    return make_uint4(r[0], r[1], r[2], r[3]);
}

constexpr int WT = 256;

// blockIdx (row block, kv head, span); a thread widens one word of K and of V.
__global__ void __launch_bounds__(WT) kv_widen_q4_kernel(const KvView kv, const KvSpan *spans, f16 *k16, f16 *v16,
                                                         int n_pad) {
    pdl_wait();
    pdl_trigger();
    const KvSpan sp = spans[blockIdx.z];
    const int hd = kv.head_dim, wpr = hd / 8, nb = hd / 32;      // words of a row, blocks of a row
    const int r0 = sp.lo / 128 * 128, r1 = (sp.hi + 127) / 128 * 128;
    const int row = r0 + (int)(blockIdx.x * (WT / wpr) + threadIdx.x / wpr), w = threadIdx.x % wpr;
    if (row >= r1) return;
    const size_t dst = (((size_t)sp.seq * kv.n_kv_head + blockIdx.y) * n_pad + row) * hd + 32 * (w % nb) + 8 * (w / nb);
    uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
    if (row >= sp.lo && row < sp.hi) {
        const size_t e = (size_t)sp.seq * kv.seq_stride + ((size_t)blockIdx.y * kv.n_ctx + row) * hd;
        k = widen_word(reinterpret_cast<const uint32_t *>(kv.k4 + e / 2)[w], hf(kv.kd[e / 32 + w % nb]));
        v = widen_word(reinterpret_cast<const uint32_t *>(kv.v4 + e / 2)[w], hf(kv.vd[e / 32 + w % nb]));
    }
    *reinterpret_cast<uint4 *>(k16 + dst) = k;
    *reinterpret_cast<uint4 *>(v16 + dst) = v;
}

__global__ void __launch_bounds__(WT) kv_rows_q4_kernel(const uint8_t *codes, const f16 *scales, const KvView kv,
                                                        const int *pos, const int *seq, f16 *out, int T, uint32_t *err) {
    const int hd = kv.head_dim, wpr = hd / 8, nb = hd / 32;
    const long long i = (long long)blockIdx.x * WT + threadIdx.x;
    const long long row = i / wpr;
    const int w = (int)(i - row * wpr);
    if (row >= (long long)T * kv.n_kv_head) return;
    const int t = (int)(row / kv.n_kv_head), j = (int)(row - (long long)t * kv.n_kv_head);
    const int p = pos[t], s = seq[t];
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (p >= 0 && p < kv.n_ctx && s >= 0 && s < kv.n_seq) {
        const size_t e = (size_t)s * kv.seq_stride + ((size_t)j * kv.n_ctx + p) * hd;
        v = widen_word(reinterpret_cast<const uint32_t *>(codes + e / 2)[w], hf(scales[e / 32 + w % nb]));
    } else if (j == 0 && w == 0) {
        raise_error(err, ERRF_BAD_INDEX);
    }
    *reinterpret_cast<uint4 *>(out + (size_t)row * hd + 32 * (w % nb) + 8 * (w / nb)) = v;
}

}  // namespace

int attn_q4_chunks(int H, int Hkv) { return (H / Hkv + GC - 1) / GC; }

int attn_q4_pick_split(int T, int H, int Hkv, int n_ctx) {
    const int mx = (n_ctx + MIN_KEYS - 1) / MIN_KEYS;
    long long s = 4LL * SMS / ((long long)T * Hkv * attn_q4_chunks(H, Hkv));
    if (s > MAX_SPLIT) s = MAX_SPLIT;
    if (s > mx) s = mx;
    return s < 1 ? 1 : (int)s;
}

size_t attn_q4_part_floats(int T, int H, int hd, int n_split) { return (size_t)T * H * n_split * (hd + 2); }

cudaError_t launch_attn_decode_q4(const AttnDecodeArgs &a, const Launch &l) {
    const int Hkv = a.kv.n_kv_head;
    if (a.T < 1 || a.T > 65535 || a.n_split < 1 || a.n_split > MAX_SPLIT || Hkv < 1 || a.H % Hkv || !a.kv.k4)
        return cudaErrorInvalidValue;
    const int chunks = attn_q4_chunks(a.H, Hkv);
    if ((long long)Hkv * chunks > 65535) return cudaErrorInvalidValue;
    const dim3 grid(a.n_split, Hkv * chunks, a.T), block(THREADS);
    if (a.kv.head_dim == 32) return launch_kernel(attn_decode_q4_kernel<32>, grid, block, 0, l, a, chunks);
    if (a.kv.head_dim == 64) return launch_kernel(attn_decode_q4_kernel<64>, grid, block, 0, l, a, chunks);
    if (a.kv.head_dim == 128) return launch_kernel(attn_decode_q4_kernel<128>, grid, block, 0, l, a, chunks);
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_widen_q4(const KvView &kv, const KvSpan *spans, int n_spans, int max_rows, f16 *k16, f16 *v16,
                               int n_pad, const Launch &l) {
    if (n_spans < 1) return cudaSuccess;
    if (n_spans > 65535 || kv.n_kv_head > 65535 || n_pad % 128 || n_pad < kv.n_ctx || !kv.k4) return cudaErrorInvalidValue;
    // a span touches at most max_rows / 128 + 2 tiles of 128 rows
    const int rows = (max_rows / 128 + 2) * 128, per = WT / (kv.head_dim / 8);
    return launch_kernel(kv_widen_q4_kernel, dim3((rows + per - 1) / per, kv.n_kv_head, n_spans), dim3(WT), 0, l, kv,
                         spans, k16, v16, n_pad);
}

cudaError_t launch_kv_rows_q4(const uint8_t *codes, const f16 *scales, const KvView &kv, const int *pos,
                              const int *seq, f16 *out, int T, uint32_t *err, const Launch &l) {
    const long long n = (long long)T * kv.n_kv_head * (kv.head_dim / 8);
    if (T < 1 || (n + WT - 1) / WT >= (1ll << 31)) return cudaErrorInvalidValue;
    return launch_kernel(kv_rows_q4_kernel, dim3((unsigned)((n + WT - 1) / WT)), dim3(WT), 0, l, codes, scales, kv, pos,
                         seq, out, T, err);
}

}  // namespace llm
