// Queries and keys normed per head, rotated by their position, and the keys
// and values appended to the cache, in one pass over the QKV projection's
// output ("Inside the inference engine: model architectures and forward
// pass", section "Detailed explanation: Llama's forward pass in Go": RoPE on Q
// and K, then the cache's Put; the per-head norm is RMSNorm over head_dim with
// a gain shared by the heads, as model families with normed queries and keys
// apply it between the projection and the rotation):
//   u = x * gain / sqrt(mean(x^2) + eps),  (u0, u1) -> (u0 cos - u1 sin, u0 sin + u1 cos)
// on adjacent pairs.  A model without such gains skips the norm; it comes here
// when its cache is Q4_0, whose blocks need 32 neighbouring elements at once,
// which no projection epilogue holds.
//
// head_dim / 4 lanes take one head of one row, four elements (two rotation
// pairs) a lane, so the norm's sum and a block's largest magnitude are a few
// shuffles and every access is a vector.  A warp takes HPW heads of a row in
// turn: their loads go out together and the row's position, cosines and gains
// are read once.  Bound by memory: 4 bytes read and about 2 written an element.
//
// Q4_0 codes are those of the exact values.  A float32 value carries a few
// ulp of error from the norm and the rotation, which matters only next to a
// border between two codes; a row with an element within NEAR of one (about
// one row in 200) is encoded again from float64 arithmetic.
#include "common.cuh"
#include "launch.cuh"
#include "q4.cuh"

namespace llm {

namespace {

constexpr int THREADS = 256;
// Distance from a code border, in codes, under which float32 does not settle
// the code: |v / d| <= 8 with a relative error below 24 * 2^-24 gives 1.2e-5.
constexpr float NEAR = 2e-5f;

__device__ __forceinline__ float inv_sqrt(float v) { return rsqrtf(v); }         // 2 ulp
__device__ __forceinline__ double inv_sqrt(double v) { return 1.0 / sqrt(v); }

template <int W, class R>
__device__ __forceinline__ R group_sum(R v) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The head's values after norm and rotation, in R.
template <int HD, class R>
__device__ __forceinline__ void transform(const float (&x)[4], const float (&gain)[4], const float4 cs, bool norm,
                                          bool turn, float eps, R (&u)[4]) {
    // the shuffles run for every lane: heads without a norm share the warp
    R ss = R(0);
#pragma unroll
    for (int e = 0; e < 4; ++e) ss += R(x[e]) * R(x[e]);
    ss = group_sum<HD / 4>(ss);
    const R r = inv_sqrt(ss / R(HD) + R(eps));
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = norm ? R(x[e]) * r * R(gain[e]) : R(x[e]);
    if (turn) {
        const R a0 = u[0] * R(cs.x) - u[1] * R(cs.y), b0 = u[0] * R(cs.y) + u[1] * R(cs.x);
        const R a1 = u[2] * R(cs.z) - u[3] * R(cs.w), b1 = u[2] * R(cs.w) + u[3] * R(cs.z);
        u[0] = a0; u[1] = b0; u[2] = a1; u[3] = b1;
    }
}

// The codes of a lane's four elements and the scale of its block (8 lanes).
// Returns whether a value lies so near a border that R does not settle it.
template <class R>
__device__ __forceinline__ bool encode(const R (&u)[4], int lane, R &d, int (&c)[4]) {
    R m = u[0];
#pragma unroll
    for (int e = 1; e < 4; ++e)
        if (fabs(u[e]) > fabs(m)) m = u[e];
    R top = fabs(m);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
        const R other = __shfl_xor_sync(0xffffffffu, top, o);
        top = other > top ? other : top;
    }
    // the first element of that magnitude gives the sign
    const unsigned has = __ballot_sync(0xffffffffu, fabs(m) == top) >> (lane & ~7) & 0xffu;
    m = __shfl_sync(0xffffffffu, m, (lane & ~7) + (has ? __ffs(has) - 1 : 0));
    d = m * R(-0.125);
    bool near = false;
    if constexpr (sizeof(R) == 4) {
        // the quotients by one reciprocal; scales that it does not reach are left to float64
        const float inv = d != 0.f ? __frcp_rn(d) : 0.f;
        near = d != 0.f && !(fabsf(d) > 1e-30f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float q = u[e] * inv, k = rintf(q);            // in [-8, 8]: the top itself is at -8
            c[e] = min(max((int)k + 8, 0), 15);
            near |= fabsf(fabsf(q - k) - 0.5f) < NEAR || q > 8.f - NEAR;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = q4::code_of(u[e], d);
    }
    return near;
}

// grid (row, block of heads)
template <int HD, int HPW>
__global__ void __launch_bounds__(THREADS) qk_norm_rope_kernel(const QkNormArgs a) {
    constexpr int L = HD / 4, PER = 32 / L;           // lanes of a head, heads of a warp at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % L, e0 = 4 * sub;
    const int Hkv = a.kv.n_kv_head, heads = a.H + 2 * Hkv;
    const int t = blockIdx.x, first = ((int)blockIdx.y * (THREADS / 32) + warp) * HPW * PER + lane / L;
    pdl_wait();
    pdl_trigger();
    if (first - lane / L >= heads) return;            // whole warps
    const int pos = a.pos[t], seq = a.seq[t];
    const bool ok = pos >= 0 && pos < a.kv.n_ctx && seq >= 0 && seq < a.kv.n_seq;
    // every lane stays for the shuffles; heads past the last repeat it and store nothing
    const float *row = a.qkv + (size_t)t * a.ld + e0;
    float4 xv[HPW];
#pragma unroll
    for (int i = 0; i < HPW; ++i) xv[i] = *reinterpret_cast<const float4 *>(row + (size_t)min(first + i * PER, heads - 1) * HD);
    float4 turn = make_float4(1.f, 0.f, 1.f, 0.f);
    if (ok) turn = *reinterpret_cast<const float4 *>(a.rope + (size_t)pos * (HD / 2) + 2 * sub);
    const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 gq = a.q_gain ? *reinterpret_cast<const float4 *>(a.q_gain + e0) : one;
    const float4 gk = a.k_gain ? *reinterpret_cast<const float4 *>(a.k_gain + e0) : one;
    if (!ok && first == 0 && sub == 0) raise_error(a.err, ERRF_BAD_INDEX);
    bool out_of_range = false;
#pragma unroll
    for (int i = 0; i < HPW; ++i) {
        const int h = first + i * PER;
        const bool in = h < heads, is_q = h < a.H, is_k = !is_q && h < a.H + Hkv;
        const bool norm = is_q ? a.q_gain != nullptr : is_k && a.k_gain != nullptr;
        const float4 gv = is_q ? gq : gk, cs = is_q || is_k ? turn : make_float4(1.f, 0.f, 1.f, 0.f);
        const float x[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
        const float gain[4] = {gv.x, gv.y, gv.z, gv.w};
        float u[4];
        transform<HD, float>(x, gain, cs, norm, is_q || is_k, a.eps, u);
        const bool bad = f16_bad(u[0]) | f16_bad(u[1]) | f16_bad(u[2]) | f16_bad(u[3]);
        if (is_q && in) {
            const size_t off = (size_t)t * a.H * HD + (size_t)h * HD + e0;
            if (!ok) u[0] = u[1] = u[2] = u[3] = 0.f;  // a row outside the cache has zero queries
            if (a.q32) {
                *reinterpret_cast<float4 *>(a.q32 + off) = make_float4(u[0], u[1], u[2], u[3]);
            } else {
                out_of_range |= bad && ok;
                *reinterpret_cast<uint2 *>(a.q16 + off) = make_uint2(pack_h2(u[0], u[1]), pack_h2(u[2], u[3]));
            }
        }
        const int j = h - a.H - (is_k ? 0 : Hkv);
        const bool put = in && ok && !is_q;
        const size_t base = put ? (size_t)seq * a.kv.seq_stride + ((size_t)j * a.kv.n_ctx + pos) * HD : 0;
        if (a.kv.k4) {
            if (!__any_sync(0xffffffffu, put)) continue;         // a warp of query heads
            float d;
            int c[4];
            const bool near = encode<float>(u, lane, d, c);
            if (__any_sync(0xffffffffu, near && put)) {
                double u64[4], d64;
                transform<HD, double>(x, gain, cs, norm, is_q || is_k, a.eps, u64);
                encode<double>(u64, lane, d64, c);
                d = (float)d64;
            }
            // elements 4 sub .. of the head: half of a word (8 elements)
            uint32_t w = (uint32_t)c[0] | (uint32_t)c[1] << 16 | (uint32_t)c[2] << 4 | (uint32_t)c[3] << 20;
            w |= __shfl_xor_sync(0xffffffffu, w << 8, 1);
            if (put) {
                out_of_range |= bad;
                const int blk = sub >> 3, tt = (sub & 7) >> 1;
                if (!(sub & 1))
                    reinterpret_cast<uint32_t *>((is_k ? a.kv.k4 : a.kv.v4) + base / 2)[tt * (HD / 32) + blk] = w;
                if ((sub & 7) == 0) (is_k ? a.kv.kd : a.kv.vd)[base / 32 + blk] = f2h(d);
            }
        } else if (put) {
            if (a.kv.k8) {
                *reinterpret_cast<uint32_t *>((is_k ? a.kv.k8 : a.kv.v8) + base + e0) =
                    (uint32_t)pack_e4m3x2(u[0], u[1]) | (uint32_t)pack_e4m3x2(u[2], u[3]) << 16;
            } else {
                out_of_range |= bad;
                *reinterpret_cast<uint2 *>((is_k ? a.kv.k : a.kv.v) + base + e0) =
                    make_uint2(pack_h2(u[0], u[1]), pack_h2(u[2], u[3]));
            }
        }
    }
    if (out_of_range) raise_error(a.err, ERRF_F16_RANGE);
}

// Context shift of a sequence's Q4_0 cache (kv_shift_kernel's of the other
// caches, with its order of reads and writes): rows [p0 + n, end) move down by
// n, a key's values rotated by -n and encoded again, a value row copied.  One
// CTA per (layer, kv head) walks the rows upward, all its lanes' rows read
// before any is written.
constexpr int SHIFT_THREADS = 512;

template <int HD>
__global__ void __launch_bounds__(SHIFT_THREADS) kv_shift_q4_kernel(KvView kv, int p0, int n, int end, const float2 *rope) {
    constexpr int L = HD / 4, ROWS = SHIFT_THREADS / L, NB = HD / 32;
    const size_t base = (size_t)blockIdx.x * kv.n_ctx * HD;      // (layer, head) block of this sequence, in elements
    const int lane = threadIdx.x & 31, sub = threadIdx.x % L, r = threadIdx.x / L;
    const int blk = sub >> 3, word = ((sub & 7) >> 1) * NB + blk, half = 8 * (sub & 1);
    uint32_t *kw = reinterpret_cast<uint32_t *>(kv.k4 + base / 2), *vw = reinterpret_cast<uint32_t *>(kv.v4 + base / 2);
    f16 *kd = kv.kd + base / 32, *vd = kv.vd + base / 32;
    const float4 c = *reinterpret_cast<const float4 *>(rope + (size_t)n * (HD / 2) + 2 * sub);
    const float4 back = make_float4(c.x, -c.y, c.z, -c.w);
    const float gain[4] = {1.f, 1.f, 1.f, 1.f};
    for (int r0 = p0 + n; r0 < end; r0 += ROWS) {
        const bool in = r0 + r < end;
        const size_t src = in ? r0 + r : r0, dst = src - n;
        const uint32_t w = kw[src * (HD / 8) + word] >> half, wv = vw[src * (HD / 8) + word];
        const float d = hf(kd[src * NB + blk]);
        const f16 dv = vd[src * NB + blk];
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (float)((int)((w >> q4::shift_of(e)) & 15u) - 8) * d;     // exact
        float u[4], nd;
        int code[4];
        transform<HD, float>(x, gain, back, false, true, 0.f, u);
        const bool near = encode<float>(u, lane, nd, code);
        if (__any_sync(0xffffffffu, near)) {
            double u64[4], d64;
            transform<HD, double>(x, gain, back, false, true, 0.f, u64);
            encode<double>(u64, lane, d64, code);
            nd = (float)d64;
        }
        uint32_t out = (uint32_t)code[0] | (uint32_t)code[1] << 16 | (uint32_t)code[2] << 4 | (uint32_t)code[3] << 20;
        out |= __shfl_xor_sync(0xffffffffu, out << 8, 1);
        __syncthreads();
        if (in) {
            if (half == 0) {
                kw[dst * (HD / 8) + word] = out;
                vw[dst * (HD / 8) + word] = wv;
            }
            if ((sub & 7) == 0) {
                kd[dst * NB + blk] = f2h(nd);
                vd[dst * NB + blk] = dv;
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_kv_shift_q4(const KvView &kv0, int n_layer, int seq, int p0, int n, int end, const float2 *rope,
                               const Launch &l) {
    const int hd = kv0.head_dim;
    if (n < 1 || p0 < 0 || p0 + n > end || end > kv0.n_ctx || seq < 0 || seq >= kv0.n_seq || !kv0.k4)
        return cudaErrorInvalidValue;
    if (p0 + n == end) return cudaSuccess;                  // nothing after the dropped rows
    KvView kv = kv0;
    const size_t so = (size_t)seq * kv0.seq_stride;
    kv.k4 += so / 2; kv.v4 += so / 2; kv.kd += so / 32; kv.vd += so / 32;
    const dim3 grid(n_layer * kv0.n_kv_head), block(SHIFT_THREADS);
    if (hd == 32) return launch_kernel(kv_shift_q4_kernel<32>, grid, block, 0, l, kv, p0, n, end, rope);
    if (hd == 64) return launch_kernel(kv_shift_q4_kernel<64>, grid, block, 0, l, kv, p0, n, end, rope);
    if (hd == 128) return launch_kernel(kv_shift_q4_kernel<128>, grid, block, 0, l, kv, p0, n, end, rope);
    return cudaErrorInvalidValue;
}

cudaError_t launch_qk_norm_rope(const QkNormArgs &a, const Launch &l) {
    const int hd = a.kv.head_dim, heads = a.H + 2 * a.kv.n_kv_head;
    if (a.T < 1 || (!a.q32 && !a.q16) || (hd != 32 && hd != 64 && hd != 128)) return cudaErrorInvalidValue;
    // few rows: one head a warp step, so that they spread over the SMs; many:
    // MANY heads a warp share the row's loads
    constexpr int MANY = 4;
    const int per = 128 / hd * (THREADS / 32);        // heads a CTA takes at once
    const bool many = (long long)a.T * ((heads + per - 1) / per) > 2048;
    const dim3 grid(a.T, (heads + per * (many ? MANY : 1) - 1) / (per * (many ? MANY : 1))), block(THREADS);
#define QK_CASE(HDV)                                                                                  \
    if (hd == HDV)                                                                                    \
        return many ? launch_kernel(qk_norm_rope_kernel<HDV, MANY>, grid, block, 0, l, a)             \
                    : launch_kernel(qk_norm_rope_kernel<HDV, 1>, grid, block, 0, l, a);
    QK_CASE(32) QK_CASE(64) QK_CASE(128)
#undef QK_CASE
    return cudaErrorInvalidValue;
}

}  // namespace llm
