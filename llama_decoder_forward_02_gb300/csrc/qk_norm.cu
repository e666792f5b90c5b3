// Queries and keys normed per head, rotated by their position, and the keys
// and values appended to the cache, in one pass over the QKV projection's
// output ("Inside the inference engine: model architectures and forward
// pass", section "Detailed explanation: Llama's forward pass in Go": RoPE on Q
// and K, then the cache's Put; the per-head norm is RMSNorm over head_dim with
// a gain shared by the heads, as model families with normed queries and keys
// apply it between the projection and the rotation):
//   u = x * gain / sqrt(mean(x^2) + eps),  (u0, u1) -> (u0 cos - u1 sin, u0 sin + u1 cos)
// on adjacent pairs.  A model without such gains skips the norm; it comes here
// when its cache is Q4_0, whose blocks need 32 neighbouring elements at once: of
// the projections' epilogues only that of the GEMV over Q4_0 rows holds them.
//
// head_dim / 8 lanes take one head of one row, eight elements (four rotation
// pairs, one word of codes) a lane, so the norm's sum and a block's largest
// magnitude are a few shuffles for several heads at once and every access is a
// vector; a CTA takes a row, whose position, cosines and gains each lane reads
// once.  Bound by memory: 4 bytes read and about 2 written an element.  4096
// rows of 32 + 8 + 8 heads of 128 into an fp16 cache take 29.6 us, 76% of the
// copy bandwidth for their 153 MB (five CTAs of 48 registers an SM; four took
// 32.8).  With four elements a lane the shuffles, addresses and branches of
// twice as many lanes took 42.7 us, bound by issue.
//
// Into a Q4_0 cache 512 rows take 7.2 us (4.8 into an fp16 one), 8 rows 3.7.
//
// Q4_0 codes are those of the exact values.  A float32 value carries a few
// ulp of error from the norm and the rotation, which matters only next to a
// border between two codes; a row with an element next to one (about one row in
// 200) is encoded again from pairs of floats (2^-42).
#include "common.cuh"
#include "launch.cuh"
#include "q4.cuh"

namespace llm {

namespace {

constexpr int THREADS = 256;

template <int W>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

constexpr int E = 8;                      // elements of a lane

// The head's values after norm and rotation.
template <int HD>
__device__ __forceinline__ void transform(const float (&x)[E], const float (&gain)[E], const float2 (&cs)[E / 2], bool norm,
                                          bool turn, float eps, float (&u)[E]) {
    // the shuffles run for every lane: heads without a norm share the warp
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) ss += x[e] * x[e];
    ss = group_sum<HD / E>(ss);
    const float r = rsqrtf(ss / (float)HD + eps);                    // 2 ulp
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float a = norm ? x[e] * r * gain[e] : x[e], b = norm ? x[e + 1] * r * gain[e + 1] : x[e + 1];
        const float2 c = cs[e / 2];
        u[e] = turn ? a * c.x - b * c.y : a;
        u[e + 1] = turn ? a * c.y + b * c.x : b;
    }
}

// ... times up (a power of two) as pairs, good to 2^-42.
template <int HD>
__device__ __forceinline__ void transform(const float (&x)[E], const float (&gain)[E], const float2 (&cs)[E / 2], bool norm,
                                          bool turn, float eps, float up, q4::Pair (&u)[E]) {
    q4::Pair r{0.f, 0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) r = r + q4::two_prod(x[e], x[e]);
#pragma unroll
    for (int o = HD / E / 2; o > 0; o >>= 1) r = r + q4::shfl_xor(r, o);
    // 1 / sqrt(v) by one Newton step from float32's
    const q4::Pair v = q4::Pair{r.h / (float)HD, r.l / (float)HD} + q4::Pair{eps, 0.f};
    const float r0 = rsqrtf(v.h);
    const q4::Pair one = v * r0 * r0;
    r = q4::settle(r0, 0.5f * r0 * __fsub_rn(__fsub_rn(1.f, one.h), one.l));
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        q4::Pair a{x[e] * up, 0.f}, b{x[e + 1] * up, 0.f};
        if (norm) {
            a = q4::two_prod(x[e], gain[e] * up) * r;
            b = q4::two_prod(x[e + 1], gain[e + 1] * up) * r;
        }
        const float2 c = cs[e / 2];
        u[e] = turn ? a * c.x + b * -c.y : a;
        u[e + 1] = turn ? a * c.y + b * c.x : b;
    }
}

// The codes of a lane's elements and the scale of its block (4 lanes).
// Returns whether a value lies so near a border that float32 does not settle it.
__device__ __forceinline__ bool encode(const float (&u)[E], int lane, float &d, uint32_t &word) {
    float m = u[0];
#pragma unroll
    for (int e = 1; e < E; ++e)
        if (fabsf(u[e]) > fabsf(m)) m = u[e];
    float top = fabsf(m);
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, top, o);
        top = other > top ? other : top;
    }
    // the first element of that magnitude gives the sign
    const unsigned has = __ballot_sync(0xffffffffu, fabsf(m) == top) >> (lane & ~3) & 0xfu;
    d = __shfl_sync(0xffffffffu, m, (lane & ~3) + (has ? __ffs(has) - 1 : 0)) * -0.125f;
    // the quotients by one reciprocal; scales that it does not reach are left to the exact form
    const float inv = d != 0.f ? __frcp_rn(d) : 0.f;
    bool near = d != 0.f && !(fabsf(d) > q4::TINY);
    word = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float q = u[e] * inv, k = rintf(q);                // in [-8, 8]: the top itself is at -8
        word |= (uint32_t)min(max((int)k + 8, 0), 15) << q4::shift_of(e);
        near |= q4::near_border(q, k);
    }
    return near;
}
__device__ __forceinline__ void encode(const q4::Pair (&u)[E], int lane, float &d, uint32_t &word) {
    q4::Pair m = u[0];
#pragma unroll
    for (int e = 1; e < E; ++e)
        if (q4::larger(q4::magnitude(u[e]), q4::magnitude(m))) m = u[e];
    const q4::Pair mine = q4::magnitude(m);
    q4::Pair top = mine;
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) {
        const q4::Pair other = q4::shfl_xor(top, o);
        if (q4::larger(other, top)) top = other;
    }
    const unsigned has = __ballot_sync(0xffffffffu, mine.h == top.h && mine.l == top.l) >> (lane & ~3) & 0xfu;
    m = q4::shfl(m, (lane & ~3) + (has ? __ffs(has) - 1 : 0));
    const q4::Pair d2{m.h * -0.125f, m.l * -0.125f};
    word = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) word |= (uint32_t)q4::code_of(u[e], d2) << q4::shift_of(e);
    d = d2.h;
}

// The word and scale of the exact values.
template <int HD>
__device__ __forceinline__ void encode_exact(const float (&x)[E], const float (&gain)[E], const float2 (&cs)[E / 2], bool norm,
                                             bool turn, float eps, const float (&u)[E], bool used, int lane, float &d, uint32_t &word) {
    const bool near = encode(u, lane, d, word);
    if (__any_sync(0xffffffffu, near && used)) {
        const float up = fabsf(d) > q4::TINY || d == 0.f ? 1.f : q4::RAISE;     // the same for the lanes of a block
        q4::Pair u2[E];
        transform<HD>(x, gain, cs, norm, turn, eps, up, u2);
        encode(u2, lane, d, word);
        d /= up;
    }
}

__device__ __forceinline__ void load8(float (&v)[E], const float *p) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// grid (row, part): part p of gridDim.y takes the warps' heads p, p + parts, ..
// Q4: the cache is Q4_0 (its exact path would take registers from the others).
// Four or five CTAs an SM keep the loads in flight.
template <int HD, bool Q4>
__global__ void __launch_bounds__(THREADS, Q4 ? 4 : 5) qk_norm_rope_kernel(const QkNormArgs a) {
    constexpr int L = HD / E, PER = 32 / L;           // lanes of a head, heads of a warp at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % L, e0 = E * sub;
    const int Hkv = a.kv.n_kv_head, heads = a.H + 2 * Hkv;
    const int t = blockIdx.x;
    int h0 = ((int)blockIdx.y * (THREADS / 32) + warp) * PER;        // the warp's first head
    const int step = (int)gridDim.y * (THREADS / 32) * PER;
    const float *row = a.qkv + (size_t)t * a.ld + e0;
    // every lane stays for the shuffles; heads past the last repeat it and store nothing
    const float *first = row + (size_t)min(h0 + lane / L, heads - 1) * HD;
    float next[E];
    if (!a.early) {
        pdl_wait();
        pdl_trigger();
        if (h0 >= heads) return;                      // whole warps
        load8(next, first);
    }
    const int pos = a.pos[t], seq = a.seq[t];
    const bool ok = pos >= 0 && pos < a.kv.n_ctx && seq >= 0 && seq < a.kv.n_seq;
    float2 turn[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; e += 2) {
        float4 v = make_float4(1.f, 0.f, 1.f, 0.f);
        if (ok) v = *reinterpret_cast<const float4 *>(a.rope + (size_t)pos * (HD / 2) + e0 / 2 + e);
        turn[e] = make_float2(v.x, v.y);
        turn[e + 1] = make_float2(v.z, v.w);
    }
    if (a.early) {
        pdl_wait();
        pdl_trigger();
        if (h0 >= heads) return;
        load8(next, first);
    }
    if (!ok && h0 == 0 && lane == 0) raise_error(a.err, ERRF_BAD_INDEX);
    bool out_of_range = false;
    for (; h0 < heads; h0 += step) {
        const int h = h0 + lane / L;
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = next[e];
        if (h0 + step < heads) load8(next, row + (size_t)min(h + step, heads - 1) * HD);
        const bool in = h < heads, is_q = h < a.H, is_k = !is_q && h < a.H + Hkv;
        const float *gp = is_q ? a.q_gain : is_k ? a.k_gain : nullptr;
        float gain[E];
        if (gp) load8(gain, gp + e0);                 // a few cache lines, the same for every row
        else {
#pragma unroll
            for (int e = 0; e < E; ++e) gain[e] = 1.f;
        }
        float u[E];
        transform<HD>(x, gain, turn, gp != nullptr, is_q || is_k, a.eps, u);
        bool bad = false;
#pragma unroll
        for (int e = 0; e < E; ++e) bad |= f16_bad(u[e]);
        const uint4 packed = make_uint4(pack_h2(u[0], u[1]), pack_h2(u[2], u[3]), pack_h2(u[4], u[5]), pack_h2(u[6], u[7]));
        if (is_q && in) {
            const size_t off = (size_t)t * a.H * HD + (size_t)h * HD + e0;
            if (a.q32) {                              // a row outside the cache has zero queries
                float4 *q = reinterpret_cast<float4 *>(a.q32 + off);
                q[0] = ok ? make_float4(u[0], u[1], u[2], u[3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                q[1] = ok ? make_float4(u[4], u[5], u[6], u[7]) : make_float4(0.f, 0.f, 0.f, 0.f);
            } else {
                out_of_range |= bad && ok;
                *reinterpret_cast<uint4 *>(a.q16 + off) = ok ? packed : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        const bool put = in && ok && !is_q;
        if (!__any_sync(0xffffffffu, put)) continue;             // a warp of query heads
        const int j = h - a.H - (is_k ? 0 : Hkv);
        const size_t base = put ? (size_t)seq * a.kv.seq_stride + ((size_t)j * a.kv.n_ctx + pos) * HD : 0;
        if (Q4) {
            float d;
            uint32_t word;
            encode_exact<HD>(x, gain, turn, gp != nullptr, is_k, a.eps, u, put, lane, d, word);
            if (put) {
                out_of_range |= bad;
                const int blk = sub >> 2, tt = sub & 3;
                reinterpret_cast<uint32_t *>((is_k ? a.kv.k4 : a.kv.v4) + base / 2)[tt * (HD / 32) + blk] = word;
                if (tt == 0) (is_k ? a.kv.kd : a.kv.vd)[base / 32 + blk] = f2h(d);
            }
        } else if (put) {
            if (a.kv.k8) {
                *reinterpret_cast<uint2 *>((is_k ? a.kv.k8 : a.kv.v8) + base + e0) =
                    make_uint2((uint32_t)pack_e4m3x2(u[0], u[1]) | (uint32_t)pack_e4m3x2(u[2], u[3]) << 16,
                               (uint32_t)pack_e4m3x2(u[4], u[5]) | (uint32_t)pack_e4m3x2(u[6], u[7]) << 16);
            } else {
                out_of_range |= bad;
                *reinterpret_cast<uint4 *>((is_k ? a.kv.k : a.kv.v) + base + e0) = packed;
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
constexpr int SHIFT_THREADS = 256;

template <int HD>
__global__ void __launch_bounds__(SHIFT_THREADS) kv_shift_q4_kernel(KvView kv, int p0, int n, int end, const float2 *rope) {
    constexpr int L = HD / E, ROWS = SHIFT_THREADS / L, NB = HD / 32;
    const size_t base = (size_t)blockIdx.x * kv.n_ctx * HD;      // (layer, head) block of this sequence, in elements
    const int lane = threadIdx.x & 31, sub = threadIdx.x % L, r = threadIdx.x / L;
    const int blk = sub >> 2, at = (sub & 3) * NB + blk;
    uint32_t *kw = reinterpret_cast<uint32_t *>(kv.k4 + base / 2), *vw = reinterpret_cast<uint32_t *>(kv.v4 + base / 2);
    f16 *kd = kv.kd + base / 32, *vd = kv.vd + base / 32;
    float2 back[E / 2];                               // R(-n): (a, b) -> (a cos + b sin, -a sin + b cos)
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
        const float2 c = rope[(size_t)n * (HD / 2) + E / 2 * sub + e];
        back[e] = make_float2(c.x, -c.y);
    }
    const float gain[E] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    for (int r0 = p0 + n; r0 < end; r0 += ROWS) {
        const bool in = r0 + r < end;
        const size_t src = in ? r0 + r : r0, dst = src - n;
        const uint32_t w = kw[src * (HD / 8) + at], wv = vw[src * (HD / 8) + at];
        const float d = hf(kd[src * NB + blk]);
        const f16 dv = vd[src * NB + blk];
        float x[E], u[E], nd;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = (float)((int)((w >> q4::shift_of(e)) & 15u) - 8) * d;     // exact
        uint32_t out;
        transform<HD>(x, gain, back, false, true, 0.f, u);
        encode_exact<HD>(x, gain, back, false, true, 0.f, u, true, lane, nd, out);
        __syncthreads();
        if (in) {
            kw[dst * (HD / 8) + at] = out;
            vw[dst * (HD / 8) + at] = wv;
            if ((sub & 3) == 0) {
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
    // few rows: the heads of a row spread over several CTAs; many: one CTA a row
    const int per = 32 / (hd / E) * (THREADS / 32), parts = (heads + per - 1) / per;      // heads a CTA takes at once
    const dim3 grid(a.T, (long long)a.T * parts > 4 * 152 ? 1 : parts), block(THREADS);
    if (hd == 32) return launch_kernel(a.kv.k4 ? qk_norm_rope_kernel<32, true> : qk_norm_rope_kernel<32, false>, grid, block, 0, l, a);
    if (hd == 64) return launch_kernel(a.kv.k4 ? qk_norm_rope_kernel<64, true> : qk_norm_rope_kernel<64, false>, grid, block, 0, l, a);
    if (hd == 128) return launch_kernel(a.kv.k4 ? qk_norm_rope_kernel<128, true> : qk_norm_rope_kernel<128, false>, grid, block, 0, l, a);
    return cudaErrorInvalidValue;
}

}  // namespace llm
