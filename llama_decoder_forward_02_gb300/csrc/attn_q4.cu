// Decode attention over a Q4_0 cache ("LLama.cpp — how it works", "KV-cache": a
// quantised cache where memory is short; the attention itself as in
// attn_decode.cu): for each row t and query head h, o = softmax(q K^T /
// sqrt(hd)) V over the visible positions of sequence seq[t], K and V standing
// for d * (c - 8) (q4.cuh).
//
// Bound by HBM reads of K and V: 9/8 bytes a (key, element), which
// leaves an SM about 100 clocks for 16 keys of 128 elements at the copy
// bandwidth.  Widening every code on the CUDA cores costs more than that, so
// the codes go to mma.sync (q4.cuh): K's as the fp16 subnormals c * 2^-24 that
// masking a word leaves, V's as c - 8.
//   * S^T = K q^T with 16 keys as the M side.  A block of 32 dimensions is one
//     fp32 sum of two mma (the second's q divided by 16 for the nibbles that
//     stand four bits higher), less 8 sum(q) of the block, made once, for the
//     offset, and scaled by the key's d in fp32.
//   * The N side has 8 columns and a kv head rarely 8 query heads, so each
//     head takes two: q, times a power of two that brings its head's largest
//     element to 2^14 .. 2^15, as the sum of two fp16 numbers (22 bits), and so
//     its weights.  Four heads fill a column tile, larger groups take NT = 2.
//   * O^T += V^T w with 16 dimensions as the M side and w = p * d[key][block],
//     again as two fp16 numbers; neighbouring keys' halves of a word are put
//     together by one byte permute.  S^T comes out with keys along the lanes'
//     rows and w is wanted with heads there: a register transpose of the warp
//     (movmatrix) for each block.  w is held times a power of two that brings
//     the largest |d| a warp has met to 2^14 .. 2^15, so that both parts stay
//     normal numbers down to 2^-28 of it whatever V's size.  (With V's codes as
//     subnormals too and 8 sum(w) taken off at the end, w times 8: the parts'
//     rounding came in as error * c instead of error * (c - 8), and w of V near
//     1e-3 lost it altogether, 9.4e-4 of o's norm.)
// So neither q, K, V nor the weights are rounded to fewer than 22 bits on the
// way to the fp32 sums; only o is.
//
// A warp walks every NW-th group of 16 keys of its CTA's span through a ring
// of its own, filled by cp.async (16-byte chunks swizzled so that both K's and
// V's fragment reads are free of bank conflicts); warps meet only at the end.
// The running maximum of a head is raised by a warp-uniform branch when a key
// passes it.  Splits over the keys leave (numerators, sum, max) and are merged
// in split order, by the cluster they form or, over long caches, by the CTA that
// arrives last: results do not depend on timing and nothing spins.
//
// Measured, calls in a row in a captured graph, 32 query and 8 kv heads of 128,
// and the time the bytes take at the copy bandwidth: one row of 2100 keys 4.4 us
// (0.4), of 32000 keys 12.4 (5.4), eight rows of 748 to 3415 keys 10.1 (3.0); with
// V's codes as subnormals too and weights times 8 they were 4.4, 12.0 and 9.6.  Of
// the 12.0, which calls from C stretched to 12.9: 1.3 to q's fragments, 6.9 of loop
// (5.3 TB/s), 0.9 for the warps' sums, 2.4 for the count, the reads and the merge,
// 1.4 to the next call.  The schedulers issue in 54% of the SM's clocks (ALU 43%)
// over the whole kernel.  In a cluster each split
// sends its share to the rank that merges it before the one barrier they meet
// at; reading it there after the barrier, with a second one to leave by, took
// 0.7 more.
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "q4.cuh"

namespace llm {

namespace {

constexpr int GC = 8;                    // query heads of a chunk
constexpr int KG = 16;                   // keys of a group
constexpr int NST = 4;                   // ring stages of a warp
constexpr int MAX_SPLIT = ATTN_DECODE_MAX_SPLIT;
constexpr int MIN_GRP = 8;               // groups of a split, at least
constexpr int MERGE_AHEAD = 40;          // splits whose partials a merging thread asks for at once
constexpr int MAX_CLUSTER = 8;           // splits merged in a cluster
constexpr int CLUSTER_CTX = 8192;        // longest cache whose splits always are one cluster
constexpr int BALANCE_T = 128;           // most rows that share the splits of a launch ...
constexpr int BALANCE_UNITS = 2048;      // ... and most (row, kv head, chunk)s, each of which has a counter
constexpr int SMS = 152;                 // of the one GPU this library is compiled for: scratch sizes follow from it

template <int HD, int NW>
struct Ring {
    static constexpr int NB = HD / 32;               // blocks of a row
    static constexpr int ROW = HD / 2;               // bytes of a row's codes
    static constexpr int CODES = KG * ROW;           // ... of a group's
    static constexpr int SCALES = HD == 32 ? 0 : KG * NB * 2;   // ... and of its scales (HD 32: read from global)
    static constexpr int STAGE = 2 * CODES + 2 * SCALES;
    static constexpr size_t BYTES = (size_t)NW * NST * STAGE;
    static constexpr size_t MERGE = (size_t)NW * GC * (HD + 2) * sizeof(float);
    static constexpr size_t QFRAG = (size_t)2 * NB * (32 * 16 + 16);      // q's fragments, two tiles at most
    static constexpr size_t WGT = BYTES > MERGE ? BYTES : MERGE;          // split weights, after the rings or the results
    static constexpr size_t SMEM = BYTES + QFRAG > WGT + GC * MAX_SPLIT * sizeof(float) ? BYTES + QFRAG : WGT + GC * MAX_SPLIT * sizeof(float);
    // a cluster's splits send a CTA its share of their results behind all that, where another may still be reading q
    static constexpr size_t INBOX = ((BYTES + QFRAG > MERGE ? BYTES + QFRAG : MERGE) + 15) & ~(size_t)15;
    static constexpr size_t SMEM_CL = INBOX + (size_t)GC * (HD / 2) * sizeof(float4);
    // byte offset of word block `part` (4 NB bytes, lane t4 of a K row) of row r
    __device__ static __forceinline__ int at(int r, int part) {
        if (HD == 128) return r * ROW + ((part ^ ((r >> 1) & 3)) << 4);
        if (HD == 64) return r * ROW + (((part >> 1) ^ ((r >> 2) & 1)) << 4) + (part & 1) * 8;
        return r * ROW + part * 4;
    }
};

template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, bool pred) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" :: "r"(dst), "l"(src), "n"(N), "r"(pred ? N : 0));
}

__device__ __forceinline__ void mma_acc(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^x with a relative error of 2^-22, 0 below 2^-126
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// v as the sum of two fp16 numbers, the larger in the low half: the low 13
// mantissa bits are split off exactly, so the pair keeps 22 bits where the
// first part is normal and 2^-25 absolute below.
__device__ __forceinline__ uint32_t two_halves(float v) {
    const float hi = __uint_as_float(__float_as_uint(v) & 0xFFFFE000u);
    return pack_h2(hi, v - hi);
}

// NB words of a row part
template <int NB>
__device__ __forceinline__ void load_words(uint32_t (&w)[NB], const uint8_t *p) {
    if constexpr (NB == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (NB == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// NB fp16 scales as float
template <int NB>
__device__ __forceinline__ void load_scales(float (&d)[NB], const void *p) {
    if constexpr (NB == 1) {
        d[0] = hf(*reinterpret_cast<const f16 *>(p));
    } else {
        uint32_t w[NB / 2];
        load_words<NB / 2>(w, reinterpret_cast<const uint8_t *>(p));
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) { d[2 * i] = h2lo(w[i]); d[2 * i + 1] = h2hi(w[i]); }
    }
}

// The keys a row sees: S of them from lo on, none if its position or sequence
// lies outside the cache.
struct Row {
    int lo, S;
    bool ok;
    __device__ __forceinline__ int groups() const { return (S + KG - 1) / KG; }
};
__device__ __forceinline__ Row row_keys(const AttnDecodeArgs &a, int pos, int seq) {
    Row r;
    r.ok = pos >= 0 && pos < a.kv.n_ctx && seq >= 0 && seq < a.kv.n_seq;
    r.lo = r.ok && a.window > 0 && pos + 1 > a.window ? pos + 1 - a.window : 0;
    r.S = r.ok ? pos + 1 - r.lo : 0;
    return r;
}

// Which row and split of it CTA x of a.n_split works on, by its warp: the rows
// share the splits by their lengths, each row's being of len groups (the last
// shorter) and at least one.  With X splits, T rows and N groups in all, len =
// ceil(N / (X - T + 1)) needs no more than X, as a row with keys rounds up by
// less than one; half that allowance is tried first.  Returns the split, or -1
// where none is left for x.
__device__ __forceinline__ int find_split(const AttnDecodeArgs &a, int x, int lane, int &t, Row &rw, int &pos, int &seq,
                                          int &len, int &n_eff) {
    const int X = a.n_split, T = a.T;
    auto load = [&](int r) {
        pos = r < T ? a.pos[r] : -1;
        seq = r < T ? a.seq[r] : -1;
        rw = row_keys(a, pos, seq);
        return rw.groups();
    };
    if (T == 1) {
        pos = a.pos[0];
        seq = a.seq[0];
        rw = row_keys(a, pos, seq);
        t = 0;
        len = max(MIN_GRP, (rw.groups() + X - 1) / X);
        n_eff = max(1, (rw.groups() + len - 1) / len);
        return x < n_eff ? x : -1;
    }
    unsigned sum = 0, most = 0;
    int mine = 0;
    for (int r = lane; r < (T + 31) / 32 * 32; r += 32) {
        mine = load(r);
        sum += mine;
        most = max(most, (unsigned)mine);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    most = __reduce_max_sync(0xffffffffu, most);
    const unsigned least = max((unsigned)MIN_GRP, (most + MAX_SPLIT - 1) / MAX_SPLIT);
    auto splits = [&](int r, int groups) { return r < T ? max(1, (groups + len - 1) / len) : 0; };
    for (int take = T / 2;; take = T - 1) {
        const unsigned n = (unsigned)(X - take);
        len = (int)max(least, (sum + n - 1) / n);
        if (take == T - 1) break;
        unsigned used = 0;
        for (int r = lane; r < (T + 31) / 32 * 32; r += 32) used += splits(r, T <= 32 ? mine : load(r));
        if (__reduce_add_sync(0xffffffffu, used) <= (unsigned)X) break;
    }
    int base = 0;
    for (int r0 = 0; r0 < T; r0 += 32) {
        const int n = splits(r0 + lane, T <= 32 ? mine : load(r0 + lane));
        int end = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, end, d);
            if (lane >= d) end += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + end > x);
        if (past) {
            const int l = __ffs(past) - 1;
            t = r0 + l;
            n_eff = __shfl_sync(0xffffffffu, n, l);
            const int first = base + __shfl_sync(0xffffffffu, end, l) - n_eff;
            pos = __shfl_sync(0xffffffffu, pos, l);
            seq = __shfl_sync(0xffffffffu, seq, l);
            rw = row_keys(a, pos, seq);
            return x - first;
        }
        base += __shfl_sync(0xffffffffu, end, 31);
    }
    return -1;
}

// CL: the splits of a (row, kv head, chunk) are the CTAs of one cluster and are
// merged through distributed shared memory; else through a.part by the CTA that
// arrives last.
template <int HD, int NT, int NW, bool CL>
__global__ void __launch_bounds__(NW * 32, NT == 1 && NW == 8 ? 2 : 1) attn_decode_q4_kernel(const AttnDecodeArgs a, int chunks) {
    using R = Ring<HD, NW>;
    constexpr int NB = R::NB, REC = HD + 2, THREADS = NW * 32;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ int s_last;
    const int j = chunks == 1 ? blockIdx.y : blockIdx.y / chunks, ck = blockIdx.y - j * chunks;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int Hkv = a.kv.n_kv_head, G = a.H / Hkv, h0 = j * G + ck * GC, gn = min(GC, G - ck * GC);
    if (!a.early) {
        pdl_wait();
        pdl_trigger();
    }
    int sp = blockIdx.x, t = blockIdx.z, pos, seq, n_eff;
    Row rw;
    int len;                                          // groups of a split
    if constexpr (CL) {
        pos = a.pos[t];
        seq = a.seq[t];
        rw = row_keys(a, pos, seq);
        len = max(MIN_GRP, (rw.groups() + a.n_split - 1) >> (31 - __clz(a.n_split)));
        n_eff = a.n_split;                            // all stay for the cluster's barriers
    } else {
        sp = find_split(a, blockIdx.x, lane, t, rw, pos, seq, len, n_eff);
        if (sp < 0) {
            if (a.early) pdl_wait();                  // no CTA leaves before the kernel ahead is done
            return;
        }
    }
    if (!rw.ok && tid == 0 && sp == 0 && blockIdx.y == 0) raise_error(a.err, ERRF_BAD_INDEX);
    const long long at = (long long)sp * len * KG;    // first key of the split
    const int kb = rw.lo + (int)min((long long)rw.S, at), ke = rw.lo + (int)min((long long)rw.S, at + (long long)len * KG);
    const size_t row0 = rw.ok ? ((size_t)seq * a.kv.seq_stride + (size_t)j * a.kv.n_ctx * HD) / HD : 0;   // rows before the head's

    // ---- this warp's groups: keys kb + KG (warp + NW i)
    uint8_t *ring = smem_raw + (size_t)warp * NST * R::STAGE;
    const int n_grp = ke > kb + KG * warp ? (ke - kb - KG * warp + NW * KG - 1) / (NW * KG) : 0;
    // this lane's rows and chunks of a group; sources of the next group to request
    constexpr int CH = R::ROW / 16, PER = KG * CH, NCP = (PER + 31) / 32;   // 16-byte chunks of a row, of a group
    constexpr int RSTEP = 32 / CH;                                          // rows between a lane's chunks
    const int cr = lane / CH, cc = lane - cr * CH, left0 = ke - kb - KG * warp;
    const uint8_t *ksrc = a.kv.k4 + (row0 + kb + KG * warp + cr) * R::ROW + cc * 16;
    const uint8_t *vsrc = a.kv.v4 + (row0 + kb + KG * warp + cr) * R::ROW + cc * 16;
    const f16 *ssrc = (lane < 16 ? a.kv.kd : a.kv.vd) + (row0 + kb + KG * warp + (lane & 15)) * NB;
    const uint32_t ring0 = smem_u32(ring);
    int left = left0, want = 0;                       // keys from the next requested group on; its ring slot
    auto request = [&]() {
        if (left > 0) {
            const uint32_t st = ring0 + (uint32_t)want * R::STAGE;
#pragma unroll
            for (int q = 0; q < NCP; ++q) {
                const int r = cr + q * RSTEP;
                if (PER % 32 == 0 || lane < PER) {
                    const bool in = r < left;         // rows past the span are zeros, their address the span's first
                    const uint32_t dst = st + R::at(r, HD == 128 ? cc : HD == 64 ? 2 * cc : 0);
                    const int o = in ? q * RSTEP * R::ROW : -cr * R::ROW;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(ksrc + o), "r"(in ? 16 : 0));
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst + R::CODES), "l"(vsrc + o), "r"(in ? 16 : 0));
                }
            }
            if constexpr (HD != 32) {
                const int r = lane & 15;
                const bool in = r < left;
                cp_async_small<NB * 2>(st + 2 * R::CODES + (lane < 16 ? 0 : R::SCALES) + r * NB * 2, in ? ssrc : ssrc - r * NB, in);
            }
            left -= NW * KG;
            ksrc += NW * KG * R::ROW;
            vsrc += NW * KG * R::ROW;
            ssrc += NW * KG * NB;
            want = want + 1 == NST ? 0 : want + 1;
        }
        cp_async_commit();
    };
    // ---- q as the N side: column g of tile n is half g % 2 of head 4 n + g / 2.
    // The fragments are the same for every warp: each makes some blocks' and
    // leaves them in shared memory.  q times the power of two that brings its
    // head's largest element to 2^14 .. 2^15, as it is for the nibbles at bits 0
    // and 8 and divided by 16 for those four bits higher.
    uint4 *qf = reinterpret_cast<uint4 *>(smem_raw + R::BYTES);            // [NT * NB][32]
    float *q8 = reinterpret_cast<float *>(qf + NT * NB * 32);              // [NT * NB][4]: 8 sum(q) * 2^-24 of the columns' head
    __shared__ float s_qmax[NT * NB][4];                                   // a block's largest |q| by head
    static_assert(NT * NB <= NW, "a warp makes one block's fragments");
    int asked = 0;                                    // groups requested
    if (a.early) {                                    // cells that no row of this launch's batch was appended to
        while (asked < NST - 1 && kb + KG * (warp + NW * asked) + KG <= pos + 1 - a.T) {
            request();
            ++asked;
        }
        pdl_wait();
        pdl_trigger();
    }
    float4 x0 = make_float4(0.f, 0.f, 0.f, 0.f), x1 = x0;
    if (warp < NT * NB && 4 * (warp / NB) + (g >> 1) < gn) {
        const float4 *qp = reinterpret_cast<const float4 *>(a.q + ((size_t)t * a.H + h0 + 4 * (warp / NB) + (g >> 1)) * HD +
                                                            32 * (warp % NB) + 8 * t4);
        x0 = __ldcg(qp);                              // through L2: q is rewritten between uses; ahead of the
        x1 = __ldcg(qp + 1);                          // ring's burst, behind which it would wait 2 us
    }
#pragma unroll
    for (int i = 0; i < NST - 1; ++i)
        if (i >= asked) request();
    if constexpr (CL) cluster_arrive_relaxed();       // started: the others may write to this CTA once they have waited
    const float qv[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    if (warp < NT * NB) {
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(qv[e]));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        if (t4 == 0 && !(g & 1)) s_qmax[warp][g >> 1] = most;
    }
    __syncthreads();
    // exponent of the largest element of a head: 2^(e - 127) .. 2^(e - 126)
    auto q_exp = [&](int n, int h) {
        float most = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) most = fmaxf(most, s_qmax[n * NB + b][h]);
        return (int)min(max(__float_as_uint(most) >> 23, 14u), 243u);
    };
    if (warp < NT * NB) {
        const int u = warp;
        const float up = __uint_as_float((uint32_t)(268 - q_exp(warp / NB, g >> 1)) << 23);      // 2^(141 - e)
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = qv[e] * up;
            const uint32_t two = two_halves((e & 2) ? x * 0.0625f : x);   // elements 2, 3, 6, 7: nibbles four bits up
            h[e] = g & 1 ? two >> 16 : two & 0xFFFFu;
        }
        const uint4 f = make_uint4(h[0] | h[1] << 16, h[4] | h[5] << 16, h[2] | h[3] << 16, h[6] | h[7] << 16);
        qf[u * 32 + lane] = f;
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        mma_acc(c, 0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u, f.x, f.y);
        mma_acc(c, 0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u, f.z, f.w);
        if (g == 0) q8[u * 4 + t4] = c[0] + c[1];
    }
    __syncthreads();
    uint32_t qb[NT][NB][4];
    float off[NT][NB];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint4 f = qf[(n * NB + b) * 32 + lane];
            qb[n][b][0] = f.x; qb[n][b][1] = f.y; qb[n][b][2] = f.z; qb[n][b][3] = f.w;
            off[n][b] = q8[(n * NB + b) * 4 + t4];
        }
    // from the sums to scores in base 2: the 2^24 of the codes, q's power of two, log2(e) / sqrt(hd)
    float undo[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        undo[n] = __uint_as_float((uint32_t)(q_exp(n, t4) + 10) << 23) * (1.4426950408889634f / sqrtf((float)HD));

    // sums of the lane's head(s) 4 n + t4: O^T tiles of 16 dimensions (two a block), weights
    float o[NT][NB][2][4], m[NT], l[NT];
    // o is held sig times as large, a power of two that brings this warp's largest |d| of V to 2^14 or more; one of
    // top or more lowers it
    float sig = 0x1p39f, unsig = 0x1p-39f, top = 0x1p-24f;
    const q4::Widen wd;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n] = -INFINITY; l[n] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][b][0][e] = o[n][b][1][e] = 0.f;
        }
    }
    const uint32_t sel = g & 1 ? 0x7632u : 0x5410u;       // V: lane g takes half g % 2 of words of part g / 2

    int slot = 0, valid = left0;                      // keys from this group on
    for (int i = 0; i < n_grp; ++i) {
        cp_async_wait<NST - 2>();
        __syncwarp();
        request();                                        // into the slot read in step i - 1
        const uint8_t *st = ring + (size_t)slot * R::STAGE;
        const bool in0 = g < valid, in1 = g + 8 < valid;
        uint32_t kw[2][NB];
        load_words<NB>(kw[0], st + R::at(g, t4));
        load_words<NB>(kw[1], st + R::at(g + 8, t4));
        float dk[2][NB], dv[2][NB];
        if constexpr (HD == 32) {
            const size_t r = row0 + kb + KG * (warp + NW * i) + g;
            dk[0][0] = in0 ? hf(a.kv.kd[r]) : 0.f; dk[1][0] = in1 ? hf(a.kv.kd[r + 8]) : 0.f;
            dv[0][0] = in0 ? hf(a.kv.vd[r]) : 0.f; dv[1][0] = in1 ? hf(a.kv.vd[r + 8]) : 0.f;
        } else {
            const uint8_t *sc = st + 2 * R::CODES + g * NB * 2;
            load_scales<NB>(dk[0], sc);
            load_scales<NB>(dk[1], sc + 8 * NB * 2);
            load_scales<NB>(dv[0], sc + R::SCALES);
            load_scales<NB>(dv[1], sc + R::SCALES + 8 * NB * 2);
        }
        float s[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t u = kw[0][b], v = kw[1][b], u8 = u >> 8, v8 = v >> 8;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                mma_acc(c, u & 0x000F000Fu, v & 0x000F000Fu, u8 & 0x000F000Fu, v8 & 0x000F000Fu, qb[n][b][0], qb[n][b][1]);
                mma_acc(c, u & 0x00F000F0u, v & 0x00F000F0u, u8 & 0x00F000F0u, v8 & 0x00F000F0u, qb[n][b][2], qb[n][b][3]);
                s[n][0] = fmaf(dk[0][b], (c[0] + c[1]) + off[n][b], s[n][0]);
                s[n][1] = fmaf(dk[1][b], (c[2] + c[3]) + off[n][b], s[n][1]);
            }
        }
        // m and s in units of 1 / undo
        float dmax = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) dmax = fmaxf(dmax, fmaxf(fabsf(dv[0][b]), fabsf(dv[1][b])));
        bool raise = dmax >= top;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            s[n][0] = in0 ? s[n][0] : -INFINITY;
            s[n][1] = in1 ? s[n][1] : -INFINITY;
            raise |= fmaxf(s[n][0], s[n][1]) > m[n];
        }
        if (__any_sync(0xffffffffu, raise)) {
            const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(dmax));     // of floats from 0 on
            float drop = 1.f;
            if (most >= __float_as_uint(top)) {
                // 2^(e - 127) .. 2^(e - 126): sig = 2^(141 - e) from then on
                const uint32_t e = min(most >> 23, 253u);
                top = __uint_as_float((e + 1) << 23);
                sig = __uint_as_float((268 - e) << 23);
                drop = sig * unsig;
                unsig = __uint_as_float((e - 14) << 23);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float mx = fmaxf(s[n][0], s[n][1]);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                mx = fmaxf(mx, m[n]);
                const float f = mx == -INFINITY ? 1.f : exp2f((m[n] - mx) * undo[n]);
                m[n] = mx;
                l[n] *= f;
                const float fo = f * drop;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) { o[n][b][0][e] *= fo; o[n][b][1][e] *= fo; }
                }
            }
        }
        float p[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float m0 = m[n] == -INFINITY ? 0.f : m[n];
            p[n][0] = exp2_fast((s[n][0] - m0) * undo[n]);
            p[n][1] = exp2_fast((s[n][1] - m0) * undo[n]);
            l[n] += p[n][0] + p[n][1];
            p[n][0] *= sig;
            p[n][1] *= sig;
        }
        uint32_t vw[4][NB];
#pragma unroll
        for (int q = 0; q < 4; ++q) load_words<NB>(vw[q], st + R::CODES + R::at(2 * t4 + (q & 1) + 8 * (q >> 1), g >> 1));
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t u = __byte_perm(vw[0][b], vw[1][b], sel), v = __byte_perm(vw[2][b], vw[3][b], sel);
            const uint32_t u8 = u >> 8, v8 = v >> 8;
            const uint32_t ul = wd.low(u), uh = wd.high(u), ul8 = wd.low(u8), uh8 = wd.high(u8);
            const uint32_t vl = wd.low(v), vh = wd.high(v), vl8 = wd.low(v8), vh8 = wd.high(v8);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float w0 = p[n][0] * dv[0][b], w1 = p[n][1] * dv[1][b];
                const uint32_t b0 = transpose8x8(two_halves(w0)), b1 = transpose8x8(two_halves(w1));
                mma_acc(o[n][b][0], ul, ul8, vl, vl8, b0, b1);
                mma_acc(o[n][b][1], uh, uh8, vh, vh8, b0, b1);
            }
        }
        valid -= NW * KG;
        slot = slot + 1 == NST ? 0 : slot + 1;
    }
    cp_async_wait<0>();
    __syncthreads();                                      // the rings become the warps' results

    // the warps' largest maximum of each head, then their results in its units
    float *wst = reinterpret_cast<float *>(smem_raw);     // [NW][GC][REC]: numerators, sum
    float *wgt = reinterpret_cast<float *>(smem_raw + R::WGT);   // [GC][MAX_SPLIT]
    __shared__ float s_max[NW][GC];
    if (g == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s_max[warp][4 * n + t4] = m[n] * undo[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, s_max[w][4 * n + t4]);
        const float f = m[n] == -INFINITY ? 0.f : exp2_fast(m[n] * undo[n] - M);
        float *ws = wst + ((size_t)warp * GC + 4 * n + t4) * REC;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n] += __shfl_xor_sync(0xffffffffu, l[n], x);
        if (g == 0) ws[HD] = l[n] * f;
        const float f1 = f * unsig;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float *d = ws + 32 * b + 8 * (g >> 1) + (g & 1);
            d[0] = (o[n][b][0][0] + o[n][b][0][1]) * f1;
            d[4] = (o[n][b][0][2] + o[n][b][0][3]) * f1;
            d[2] = (o[n][b][1][0] + o[n][b][1][1]) * f1;
            d[6] = (o[n][b][1][2] + o[n][b][1][3]) * f1;
        }
    }
    __syncthreads();
    // records of a split: numerators, sum, maximum
    const bool one = !CL && n_eff == 1;
    float *part = a.part + ((size_t)h0 * a.n_split + blockIdx.x) * REC;
    const size_t part_head = (size_t)a.n_split * REC;
    // CL: rank r merges the (head, dimension pair)s [r share, (r + 1) share) of all ranks' records
    float4 *inbox = reinterpret_cast<float4 *>(smem_raw + R::INBOX);       // [rank][share]
    const int share = gn * (HD / 2) / (CL ? a.n_split : 1);
    if constexpr (CL) cluster_wait();
    for (int i = tid; i < gn * (HD / 2); i += THREADS) {
        const int h = i / (HD / 2), d = 2 * (i - h * (HD / 2));
        float2 num = make_float2(0.f, 0.f);
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float *ws = wst + ((size_t)w * GC + h) * REC;
            const float2 v = *reinterpret_cast<const float2 *>(ws + d);
            num.x += v.x;
            num.y += v.y;
            den += ws[HD];
        }
        if constexpr (CL) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < NW; ++w) M = fmaxf(M, s_max[w][h]);
            const int r = i / share;
            dsmem_st_f32x4(dsmem(inbox + sp * share + (i - r * share), (uint32_t)r), make_float4(num.x, num.y, den, M));
        } else if (one) {
            const float inv = den > 0.f ? 1.f / den : 0.f;
            *reinterpret_cast<uint32_t *>(a.o + ((size_t)t * a.H + h0 + h) * HD + d) = pack_h2(num.x * inv, num.y * inv);
        } else {
            float *rp = part + h * part_head;
            *reinterpret_cast<float2 *>(rp + d) = num;
            if (d == 0) {
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < NW; ++w) M = fmaxf(M, s_max[w][h]);
                *reinterpret_cast<float2 *>(rp + HD) = make_float2(den, M);
            }
        }
    }
    if (one) return;
    if constexpr (CL) {
        cluster_sync();
        for (int k = tid; k < share; k += THREADS) {
            const int i = sp * share + k, h = i / (HD / 2), d = 2 * (i - h * (HD / 2));
            float4 v[MAX_CLUSTER];
#pragma unroll
            for (int p = 0; p < MAX_CLUSTER; ++p) v[p] = p < a.n_split ? inbox[p * share + k] : make_float4(0.f, 0.f, 0.f, -INFINITY);
            float M = -INFINITY, den = 0.f;
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < MAX_CLUSTER; ++p) M = fmaxf(M, v[p].w);
#pragma unroll
            for (int p = 0; p < MAX_CLUSTER; ++p) {
                const float f = v[p].w == -INFINITY ? 0.f : exp2_fast(v[p].w - M);
                acc.x = fmaf(f, v[p].x, acc.x);
                acc.y = fmaf(f, v[p].y, acc.y);
                den = fmaf(f, v[p].z, den);
            }
            const float inv = den > 0.f ? 1.f / den : 0.f;
            *reinterpret_cast<uint32_t *>(a.o + ((size_t)t * a.H + h0 + h) * HD + d) = pack_h2(acc.x * inv, acc.y * inv);
        }
        return;
    }
    __syncthreads();
    unsigned *cnt = a.counters + (size_t)t * gridDim.y + blockIdx.y;
    // one thread's release covers the CTA's writes before the barrier, its
    // acquire the reads of every thread after the next
    if (tid == 0) {
        unsigned before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(cnt) : "memory");
        s_last = before == (unsigned)(n_eff - 1);
    }
    __syncthreads();
    if (!s_last) return;

    // ---- last CTA of this (row, kv head, chunk): each thread asks for its two
    // dimensions of the first MERGE_AHEAD splits while the warps find the splits'
    // weights, then sums them in split order
    const float *all = a.part + ((size_t)h0 * a.n_split + (blockIdx.x - sp)) * REC;
    float2 v[MERGE_AHEAD];
    const int mh = tid / (HD / 2), md = 2 * (tid - mh * (HD / 2));
    if (mh < gn) {
        const float *rp = all + (size_t)mh * a.n_split * REC + md;
#pragma unroll
        for (int p = 0; p < MERGE_AHEAD; ++p)
            if (p < n_eff) v[p] = __ldcg(reinterpret_cast<const float2 *>(rp + (size_t)p * REC));
    }
    for (int h = warp; h < gn; h += NW) {
        const float *rp = all + (size_t)h * a.n_split * REC + HD;
        float mx = -INFINITY;
        float2 lm[MAX_SPLIT / 32];
#pragma unroll
        for (int q = 0; q < MAX_SPLIT / 32; ++q) {
            const int p = lane + 32 * q;
            lm[q] = p < n_eff ? __ldcg(reinterpret_cast<const float2 *>(rp + (size_t)p * REC)) : make_float2(0.f, -INFINITY);
            mx = fmaxf(mx, lm[q].y);
        }
        mx = warp_max(mx);
        float den = 0.f;
#pragma unroll
        for (int q = 0; q < MAX_SPLIT / 32; ++q) {
            lm[q].y = mx == -INFINITY ? 0.f : exp2_fast(lm[q].y - mx);
            den += lm[q].y * lm[q].x;
        }
        den = warp_sum(den);
        const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
        for (int q = 0; q < MAX_SPLIT / 32; ++q)
            if (lane + 32 * q < n_eff) wgt[h * MAX_SPLIT + lane + 32 * q] = lm[q].y * inv;
    }
    __syncthreads();
    for (int i = tid; i < gn * (HD / 2); i += THREADS) {
        const int h = i / (HD / 2), d = 2 * (i - h * (HD / 2));
        const float *rp = all + (size_t)h * a.n_split * REC + d;
        float2 acc = make_float2(0.f, 0.f);
        int p = 0;
        if (i == tid) {
#pragma unroll
            for (int q = 0; q < MERGE_AHEAD; ++q)
                if (q < n_eff) {
                    const float f = wgt[h * MAX_SPLIT + q];
                    acc.x = fmaf(f, v[q].x, acc.x);
                    acc.y = fmaf(f, v[q].y, acc.y);
                }
            p = MERGE_AHEAD;
        }
#pragma unroll 16
        for (; p < n_eff; ++p) {
            const float2 w = __ldcg(reinterpret_cast<const float2 *>(rp + (size_t)p * REC));
            const float f = wgt[h * MAX_SPLIT + p];
            acc.x = fmaf(f, w.x, acc.x);
            acc.y = fmaf(f, w.y, acc.y);
        }
        *reinterpret_cast<uint32_t *>(a.o + ((size_t)t * a.H + h0 + h) * HD + d) = pack_h2(acc.x, acc.y);
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

__global__ void __launch_bounds__(WT) kv_rows_q4_kernel(const uint8_t *codes, const f16 *scales, const KvView kv,
                                                        const int *pos, const int *seq, f16 *out, int T, uint32_t *err) {
    pdl_wait();
    pdl_trigger();
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

// How the keys are split.
//
// (The times below were taken side by side, calls from C, before weights kept 22
// bits for V of any size; they are 3 to 5% more since.)
//
// Caches of up to CLUSTER_CTX positions and many rows: every (row, kv head,
// chunk) has the same number of splits, a power of two up to MAX_CLUSTER, and
// they are one cluster; about two CTAs of 8 warps an SM in all.  The merge
// inside a cluster costs a good microsecond less than the one through memory
// (8 kv heads of 128: one row of 2100 keys 4.7 us, 6.3 in 16 splits through
// memory; of 4000 keys 5.5 and 6.7; of 8000 keys 7.4 and 7.5; eight rows of 4000
// keys 11.9 and 14.7).  Clusters of sixteen take 5.4 for the 2100 keys and 7.7
// for the 8000.
//
// Longer caches: the rows share the splits by their lengths (find_split),
// merged through memory.  One or two rows of 8 kv heads get one CTA of 16 warps
// an SM, more rows two of 8.  One row of 32000 keys 12.9 us (two CTAs of 8
// warps, 32 splits: 14.8, as 104 SMs had two of them and 48 one; 38 splits
// 15.9 for their merge); four rows of 2000 to 16000 keys 13.9; eight rows of
// 1000 to 30000 keys 32 (clusters of four, whose CTAs wait for the longest
// row's, 56).
namespace {

int chunks_of(int H, int Hkv) { return (H / Hkv + GC - 1) / GC; }

struct Plan { int n_split, warps; bool cluster; };

Plan plan_of(int T, int H, int Hkv, int n_ctx) {
    const long long heads = (long long)Hkv * chunks_of(H, Hkv), units = T * heads;
    const long long most = std::max(1, n_ctx / (MIN_GRP * KG) + (n_ctx % (MIN_GRP * KG) > 0));   // splits of a row
    const bool wide = H / Hkv > 4;
    Plan p;
    p.cluster = n_ctx <= CLUSTER_CTX || T > BALANCE_T || units > BALANCE_UNITS || (long long)T * n_ctx > 1ll << 34;
    if (p.cluster) {
        long long s = std::min((wide ? 1ll : 2ll) * SMS / units, most);
        s = std::min(std::max(s, 1ll), (long long)MAX_CLUSTER);
        while (s & (s - 1)) ++s;
        p.n_split = (int)s;
        p.warps = 8;
    } else {
        p.warps = !wide && 8 * units <= SMS ? 16 : 8;
        const long long s = (wide || p.warps == 16 ? 1 : 2) * SMS / heads;
        p.n_split = (int)std::min(std::max(s, 2ll * T), T * std::min(most, (long long)MAX_SPLIT));
    }
    return p;
}

}  // namespace

size_t attn_q4_scratch_bytes(int T, int H, int Hkv, int hd, int n_ctx) {
    const Plan p = plan_of(T, H, Hkv, n_ctx);
    return BALANCE_UNITS * sizeof(unsigned) + (p.cluster ? 0 : (size_t)p.n_split * H * (hd + 2) * sizeof(float));
}

cudaError_t launch_attn_decode_q4(AttnDecodeArgs a, void *scratch, const Launch &l) {
    const int Hkv = a.kv.n_kv_head;
    if (a.T < 1 || a.T > 65535 || Hkv < 1 || a.H % Hkv || !a.kv.k4) return cudaErrorInvalidValue;
    const int chunks = chunks_of(a.H, Hkv);
    if ((long long)Hkv * chunks > 65535) return cudaErrorInvalidValue;
    const Plan p = plan_of(a.T, a.H, Hkv, a.kv.n_ctx);
    a.n_split = p.n_split;
    a.counters = (unsigned *)scratch;
    a.part = (float *)(a.counters + BALANCE_UNITS);
    const bool wide = a.H / Hkv > 4;                  // four heads fill the 8 columns of a tile; larger groups take two tiles
    const dim3 grid(p.n_split, Hkv * chunks, p.cluster ? a.T : 1), block(p.warps * 32);
#define Q4_DEC_CASE1(HDV, NT, NW)                                                                                     \
    if (a.kv.head_dim == HDV && wide == (NT == 2) && p.warps == NW && !p.cluster)                                     \
        return launch_kernel(attn_decode_q4_kernel<HDV, NT, NW, false>, grid, block, Ring<HDV, NW>::SMEM, l, a, chunks);
#define Q4_DEC_CASE(HDV)                                                                                              \
    if (a.kv.head_dim == HDV && p.cluster)                                                                            \
        return launch_cluster_kernel(wide ? attn_decode_q4_kernel<HDV, 2, 8, true> : attn_decode_q4_kernel<HDV, 1, 8, true>, \
                                     grid, block, p.n_split, Ring<HDV, 8>::SMEM_CL, l, a, chunks);                       \
    Q4_DEC_CASE1(HDV, 1, 8) Q4_DEC_CASE1(HDV, 1, 16) Q4_DEC_CASE1(HDV, 2, 8)
    Q4_DEC_CASE(32) Q4_DEC_CASE(64) Q4_DEC_CASE(128)
#undef Q4_DEC_CASE
#undef Q4_DEC_CASE1
    return cudaErrorInvalidValue;
}

cudaError_t init_attn_q4_attributes() {
    cudaError_t e = cudaSuccess;
#define Q4_DEC_ATTR1(HDV, NT, NWV, CL)                                                         \
    if (!e) e = allow_smem(attn_decode_q4_kernel<HDV, NT, NWV, CL>, CL ? Ring<HDV, NWV>::SMEM_CL : Ring<HDV, NWV>::SMEM); \
    if (!e) e = cudaFuncSetAttribute(attn_decode_q4_kernel<HDV, NT, NWV, CL>,                  \
                                     cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
#define Q4_DEC_ATTR(HDV)                                                                        \
    Q4_DEC_ATTR1(HDV, 1, 8, true) Q4_DEC_ATTR1(HDV, 1, 8, false) Q4_DEC_ATTR1(HDV, 1, 16, false) \
    Q4_DEC_ATTR1(HDV, 2, 8, true) Q4_DEC_ATTR1(HDV, 2, 8, false)
    Q4_DEC_ATTR(32) Q4_DEC_ATTR(64) Q4_DEC_ATTR(128)
#undef Q4_DEC_ATTR
#undef Q4_DEC_ATTR1
    return e;
}

cudaError_t launch_kv_rows_q4(const uint8_t *codes, const f16 *scales, const KvView &kv, const int *pos,
                              const int *seq, f16 *out, int T, uint32_t *err, const Launch &l) {
    const long long n = (long long)T * kv.n_kv_head * (kv.head_dim / 8);
    if (T < 1 || (n + WT - 1) / WT >= (1ll << 31)) return cudaErrorInvalidValue;
    return launch_kernel(kv_rows_q4_kernel, dim3((unsigned)((n + WT - 1) / WT)), dim3(WT), 0, l, codes, scales, kv, pos,
                         seq, out, T, err);
}

}  // namespace llm
