// Attention of the nodes of trees of drafted tokens over a cache ("Inside the
// inference engine: model architectures and forward pass", section "KV Cache:
// memory for causal attention"; the mask of a node is its sequence's earlier
// cells and the path to it): for row t of tree i and query head h
//   o[t][h] = softmax_c(q[t][h] . K[c] / sqrt(hd)) V[c]
// over the cells c < base[i] (with a window those c > pos[t] - window) and the
// cells base[i] + j whose bit j of mask[t] is set.  A row that sees nothing is zero; one
// that sees scores of -inf alone is NaN.
//
// The rows of a tree that share a kv head, its nodes times the query heads of the
// group, see the same earlier cells: 128 of them are one tile of tcgen05.mma, which
// reads each K and V tile of 128 keys once for all of them.  The keys are split over
// the CTAs of a cluster, and where there are still SMs left over several clusters.
//
// Precision.  q, K and V are fp16 (an E4M3 value is one exactly); a weight
// p = 2^((s - z) c + x), the exponent in fp32 with one rounding, enters O as two fp16
// numbers of 22 bits together (below 2^-3, where the low one has no full 11, to 2^-24).
// Rounded to one, o is off by 1.4 times its own rounding.
// z and x are a row's reference, raised, with O rescaled, only when a tile passes it by
// 2^8.  Usually z is 0 and x a whole number, so that changing it is exact: 7 (weights far
// below the largest stay normal fp16 numbers) less the row's largest s c so far, rounded
// up.  From 2^22 on, where steps of fp32 would come to swallow the 7 and the row's
// weights with it, z is the largest score so far and x is 7; a tile's scores are brought to
// s - z in the branch that raises references, which other rows seldom take.  So a row's
// largest weight lies in [2^6, 2^15] whatever its scores, and its weights have 22 bits down
// to 2^-9 of that, and 2^-30 of it below.
//
// A CTA: warps 0-7 softmax (two threads a row, 64 keys each), 8 issues S = q K^T, 9
// O += P V, 10 brings K and 11 V by TMA, of an E4M3 cache to warps 12-15 and 16-19, which
// widen them.
// Tensor memory: three S buffers of 128 columns, P in the place of the S it came
// from (of each 32 columns 16 of high pairs, 16 of low pairs), O.
//
// Joining: a CTA sends its rows of O, their references and sums to the ranks that own
// them (rows / cluster size each), one cluster barrier later every rank joins its
// rows.  With several clusters a rank leaves its rows in memory and the last one to
// come joins them, in the clusters' order whichever it is.  (Sent by the copy engine
// the rows take half as long, but have to be laid down first: no gain.)
//
// Cells that a row does not see may hold anything: a masked score is replaced, and
// in tiles that not every row sees whole, V is read over before its product: rows
// outside the tree's cells become zero, and a value that is not finite makes the
// rows that see its cell NaN and is zero for the others.
//
// What bounds it: not memory (64 nodes of 32000 cells, 8 kv heads of 128: 51 us, 2.6 TB/s)
// nor the tensor pipe, but the chain of a tile, which one row tile an SM cannot overlap
// with another's: S, its maximum, 2^x and the split (10.6 cycles a warp and score), P V
// take 1.2 us for 128 keys, before them 8 us to start and after them 6 us to join.
// Left out to see, the low products, the loads or the exponentials change it little.
//
// Every mbarrier wait is bounded; on a timeout the CTA raises ERRF_WAIT_TIMEOUT,
// waits (bounded) for its own copies in flight, takes part in the cluster's barriers
// and frees its tensor memory.  The shared memory of a CTA leaves no room for another
// that allocates tensor memory, so the allocation never waits.
#include <cuda.h>

#include "attn_tc.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "tma.cuh"

namespace llm {

namespace {

using tcg::sdesc;
using tcg::tc_fence_after;
using tcg::tc_fence_before;
using tcg::tmem_ld32;
using namespace tca;

constexpr float LIFT = 7.f;                  // a row's largest weight is at least 2^(LIFT - 1), and
constexpr float MOST = LIFT + 8.f;           // at most 2^MOST
constexpr float FAR = 4194304.f;             // s c from which on a reference is a score (whole numbers are exact up to 2^24)
constexpr float NONE = 1e30f;                // x of a row without a reference, which is below every other
constexpr int BQ = 128, BKEY = 128;
constexpr int SM_WARPS = 8, PARTS = 2, S_WARP = 8, PV_WARP = 9, K_WARP = 10, V_WARP = 11, W_WARP = 12, W_WARPS = 8;
constexpr int threads(bool f8) { return (W_WARP + (f8 ? W_WARPS : 0)) * 32; }
// Registers of a thread of the E4M3 kernel: at its launch, of the softmax (which at 96 spills a row's scores:
// 16 nodes of 32000 cells 48.5 us, not 33.6), the widening and the issuers.  256 x 128 + 256 x 72 + 128 x 80 = 640 x 96.
// With four widening warps and 128 registers for all the case takes 34.1 us.
constexpr int L_REGS = 96, SM_REGS = 128, W_REGS = 72, I_REGS = 80;
static_assert(SM_WARPS * SM_REGS + W_WARPS * W_REGS + (W_WARP - S_WARP) * I_REGS <= threads(true) / 32 * L_REGS, "registers");
constexpr uint32_t BOX = 128 * 128;          // bytes of one 128-row x 64-column fp16 box
constexpr int NS = 3;                        // S buffers
constexpr uint32_t TMEM_COLS = 512;          // S_b / P_b [128 b, 128 b + 128), O [384, 384 + HD)
constexpr int MAX_CLUSTER = 8;
constexpr int SLOTS = 64;                    // (group, cluster) results that go through memory
constexpr int COUNTERS = 1024;

// HD: head_dim as the tiles hold it (head_dim 32: 64, the rest zeros).
template <int HD, bool F8>
struct Cfg {
    static constexpr int NBX = HD / 64;                         // 64-column boxes of a row
    static constexpr int ST = HD == 128 ? 2 : F8 ? 4 : 5;       // stages of each ring
    static constexpr int RAWS = HD == 128 ? 2 : 4;              // E4M3 tiles of K, and of V, on their way
    static constexpr uint32_t TILE = NBX * BOX, RAW = BKEY * HD;
    static constexpr uint32_t K_OFF = TILE;
    static constexpr uint32_t V_OFF = K_OFF + ST * TILE;
    // rows of O from the other ranks; before them, once every rank has read its own, the E4M3 tiles
    static constexpr uint32_t RECV_OFF = V_OFF + ST * TILE;
    static constexpr uint32_t RECV = BQ * HD * 4 / MAX_CLUSTER * (MAX_CLUSTER - 1);
    static constexpr uint32_t ML_OFF = RECV_OFF + RECV;         // their references and sums [rank][row][4]
    static constexpr uint32_t RECV_END = ML_OFF + BQ * 16, RAW_END = RECV_OFF + (F8 ? 2 * RAWS * RAW : 0);
    static constexpr uint32_t X_OFF = RECV_END > RAW_END ? RECV_END : RAW_END;      // the exchange of a row's parts [2][part][row]
    static constexpr uint32_t BAR_OFF = X_OFF + 2 * PARTS * BQ * 4;
    static constexpr uint32_t MISC_OFF = BAR_OFF + 512;
    static constexpr size_t SMEM = MISC_OFF + 128;
    static constexpr uint32_t O_COL = NS * BKEY;
    // kind::f16 instruction descriptors: D fp32 (bit 4), A and B fp16, M = 128
    // (M >> 4 at bit 24), N >> 3 at bit 17; bit 16 marks B as MN-major
    static constexpr uint32_t IDESC_S = (1u << 4) | ((uint32_t)(BKEY >> 3) << 17) | ((uint32_t)(BQ >> 4) << 24);
    static constexpr uint32_t IDESC_O =
        (1u << 4) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | ((uint32_t)(BQ >> 4) << 24);
    // barriers, in units of eight bytes
    static constexpr int B_Q = 0, B_ASKED = 1, B_S_FULL = 2, B_P_FULL = B_S_FULL + NS, B_PV_DONE = B_P_FULL + NS,
                         B_K_FULL = B_PV_DONE + NS, B_K_EMPTY = B_K_FULL + ST, B_V_FULL = B_K_EMPTY + ST,
                         B_V_EMPTY = B_V_FULL + ST, B_RAW_FULL = B_V_EMPTY + ST, B_RAW_EMPTY = B_RAW_FULL + 2 * RAWS,
                         B_COUNT = B_RAW_EMPTY + 2 * RAWS;
    static_assert(8 * B_COUNT <= 512, "barriers");
    // more than half of an SM's shared memory, and so much that no other kernel with tensor memory fits beside
    static_assert(SMEM <= 227 * 1024 && SMEM >= 190 * 1024, "one CTA an SM");
};

// Shared words behind the barriers.
struct Misc {
    int abort;
    uint32_t tmem;
    int lo_min, lo_max;                       // the rows' first visible cells
    int base, end;                            // the tree's (of one that does not fit 0)
    uint32_t bad[3][4];                       // keys of a tile whose V is not finite, three tiles in turn
    int last;
};
static_assert(sizeof(Misc) <= 128, "shared words");

// Loads and stores of 32 columns of tensor memory that are waited for together.
__device__ __forceinline__ void tmem_ask32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// ... the wait, which the registers asked for pass through
__device__ __forceinline__ void tmem_come32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}
__device__ __forceinline__ void tmem_put32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
           "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
           "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
           "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_put_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(is));
    return is != 0;
}
// A whole warp's bounded wait.  Most of them find the phase over: one look and a vote, with the loop out of the way,
// save 0.08 us a tile (64 nodes of 32000 cells 55.1 -> 52.5 us).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *err) {
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), 1)) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
}
__device__ __forceinline__ void st_shared(uint32_t at, const uint4 &v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
// Through L2, where it stands among the asynchronous copies' issues.
__device__ __forceinline__ uint4 ld_global(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
// A 16-byte chunk of a row of a box, as TMA's 128-byte swizzle places it.
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int row, int chunk) {
    return tile + (uint32_t)(chunk >> 3) * BOX + (uint32_t)row * 128u + (uint32_t)(((chunk & 7) ^ (row & 7)) << 4);
}
// Two floats in one register pair, for the packed forms of add and fma.
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
    unsigned long long v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
// Two weights as hi and lo fp16 pairs: the low 13 mantissa bits are split off exactly.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    const uint32_t ah = __float_as_uint(a) & 0xFFFFE000u, bh = __float_as_uint(b) & 0xFFFFE000u;
    hi = pack_h2(__uint_as_float(ah), __uint_as_float(bh));
    const float2 l = unpack2(fma2(pack2(__uint_as_float(ah), __uint_as_float(bh)), pack2(-1.f, -1.f), pack2(a, b)));
    lo = pack_h2(l.x, l.y);
}
__device__ __forceinline__ bool not_finite(uint32_t h2) {
    return (h2 & 0x7C00u) == 0x7C00u || (h2 & 0x7C000000u) == 0x7C000000u;
}

// The tree of a group of rows and what of it lies in the call and the cache.
struct Tree {
    int r0, n, seq, base;                     // n: nodes whose rows are written
    bool ok;
    __device__ __forceinline__ Tree(const AttnTreeArgs &a, int i) {
        r0 = a.row0[i];
        n = a.row0[i + 1] - r0;
        seq = a.seq[i];
        base = a.base[i];
        ok = r0 >= 0 && n >= 0 && n <= a.max_nodes && r0 <= a.T - n && seq >= 0 && seq < a.kv.n_seq && base >= 0 &&
             base <= a.kv.n_ctx - n;
        n = min(max(n, 0), a.max_nodes);
    }
};

// A row's reference: weights are 2^((s - z) c + x).
struct Ref { float z, x; };
// The exponent of the factor that takes sums from one reference to another: of usual ones the difference of x exactly, else with
// one rounding.
__device__ __forceinline__ float shift(const Ref &from, const Ref &to, float c) { return fmaf(from.z - to.z, c, to.x - from.x); }

// Joined, references are pairs of floats R + R2, R2 zero but for scores; the highest has the largest R, and of those the
// largest R2.
template <typename Of>
__device__ __forceinline__ float rest_of(float M, int n, Of &&of) {
    float M2 = -INFINITY;
#pragma unroll 1
    for (int s = 0; s < n; ++s) {
        const float4 v = of(s);
        if (v.x == M) M2 = fmaxf(M2, v.z);
    }
    return M2;
}
// The factor from one to another.  R - M is exact where that matters, within a factor of two.
__device__ __forceinline__ float moved(float R, float R2, float M, float M2) { return ex2((R - M) + (R2 - M2)); }

// Which of the keys k0 .. k0 + 31 a row sees: those from lo to base, and by the bits
// of its mask those from base to end.
__device__ __forceinline__ uint32_t visible(int k0, int lo, int base, int end, const uint32_t *mask, int words) {
    uint32_t v = 0;
    const int a0 = max(lo - k0, 0), a1 = min(base - k0, 32);
    if (a1 > a0) v = (~0u >> (32 - (a1 - a0))) << a0;
    const int j0 = k0 - base, nb = min(end - k0, 32);
    if (j0 > -32 && nb > 0) {
        const int i0 = j0 >> 5;
        auto word = [&](int i) { return i >= 0 && i < words ? __ldcg(mask + i) : 0u; };
        v |= __funnelshift_r(word(i0), word(i0 + 1), j0 & 31) & (~0u >> (32 - nb));
    }
    return v;
}

// An E4M3 tile of 128 rows as fp16, by half of the widening warps (ww among them): 16 elements of a row at a time, eight lanes
// at once four pieces each of rows r and r ^ 5, whose chunks lie in different banks where they
// are read (rows of 128 bytes swizzled by TMA, shorter ones as they are) and where they are written.
template <int HD, bool F8>
__device__ __forceinline__ void widen_tile(uint32_t raw, int hd, uint32_t tile, int ww, int lane) {
    constexpr int NBX = Cfg<HD, F8>::NBX;
    const int r8 = (lane >> 3) ^ (lane & 4 ? 5 : 0), piece = lane & 3;
    auto row_of = [&](int i) { return ww * (BKEY / (W_WARPS / 2)) + i / NBX * 8 + r8; };
    constexpr int N = 2 * NBX;                           // pieces in flight
#pragma unroll
    for (int i0 = 0; i0 < BKEY / (W_WARPS / 2) / 8 * NBX; i0 += N) {
        uint4 x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = row_of(i0 + i), at = (i0 + i) % NBX * 4 + piece;      // 16-byte chunk of the raw row
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (NBX == 2) x[i] = ld_shared(raw + (uint32_t)row * 128u + (uint32_t)((at ^ (row & 7)) << 4));
            else if (16 * at < hd) x[i] = ld_shared(raw + (uint32_t)(row * hd + 16 * at));
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[2 * j] = e4m3x2_to_h2((uint16_t)w[j]);
                h[2 * j + 1] = e4m3x2_to_h2((uint16_t)(w[j] >> 16));
            }
            const int row = row_of(i0 + i), c = (i0 + i) % NBX * 8 + piece * 2;
            st_shared(chunk_at(tile, row, c), make_uint4(h[0], h[1], h[2], h[3]));
            st_shared(chunk_at(tile, row, c + 1), make_uint4(h[4], h[5], h[6], h[7]));
        }
    }
}

// grid (splits, (tree, kv head, row tile)); the splits are clusters of `cs` CTAs.
template <int HD, bool F8>
__global__ void __launch_bounds__(threads(F8), 1)
attn_tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnTreeArgs a,
                 const int row_tiles, const int cs) {
    using C = Cfg<HD, F8>;
    constexpr int NBX = C::NBX, ST = C::ST;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base_sm = smem_u32(smem_raw);
    Misc &misc = *reinterpret_cast<Misc *>(smem_raw + C::MISC_OFF);
    float *const xch = reinterpret_cast<float *>(smem_raw + C::X_OFF);
    float4 *const ml = reinterpret_cast<float4 *>(smem_raw + C::ML_OFF);        // R, sum, R2
    const uint32_t bar = base_sm + C::BAR_OFF;
    auto s_full = [&](int b) { return bar + 8u * (C::B_S_FULL + b); };
    auto p_full = [&](int b) { return bar + 8u * (C::B_P_FULL + b); };        // P_t written
    auto pv_done = [&](int b) { return bar + 8u * (C::B_PV_DONE + b); };      // O += P_t V_t done
    auto k_full = [&](int s) { return bar + 8u * (C::B_K_FULL + s); };
    auto k_empty = [&](int s) { return bar + 8u * (C::B_K_EMPTY + s); };
    auto v_full = [&](int s) { return bar + 8u * (C::B_V_FULL + s); };
    auto v_empty = [&](int s) { return bar + 8u * (C::B_V_EMPTY + s); };
    auto raw_full = [&](int s) { return bar + 8u * (C::B_RAW_FULL + s); };
    auto raw_empty = [&](int s) { return bar + 8u * (C::B_RAW_EMPTY + s); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &misc.abort;

    if (!F8) cluster_arrive_relaxed();                   // started: the others may write here once they have waited
    pdl_wait();
    pdl_trigger();
    const int hd = a.kv.head_dim, Hkv = a.kv.n_kv_head, G = a.H / Hkv;
    const int group = blockIdx.y, mt = group % row_tiles, j = group / row_tiles % Hkv;
    const Tree tr(a, group / row_tiles / Hkv);           // on its way while the barriers are made
    if (warp == K_WARP) {
        for (int i = lane; i < C::B_COUNT; i += 32) {
            const bool of_softmax = i == C::B_Q || i == C::B_ASKED || (i >= C::B_P_FULL && i < C::B_PV_DONE);
            const bool of_widening = F8 && ((i >= C::B_K_FULL && i < C::B_K_EMPTY) || (i >= C::B_V_FULL && i < C::B_V_EMPTY) || i >= C::B_RAW_EMPTY);
            mbar_init(bar + 8u * i, of_softmax ? SM_WARPS : of_widening ? W_WARPS / 2 : 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (lane < 2) asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(lane ? &tmV : &tmK)) : "memory");
    } else if (warp == S_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&misc.tmem)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (tid == 0) {
        misc.abort = 0;
        misc.lo_min = a.kv.n_ctx;
        misc.lo_max = 0;
        misc.base = tr.ok ? tr.base : 0;
        misc.end = tr.ok ? tr.base + tr.n : 0;
        for (int i = 0; i < 12; ++i) misc.bad[i / 4][i % 4] = 0u;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc.tmem;

    const int rows = min(max(tr.n * G - mt * BQ, 0), BQ);          // rows of this tile
    const int base = tr.base, end = tr.base + tr.n;
    if (!tr.ok && mt == 0 && j == 0 && blockIdx.x == 0 && tid == 0) raise_error(a.err, ERRF_BAD_INDEX);
    // thread r (and r + 128) of the softmax has row r: query head j G + g of node `node`
    const int r = tid & (BQ - 1), node = (mt * BQ + r) / G, g = (mt * BQ + r) - node * G;
    const bool row_ok = r < rows && tr.ok;
    int lo = 0, lo_min = 0, lo_max = 0;
    if (a.window > 0) {
        if (warp < 4 && row_ok) {
            const int pos = a.pos[tr.r0 + node];          // any number
            lo = pos >= a.window ? min(pos - a.window + 1, base) : 0;
            atomicMin(&misc.lo_min, lo);
            atomicMax(&misc.lo_max, lo);
            xch[r] = __int_as_float(lo);
        }
        __syncthreads();
        lo_min = misc.lo_min;
        lo_max = misc.lo_max;
        lo = __float_as_int(xch[r]);
        __syncthreads();
    }
    // this CTA's tiles of 128 keys
    const int first = lo_min / BKEY, all = tr.ok && rows > 0 ? (end + BKEY - 1) / BKEY - first : 0;
    const int S = gridDim.x, split = blockIdx.x;
    const int kt0 = first + (int)((long long)all * split / S), nt = first + (int)((long long)all * (split + 1) / S) - kt0;

    const float c = 1.4426950408889634f / sqrtf((float)hd);       // scores to exponents of two
    Ref ref{0.f, NONE};
    float l_row = -1.f;                                  // no sums
    bool have = false;                                   // O holds this CTA's sums
    if constexpr (F8) {
        // no warp waits for another before its own of these three, so the softmax's does end
        if (warp < SM_WARPS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(SM_REGS));
        else if (warp < W_WARP) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(I_REGS));
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(W_REGS));
    }
    if (nt == 0) {
        // nothing to do: on to the joining
    } else if (warp < SM_WARPS) {
        constexpr int HK = BKEY / PARTS, QC = HD / 8 / PARTS;      // keys of a part; 16-byte chunks of a row's q or a key's V
        const int quarter = warp & 3, part = warp >> 2;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t o_col = C::O_COL + part * (HD / 2);   // the part's O columns
        const bool active = quarter * 32 < rows;             // the warp's lanes hold rows
        // q: this part's chunks of the row (rows past the last are zero), asked for ahead of K and V, behind which it
        // would queue for microseconds
        {
            const f16 *src = a.q + ((size_t)(tr.r0 + node) * a.H + (size_t)j * G + g) * hd;
            uint4 x[QC];
#pragma unroll
            for (int i = 0; i < QC; ++i) {
                const int c = part * QC + i;
                x[i] = make_uint4(0u, 0u, 0u, 0u);
                if (row_ok && 8 * c < hd) x[i] = ld_global(reinterpret_cast<const uint4 *>(src) + c);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + 8u * C::B_ASKED);
#pragma unroll
            for (int i = 0; i < QC; ++i) st_shared(chunk_at(base_sm, r, part * QC + i), x[i]);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + 8u * C::B_Q);
        }
        // a row's two values, this part's among them; two buffers in turn, so that a part one tile ahead does not
        // overwrite what the others have not read
        auto post = [&](int turn, float v) { xch[((turn & 1) * PARTS + part) * BQ + r] = v; };
        auto collect = [&](int turn, float (&both)[PARTS]) {
            named_sync(1 + quarter, PARTS * 32);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) both[i] = xch[((turn & 1) * PARTS + i) * BQ + r];
        };
        // ok stays uniform over each warp, and every softmax thread runs all nt
        // iterations, so the named barriers (which have no time limit) are always
        // reached by all their threads; after a timeout the iterations only pass them
        bool ok = true;
        int edges = 0;
        const int whole_from = (lo_max + BKEY - 1) / BKEY - kt0, whole_to = base / BKEY - kt0;      // tiles that every row sees whole
        float l_run = 0.f, both[PARTS];
        int b = 0, round = 0;                                // t % NS, t / NS
        for (int t = 0; t < nt; ++t, b = b + 1 == NS ? 0 : b + 1, round += b == 0) {
            const int tile0 = (kt0 + t) * BKEY;
            const uint32_t s_col = lane_base + b * BKEY + part * HK;
            const bool edge = t >= whole_to || t < whole_from;       // not every row sees the whole tile
            uint32_t vis[2] = {~0u, ~0u}, nan[2] = {0u, 0u};
            if (edge) {
                const volatile Misc &now = misc;             // held through the loop they spill: ragged trees 23.1 us, not 22.4
                const int base = now.base, end = now.end;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    vis[q] = row_ok ? visible(tile0 + part * HK + 32 * q, lo, base, end, a.mask + (size_t)(tr.r0 + node) * a.words, a.words) : 0u;
                // two threads a key read over its V
                const int sl = t % ST, key = tid >> 1, at = (tid & 1) * QC;
                // the softmax may be ahead of V by more than its ring: the stage's tile before must have landed, or this
                // wait would take the one before that for its own
                if (ST <= NS && t >= ST) ok = ok && warp_wait(pv_done((t - ST) % NS), (t - ST) / NS & 1, abort, a.err);
                ok = ok && warp_wait(v_full(sl), t / ST & 1, abort, a.err);
                if (ok) {
                    const bool in = tile0 + key >= lo_min && tile0 + key < end;
                    const uint32_t tile = base_sm + C::V_OFF + sl * C::TILE;
                    bool odd = false;
#pragma unroll
                    for (int i = 0; i < QC; ++i) {
                        const uint4 x = ld_shared(chunk_at(tile, key, at + i));
                        odd |= not_finite(x.x) || not_finite(x.y) || not_finite(x.z) || not_finite(x.w);
                    }
                    if (!in || odd) {
#pragma unroll
                        for (int i = 0; i < QC; ++i) st_shared(chunk_at(tile, key, at + i), make_uint4(0u, 0u, 0u, 0u));
                        if (in) atomicOr(&misc.bad[edges % 3][key >> 5], 1u << (key & 31));
                    }
                    fence_proxy_async();
                }
                named_sync(5, SM_WARPS * 32);
#pragma unroll
                for (int q = 0; q < 2; ++q) nan[q] = vis[q] & misc.bad[edges % 3][2 * part + q];
                // the set of the tile before has been read by all, and serves the tile after the next
                if (tid < 4) misc.bad[(edges + 2) % 3][tid] = 0u;
                ++edges;
            }
            ok = ok && warp_wait(s_full(b), round & 1, abort, a.err);
            if (active) {
                uint32_t v[2][32];
                float mx = -INFINITY;
                if (ok) {
                    tc_fence_after();
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};      // the part's maximum as a tree of four chains
#pragma unroll
                    for (int q = 0; q < 2; ++q) tmem_ask32(s_col + 32 * q, v[q]);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        tmem_come32(v[q]);
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(vis[q] >> i & 1)) v[q][i] = 0xFF800000u;
                            if (nan[q]) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (nan[q] >> i & 1) v[q][i] = 0x7FFFFFFFu;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(v[q][i]));
                    }
                    mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                }
                post(t, mx);
                collect(t, both);
                mx = fmaxf(both[0], both[1]);
                const bool raise = ok && mx != -INFINITY && !(fmaf(mx - ref.z, c, ref.x) <= MOST);
                if (__any_sync(0xffffffffu, raise || ref.z != 0.f)) {
                    float factor = 1.f;
                    if (raise) {
                        const float top = __fmul_ru(mx, c);
                        const bool score = fabsf(top) >= FAR && top < INFINITY;
                        const Ref to{score ? mx : 0.f, score ? LIFT : LIFT - ceilf(top)};
                        factor = ex2(shift(ref, to, c));
                        ref = to;
                    }
                    l_run *= factor;
                    // a raised reference rescales O, which P_{t-1} V_{t-1} must have finished
                    if (t >= 1) {
                        ok = warp_wait(pv_done(b == 0 ? NS - 1 : b - 1), (b == 0 ? round - 1 : round) & 1, abort, a.err);
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; ok && q < HD / 64; ++q) {
                            uint32_t o[32];
                            tmem_ld32(lane_base + o_col + 32 * q, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
                            tmem_st32(lane_base + o_col + 32 * q, o);
                        }
                    }
                    if (__any_sync(0xffffffffu, ref.z != 0.f)) {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[q][i] = __float_as_uint(__uint_as_float(v[q][i]) - ref.z);
                    }
                }
                if (ok) {
                    // the part's weights over the columns of S they came from: 16 of hi pairs, 16 of lo pairs
                    const unsigned long long c2 = pack2(c, c), x2 = pack2(ref.x, ref.x);
                    unsigned long long rs[2] = {0ull, 0ull};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t p[32];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 x = unpack2(fma2(pack2(__uint_as_float(v[q][2 * i]), __uint_as_float(v[q][2 * i + 1])), c2, x2));
                            const float p0 = ex2(x.x), p1 = ex2(x.y);
                            rs[i & 1] = add2(rs[i & 1], pack2(p0, p1));
                            split_pair(p0, p1, p[i], p[16 + i]);
                        }
                        tmem_put32(s_col + 32 * q, p);
                    }
                    tmem_put_done();
                    const float2 sum = unpack2(add2(rs[0], rs[1]));
                    l_run += sum.x + sum.y;
                    tc_fence_before();
                }
            }
            // (the weights of rows that do not exist are whatever S is)
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(p_full(b));
        }
        if (active) {
            post(nt, l_run);
            collect(nt, both);
            l_row = both[0] + both[1];
        }
        have = ok && warp_wait(pv_done((nt - 1) % NS), (nt - 1) / NS & 1, abort, a.err);
        tc_fence_after();
    } else if (warp == K_WARP || warp == V_WARP) {
        // ---- K or V tiles (of an E4M3 cache on their way to the widening), once q has been asked for
        if (lane == 0) {
            const bool k = warp == K_WARP;
            const int row = (int)(a.map_row0 + (long long)tr.seq * (a.kv.seq_stride / hd) + (long long)j * a.kv.n_ctx) + kt0 * BKEY;
            constexpr int N = F8 ? C::RAWS : ST;
            constexpr uint32_t BYTES = F8 ? C::RAW : C::TILE;
            const uint32_t ring = base_sm + (F8 ? C::RECV_OFF + (k ? 0 : N * BYTES) : k ? C::K_OFF : C::V_OFF);
            const uint32_t full = F8 ? raw_full(k ? 0 : N) : k ? k_full(0) : v_full(0), empty = F8 ? raw_empty(k ? 0 : N) : k ? k_empty(0) : v_empty(0);
            const bool ok = mbar_wait(bar + 8u * C::B_ASKED, 0, abort, a.err);
            int sent = 0;
            for (; ok && sent < nt; ++sent) {
                const int sl = sent % N, use = sent / N;
                if (use > 0 && !mbar_wait(empty + 8u * sl, (use - 1) & 1, abort, a.err)) break;
                mbar_expect_tx(full + 8u * sl, F8 ? (uint32_t)(BKEY * hd) : BYTES);
                for (int i = 0; i < (F8 ? 1 : NBX); ++i)
                    tma_load_2d(ring + sl * BYTES + i * BOX, k ? &tmK : &tmV, full + 8u * sl, i * 64, row + sent * BKEY);
            }
            // after a timeout: wait (bounded) for the copies in flight before the memory is released
            if (*abort)
                for (int u = max(sent - N, 0); u < sent; ++u)
                    for (uint32_t i = 0; i < WAIT_LIMIT && !mbar_try_wait(full + 8u * (u % N), u / N & 1); ++i) {
                    }
        }
    } else if (F8 && warp >= W_WARP) {
        // ---- widening, K by the first half of the warps and V by the second (all of them in turn were 8% slower),
        // each with a ring of its own, so that none waits for a phase it may be two behind
        const int ww = (warp - W_WARP) % (W_WARPS / 2);
        const bool k = warp < W_WARP + W_WARPS / 2;
        const uint32_t raws = base_sm + C::RECV_OFF + (k ? 0 : C::RAWS * C::RAW), tiles = base_sm + (k ? C::K_OFF : C::V_OFF);
        for (int t = 0; t < nt; ++t) {
            const int sl = t % ST, rs = t % C::RAWS, ring = (k ? 0 : C::RAWS) + rs;
            if (!warp_wait(raw_full(ring), t / C::RAWS & 1, abort, a.err)) break;
            if (t >= ST && !warp_wait(k ? k_empty(sl) : v_empty(sl), (t / ST - 1) & 1, abort, a.err)) break;
            widen_tile<HD, F8>(raws + rs * C::RAW, hd, tiles + sl * C::TILE, ww, lane);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(k ? k_full(sl) : v_full(sl));
                mbar_arrive(raw_empty(ring));
            }
        }
    } else if (warp == S_WARP) {
        // ---- S_t = q K_t^T into buffer t % NS, once the P that took the place of the S before has been read.  The whole
        // warp walks the loop, so that addresses and descriptors stay uniform; the elected lane issues.
        const bool leader = elect_one();
        bool ok = warp_wait(bar + 8u * C::B_Q, 0, abort, a.err);
        const uint64_t q_desc = sdesc(base_sm), k_desc = sdesc(base_sm + C::K_OFF);
        for (int t = 0; ok && t < nt; ++t) {
            const int b = t % NS, sl = t % ST;
            if (!warp_wait(k_full(sl), t / ST & 1, abort, a.err)) break;
            if (t >= NS && !warp_wait(pv_done(b), (t / NS - 1) & 1, abort, a.err)) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int f = 0; f < NBX; ++f) {
                    const uint64_t qd = q_desc + (uint32_t)f * (BOX >> 4), kd = k_desc + (uint32_t)sl * (C::TILE >> 4) + (uint32_t)f * (BOX >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) mma1(tmem + b * BKEY, qd + 2 * kk, kd + 2 * kk, C::IDESC_S, (f | kk) != 0);
                }
                commit1(k_empty(sl));
                commit1(s_full(b));
            }
            __syncwarp();
        }
    } else if (warp == PV_WARP) {
        // ---- O (+)= P_t V_t once the softmax has written P_t (and rescaled O)
        const bool leader = elect_one();
        const uint32_t o_acc = tmem + C::O_COL;
        const uint64_t v_desc = sdesc_mn(base_sm + C::V_OFF, BOX);
        for (int t = 0; t < nt; ++t) {
            const int b = t % NS, sl = t % ST;
            if (!warp_wait(v_full(sl), t / ST & 1, abort, a.err)) break;
            if (!warp_wait(p_full(b), t / NS & 1, abort, a.err)) break;
            tc_fence_after();
            if (leader) {
                const uint64_t vd = v_desc + (uint32_t)sl * (C::TILE >> 4);
#pragma unroll
                for (int kk = 0; kk < BKEY / 16; ++kk) {
                    // 16 keys: 8 columns of P's hi pairs, 16 on their lo pairs, among the 32 of their 32 keys
                    const uint32_t p = tmem + b * BKEY + kk / 2 * 32 + kk % 2 * 8;
                    mma1_ts(o_acc, p, vd + kk * (2048 >> 4), C::IDESC_O, (t | kk) != 0);
                    mma1_ts(o_acc, p + 16, vd + kk * (2048 >> 4), C::IDESC_O, 1);
                }
                commit1(v_empty(sl));
                commit1(pv_done(b));
            }
            __syncwarp();
        }
    }

    __syncwarp();
    // ---- joining.  Row r belongs to rank r / share; what it is sent lies in its shared memory, its own part over
    // its K tiles, which all products have read.
    const int rank = cs > 1 ? (int)cluster_rank() : 0, share = max((rows + cs - 1) / cs, 1);
    if constexpr (F8) {
        // Back to the registers of the launch, for what follows is every warp's.  The others take theirs only after the
        // softmax has taken and returned its own: before, theirs could be the ones that it waits for.
        if (warp < SM_WARPS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(L_REGS));
        __syncthreads();                                 // the E4M3 tiles have been read (and, after a timeout, have come)
        if (warp >= SM_WARPS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(L_REGS));
        cluster_arrive();
    }
    cluster_wait();                                      // the others' memory may be written
    auto part_at = [&](int of, int to) {                 // where rank `to` has the rows of rank `of`
        return of == to ? C::K_OFF : C::RECV_OFF + (uint32_t)((of < to ? of : of - 1) * share) * (HD * 4);
    };
    if (warp < 4 && r < rows) {
        const int to = r / share, at = r - to * share;
        const float R = ref.z == 0.f ? -ref.x : __fmul_rn(ref.z, c), R2 = ref.z == 0.f ? 0.f : fmaf(ref.z, c, -R) - ref.x;
        dsmem_st_f32x4(dsmem(ml + rank * share + at, to), make_float4(R, l_row, R2, 0.f));
    }
    if (warp < SM_WARPS && (warp & 3) * 32 < rows && have) {       // whole warps, as tensor memory is read
        const int part = warp >> 2, to = min(r / share, cs - 1), at = r - to * share;
        const uint32_t dst = dsmem(smem_raw + part_at(rank, to), to) + (uint32_t)at * (HD * 4);
#pragma unroll 1
        for (int q = 0; q < HD / 64; ++q) {
            uint32_t v[32];
            tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::O_COL + part * (HD / 2) + q * 32, v);
            if (r < rows && part * (HD / 2) < hd) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int chunk = part * (HD / 8) + q * 8 + i;
                    dsmem_st_f32x4(dst + (uint32_t)((chunk ^ (at & 7)) << 4),
                                   make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                                               __uint_as_float(v[4 * i + 3])));
                }
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (warp == S_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(TMEM_COLS) : "memory");
    }

    const int my_rows = min(share, rows - rank * share), per = hd / 4, clusters = S / cs, mine = split / cs;
    unsigned *const counters = reinterpret_cast<unsigned *>(a.scratch);
    float *const slots = reinterpret_cast<float *>(counters + COUNTERS);
    auto slot_o = [&](int ci, int row) { return slots + ((size_t)(group * clusters + ci) * BQ + row) * (HD + 4); };
    auto store = [&](int row, int chunk, const float4 &v) {
        const int at = mt * BQ + row, nd = at / G, t = tr.r0 + nd;
        if (t >= 0 && t < a.T)
            *reinterpret_cast<uint2 *>(a.o + ((size_t)t * a.H + (size_t)j * G + (at - nd * G)) * hd + 4 * chunk) =
                make_uint2(pack_h2(v.x, v.y), pack_h2(v.z, v.w));
    };
    // what a row without weights has: zeros, or NaN if it sees cells and all their scores are -inf
    auto empty = [&](int row) {
        const volatile Misc &now = misc;
        const int t = tr.r0 + (mt * BQ + row) / G, base = now.base, n = now.end - base, pos = a.window > 0 && base > 0 ? a.pos[t] : 0;
        bool sees = base > 0 && (pos < a.window || pos - a.window + 1 < base || a.window == 0);
#pragma unroll 1
        for (int w = 0; 32 * w < n; ++w) sees |= (__ldcg(a.mask + (size_t)t * a.words + w) & (~0u >> max(32 - (n - 32 * w), 0))) != 0u;
        return sees ? __int_as_float(0x7FFFFFFF) : 0.f;
    };
    for (int i = tid; i < my_rows * per; i += threads(F8)) {
        const int at = i / per, chunk = i - at * per;
        float M = -INFINITY, M2 = 0.f, L = 0.f;
        for (int s = 0; s < cs; ++s) M = fmaxf(M, ml[s * share + at].x);
        if (__builtin_expect(fabsf(M) >= FAR / 2, 0)) M2 = rest_of(M, cs, [&](int s) { return ml[s * share + at]; });
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < cs; ++s) {
            const float4 v = ml[s * share + at];
            if (v.y < 0.f) continue;                     // that rank has no sums
            const float f = moved(v.x, v.z, M, M2);
            const float4 x = *reinterpret_cast<const float4 *>(smem_raw + part_at(s, rank) + (uint32_t)at * (HD * 4) + ((chunk ^ (at & 7)) << 4));
            L = fmaf(f, v.y, L);
            o.x = fmaf(f, x.x, o.x); o.y = fmaf(f, x.y, o.y); o.z = fmaf(f, x.z, o.z); o.w = fmaf(f, x.w, o.w);
        }
        const int row = rank * share + at;
        if (clusters == 1) {
            const float inv = L == 0.f ? empty(row) : 1.f / L;
            store(row, chunk, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        } else {
            float *dst = slot_o(mine, row);
            __stcg(reinterpret_cast<float4 *>(dst) + chunk, o);
            if (chunk == 0) __stcg(reinterpret_cast<float4 *>(dst + HD), make_float4(M, L, M2, 0.f));
        }
    }
    if (clusters == 1) return;
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        unsigned *cnt = counters + group * cs + rank;
        const bool last = atomicAdd(cnt, 1u) == (unsigned)clusters - 1;
        if (last) *cnt = 0u;                             // ready for the next call
        __threadfence();
        misc.last = last;
    }
    __syncthreads();
    if (!misc.last) return;
    for (int i = tid; i < my_rows * per; i += threads(F8)) {
        const int at = i / per, chunk = i - at * per, row = rank * share + at;
        auto sums = [&](int s) { return __ldcg(reinterpret_cast<const float4 *>(slot_o(s, row) + HD)); };
        float M = -INFINITY, M2 = 0.f, L = 0.f;
        for (int s = 0; s < clusters; ++s) M = fmaxf(M, __ldcg(slot_o(s, row) + HD));
        if (__builtin_expect(fabsf(M) >= FAR / 2, 0)) M2 = rest_of(M, clusters, sums);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < clusters; ++s) {
            const float *src = slot_o(s, row);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + HD));
            const float f = moved(v.x, v.z, M, M2);
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(src) + chunk);
            L = fmaf(f, v.y, L);
            o.x = fmaf(f, x.x, o.x); o.y = fmaf(f, x.y, o.y); o.z = fmaf(f, x.z, o.z); o.w = fmaf(f, x.w, o.w);
        }
        const float inv = L == 0.f ? empty(row) : 1.f / L;
        store(row, chunk, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
}

// Clusters of 2, 4 and 8 CTAs that a device holds at once.
constexpr int MAX_DEV = 64;
int max_clusters[MAX_DEV][MAX_CLUSTER + 1];

// CTAs of a cluster and clusters of a group: the split that keeps most SMs busy, of
// equals the one with the larger clusters (a join in shared memory costs less than
// one through memory).  Several clusters only where a CTA keeps four tiles: their join
// through memory costs as much as two (8 nodes of 700 cells: 7.1 us, with up to a tile
// for each CTA 9.4; 16 of 2100: 12.3 and 15.4).  How many cells are in use is known on the
// device alone, so this goes by the cache's capacity: short trees in caches of 6144
// cells and more pay for the join all the same (9.4 and 15.5 us).
struct Plan { int cs, clusters; };
Plan plan(int groups, int n_ctx) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEV) dev = 0;
    const int tiles = (n_ctx + BKEY - 1) / BKEY;
    Plan best{1, 1};
    for (int cs = MAX_CLUSTER; cs >= 2; cs /= 2) {
        if (groups > max_clusters[dev][cs] || cs > tiles) continue;
        int k = max_clusters[dev][cs] / groups;
        if (k > tiles / (4 * cs)) k = tiles / (4 * cs);
        if (k > SLOTS / groups) k = SLOTS / groups;
        if (k < 1) k = 1;
        if (cs * k > best.cs * best.clusters) best = Plan{cs, k};
    }
    return best;
}

}  // namespace

size_t attn_tree_scratch_bytes(int, int, int, int, int hd, int) {
    return COUNTERS * sizeof(unsigned) + (size_t)SLOTS * BQ * ((hd == 128 ? 128 : 64) + 4) * sizeof(float);
}

cudaError_t launch_attn_tree(const AttnTreeArgs &a, const TmaMap &mK, const TmaMap &mV, const Launch &l) {
    const int hd = a.kv.head_dim, Hkv = a.kv.n_kv_head;
    if (Hkv < 1 || a.H % Hkv) return cudaErrorInvalidValue;
    const int row_tiles = (a.max_nodes * (a.H / Hkv) + BQ - 1) / BQ, groups = a.n_tree * Hkv * row_tiles;
    if (groups > 65535) return cudaErrorInvalidValue;
    const Plan p = plan(groups, a.kv.n_ctx);
    const CUtensorMap &k = reinterpret_cast<const CUtensorMap &>(mK), &v = reinterpret_cast<const CUtensorMap &>(mV);
    const dim3 grid(p.cs * p.clusters, groups), block(threads(a.kv.k8 != nullptr));
    const bool f8 = a.kv.k8;
    if (hd == 128)
        return launch_cluster_kernel(f8 ? attn_tree_kernel<128, true> : attn_tree_kernel<128, false>, grid, block, p.cs,
                                     f8 ? Cfg<128, true>::SMEM : Cfg<128, false>::SMEM, l, k, v, a, row_tiles, p.cs);
    if (hd == 64 || hd == 32)
        return launch_cluster_kernel(f8 ? attn_tree_kernel<64, true> : attn_tree_kernel<64, false>, grid, block, p.cs,
                                     f8 ? Cfg<64, true>::SMEM : Cfg<64, false>::SMEM, l, k, v, a, row_tiles, p.cs);
    return cudaErrorInvalidValue;
}

cudaError_t init_attn_tree_attributes() {
    cudaError_t e = allow_smem(attn_tree_kernel<128, false>, Cfg<128, false>::SMEM);
    if (!e) e = allow_smem(attn_tree_kernel<128, true>, Cfg<128, true>::SMEM);
    if (!e) e = allow_smem(attn_tree_kernel<64, false>, Cfg<64, false>::SMEM);
    if (!e) e = allow_smem(attn_tree_kernel<64, true>, Cfg<64, true>::SMEM);
    int dev = 0;
    if (!e) e = cudaGetDevice(&dev);
    if (e || dev < 0 || dev >= MAX_DEV) return e;
    for (int cs = 2; cs <= MAX_CLUSTER; cs *= 2) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(cs);
        cfg.blockDim = dim3(threads(false));
        cfg.dynamicSmemBytes = Cfg<128, false>::SMEM;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = cs;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if ((e = cudaOccupancyMaxActiveClusters(&n, attn_tree_kernel<128, false>, &cfg))) return e;
        max_clusters[dev][cs] = n;
    }
    return cudaSuccess;
}

}  // namespace llm
