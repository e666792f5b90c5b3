// Prefill attention over a Q4_0 cache ("LLama.cpp — how it works", "KV-cache":
// a quantised cache where memory is short; the attention itself as in
// attn_prefill_tc.cu): causal grouped-query attention of a ubatch's rows, K and
// V standing for d * (c - 8) (q4.cuh), with nothing rounded below 22 bits on
// the way to the fp32 sums.
//
// Precision.  q is fp16 as it comes.  A cached value d * (c - 8) has up to 14
// significant bits, so it is the exact sum of two fp16 numbers, hi = f16(d *
// (c - 8)) and lo = d * (c - 8) - hi (both whole multiples of 2^-24, which fp16
// holds down to 0).  A softmax weight p = 2^x, x in fp32, is split the same way,
// its low 13 mantissa bits into a second fp16 number.  Then
//   S = q K_hi + q K_lo,     O = p_hi V_hi + p_lo V_hi + p_hi V_lo
// (p_lo V_lo is 2^-22 of the first).  Rounding K, V and p to fp16 and x to fp16,
// as the fp16 cache's kernel does, left 5.4e-4 of o's norm on 512 rows of 2048
// keys where fp32 leaves 2.1e-4 (o's own rounding), and more as scores grow: K's
// rounding moves a score by 2^-12 of its size.
//
// The tcgen05 kernel (head_dim 64 and 128).  One CTA takes 128 query rows of
// one sequence and one query head and walks the key tiles of 128 its rows see.
// Codes are widened inside the kernel, by warps that write hi and lo tiles into
// shared memory in the swizzled layout the MMAs read: a pass that widens the
// cache to memory first would need twice a layer's fp16 cache for them, and
// reading it back 128 KB a key tile and SM where the codes are 18 KB.
//   * Units of 32 KB (16 KB of hi, 16 KB of lo), three for K and three for V:
//     a K unit is 128 keys x 64 dimensions, a V unit 64 keys x 128 dimensions
//     (head_dim 64: 128 keys x 64).
//   * Warps 0-7 softmax (two threads a row, 64 keys each), 8-11 widen K, 12-15
//     V, 16 issues S and loads q by TMA, 17 issues O.
//   * Tensor memory: three S buffers of 128 columns; P takes the place of the S
//     it came from (of each 32 columns 16 of p_hi pairs, 16 of p_lo); O beside
//     them.  S_{t+3} is issued once O += P_t V_t is done.
// The running maximum is raised, and O rescaled, only when a tile's maximum
// passes it by 8 in base 2; weights are kept 2^7 times as large, so that those
// far below the maximum stay normal fp16 numbers (below 2^-21 of it their parts
// step by 2^-31 of it).
//
// Bound by the tensor cores and the shared memory that feeds them: 40 MMAs a key
// tile where the fp16 cache's kernel has 16, 224 KB read by them and 128 KB
// written by the widening.  512 rows of 32 heads of 128 from position 1536 on, 8
// kv heads: 37.6 us; a key tile takes 1.94 us, without the widening 1.86, without
// exponentials 1.62, the MMAs alone 1.60.  (With both parts rounded to fp16, read
// back from a widened copy: 24.4 us and 1.06 a tile.)  On the way there: a branch
// for each row's bounds in the widening 76 us; four widening warps, one a
// scheduler, which issue every fourth clock at best, 64; eight 46; descriptors by a
// whole warp, so that they stay in uniform registers, 44; K and V widened by warps
// of their own, the next unit asked for only once this one's registers are read,
// 41; a third S buffer 39; 128 registers for the softmax 38.  No faster: polls that
// sleep; the next unit's codes asked for ahead of this one's widening (2.1 us a
// tile); both units of K waited for ahead of S (1.91).
//
// The mma.sync kernel (head_dim 32, and wherever the other does not apply) takes
// 64 rows a CTA and 64 keys a tile with the same split and widening.
//
// A cell whose scale stands for values beyond fp16's range (or is not finite)
// makes the rows that see it NaN and no other: its K is NaN, which the mask
// replaces, and its V is 0.  Cells that no row of a tile sees are not read.
// Every mbarrier wait is bounded; on a timeout the CTA raises
// ERRF_WAIT_TIMEOUT, stops, waits (bounded) for its own copy in flight, frees
// its tensor memory and returns.
#include <cuda.h>

#include "attn_tc.cuh"
#include "attn_tile.cuh"
#include "common.cuh"
#include "launch.cuh"
#include "q4.cuh"
#include "tma.cuh"

namespace llm {

namespace {

using tcg::sdesc;
using tcg::tc_fence_after;
using tcg::tc_fence_before;
using tcg::tmem_ld32;
using namespace tca;

constexpr float LIFT = 7.f;                  // weights are kept 2^LIFT times as large
constexpr float RESCALE_LOG2 = 8.f;          // raise the running maximum only past this margin: weights <= 2^(8 + LIFT)

// Tile i of the launch: from memory, or out of the runs passed by value
// (tile_rows rows each, the last of a run fewer).
__device__ __forceinline__ AttnTile tile_of(const AttnPrefillArgs &a, const KvRuns &runs, int n_runs, int tile_rows, int i) {
    if (a.tiles) return a.tiles[i];
    int lo = 0, hi = n_runs - 1;                       // the last run that starts at or before tile i
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (runs.run[mid].tile0 <= i) lo = mid; else hi = mid - 1;
    }
    const KvRuns::Run r = runs.run[lo];
    const int at = (i - r.tile0) * tile_rows;
    return AttnTile{r.row0 + at, min(tile_rows, r.n_rows - at), r.seq, r.pos0 + at, 0};
}

__device__ __forceinline__ bool tile_bad(const AttnTile &tl, const KvView &kv, int rows) {
    return tl.seq < 0 || tl.seq >= kv.n_seq || tl.pos0 < 0 || tl.n_rows < 1 || tl.n_rows > rows ||
           tl.pos0 + tl.n_rows > kv.n_ctx;
}

// Non-zero where a scale of the pair stands for values beyond fp16's range:
// |d| > 8188 (an infinity or a NaN too); 8 * 8188 = 65504 and 8188 is 0x6FFF.
__device__ __forceinline__ uint32_t beyond(uint32_t d) { return ((d & 0x7FFF7FFFu) + 0x10001000u) & 0x80008000u; }

// The eight values of a word of codes with scale dd (in both halves) as hi and
// lo fp16 numbers, exactly: a rounded product, and its remainder by FMA.
__device__ __forceinline__ void split_word(const q4::Widen &wd, uint32_t w, __half2 dd, uint4 &hi, uint4 &lo) {
    const uint32_t w8 = w >> 8, c[4] = {wd.low(w), wd.high(w), wd.low(w8), wd.high(w8)};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 ci = *reinterpret_cast<const __half2 *>(&c[i]);
        const __half2 v = __hmul2_rn(ci, dd), r = __hfma2(ci, dd, __hneg2(v));
        h[i] = *reinterpret_cast<const uint32_t *>(&v);
        l[i] = *reinterpret_cast<const uint32_t *>(&r);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void st_shared(uint32_t at, const uint4 &v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ __half2 dup_lo(uint32_t d) {
    const uint32_t v = __byte_perm(d, 0, 0x1010);
    return *reinterpret_cast<const __half2 *>(&v);
}
__device__ __forceinline__ __half2 dup_hi(uint32_t d) {
    const uint32_t v = __byte_perm(d, 0, 0x3232);
    return *reinterpret_cast<const __half2 *>(&v);
}

// Two weights as hi and lo fp16 pairs: the low 13 mantissa bits are split off exactly.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &hi, uint32_t &lo) {
    const float ah = __uint_as_float(__float_as_uint(a) & 0xFFFFE000u), bh = __uint_as_float(__float_as_uint(b) & 0xFFFFE000u);
    hi = pack_h2(ah, bh);
    lo = pack_h2(a - ah, b - bh);
}

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(is));
    return is != 0;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *err) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
}

constexpr int BQ = 128, BKEY = 128;
constexpr int SM_WARPS = 8, W_WARP = 8, W_WARPS = 4, S_WARP = 16, PV_WARP = 17;   // W_WARPS for K, as many for V
constexpr int TC_THREADS = 20 * 32;           // five warpgroups; the last two warps only make up the number
// Registers a thread: 96 at launch (640 threads), then by warpgroup: 2 x 128 + 2 x 72 + 80 = 480 of 480
constexpr int SM_REGS = 128, W_REGS = 72, I_REGS = 80;
constexpr uint32_t QBOX = 128 * 128;          // bytes of one 128-row x 64-column fp16 box
constexpr uint32_t UNIT = 2 * QBOX;           // hi, then lo
constexpr int NU = 3;                         // units of each ring
constexpr int NS = 3;                         // S buffers
constexpr uint32_t TMEM_COLS = 512;           // S_b / P_b [128 b, 128 b + 128), O [384, 384 + hd)

template <int HD>
struct Q4Cfg {
    static constexpr int NBX = HD / 64;                         // 64-column boxes of a row = units of a tile
    static constexpr int NB = HD / 32;                          // blocks of a row
    static constexpr uint32_t K_OFF = NBX * QBOX;
    static constexpr uint32_t V_OFF = K_OFF + NU * UNIT;
    static constexpr uint32_t BAR_OFF = V_OFF + NU * UNIT;
    static constexpr uint32_t X_OFF = BAR_OFF + 256;            // barriers; the halves' exchange
    static constexpr size_t SMEM = X_OFF + 2 * 2 * BQ * sizeof(float);
    static constexpr uint32_t O_COL = NS * BKEY;
    // V units: keys of one, bytes of one of its 64-column boxes
    static constexpr int VKEYS = BKEY / NBX;
    static constexpr uint32_t VBOX = VKEYS * 128;
    // kind::f16 instruction descriptors: D fp32 (bit 4), A and B fp16, M = 128
    // (M >> 4 at bit 24), N >> 3 at bit 17; bit 16 marks B as MN-major
    static constexpr uint32_t IDESC_S = (1u << 4) | ((uint32_t)(BKEY >> 3) << 17) | ((uint32_t)(BQ >> 4) << 24);
    static constexpr uint32_t IDESC_O =
        (1u << 4) | (1u << 16) | ((uint32_t)(HD >> 3) << 17) | ((uint32_t)(BQ >> 4) << 24);
};

// A lane's share of a unit before it is widened: two tasks of two words, their
// two scales, and for K the scales of V's same blocks.
constexpr int WT = BKEY * 4 / (W_WARPS * 32);          // tasks of a lane and unit
struct Share {
    uint2 w[WT];
    uint32_t d[WT], dv[WT];
};

// Barriers: offsets from the first in units of eight bytes.
enum {
    B_Q = 0, B_S_FULL = 1, B_P_FULL = B_S_FULL + NS, B_PV_DONE = B_P_FULL + NS, B_K_FULL = B_PV_DONE + NS,
    B_K_EMPTY = B_K_FULL + NU, B_V_FULL = B_K_EMPTY + NU, B_V_EMPTY = B_V_FULL + NU, B_COUNT = B_V_EMPTY + NU
};
static_assert(8 * (B_COUNT + 1) <= 256, "barriers, the abort flag and the tensor-memory address");

// A widening warp's work: key rows kr, kr + 8, .. of a unit and of each row part
// lane / 8 of the words of two blocks; eight lanes write eight rows' chunks, which
// the swizzle spreads over all banks.  One warp a scheduler has to keep its own
// instructions apart: no branch inside a unit (with each task's bounds tested apart
// a unit took 2400 clocks).
template <int HD>
struct Widener {
    using C = Q4Cfg<HD>;
    static constexpr int NBX = C::NBX, NB = C::NB, ROWS = 8 * WT;     // key rows of a warp and unit
    const KvView &kv;
    size_t row0;                              // cache rows before the head's
    int kt0, lo, pos_last, ww, lane;
    uint32_t base, bar;
    volatile int *abort;
    uint32_t *err;
    q4::Widen wd;

    // first key row (of its 128-key tile) and 64-column half of the warp's share of unit `half` of a tile
    template <bool K>
    __device__ __forceinline__ void place(int half, int &kr, int &f) const {
        if (NBX == 1 || K) { kr = ww * ROWS; f = half; }
        else { kr = half * 64 + ww % (64 / ROWS) * ROWS; f = ww / (64 / ROWS); }
    }
    template <bool K>
    __device__ __forceinline__ void load(int idx, Share &x) const {
        const int part = lane >> 3, r8 = lane & 7;
        int kr, f;
        place<K>(idx % NBX, kr, f);
        const int first = (kt0 + idx / NBX) * BKEY + kr;         // the warp's first row
        const uint8_t *codes = (K ? kv.k4 : kv.v4) + 4 * (part * NB + 2 * f);
        const f16 *scales = (K ? kv.kd : kv.vd) + 2 * f, *vscales = kv.vd + 2 * f;
        if (first >= lo && first + ROWS - 1 <= pos_last) {
            const size_t row = row0 + first + r8;
            codes += row * (HD / 2);
            scales += row * NB;
            vscales += row * NB;
#pragma unroll
            for (int i = 0; i < WT; ++i) {
                x.w[i] = __ldcg(reinterpret_cast<const uint2 *>(codes + i * 8 * (HD / 2)));
                x.d[i] = __ldcg(reinterpret_cast<const uint32_t *>(scales + i * 8 * NB));
                x.dv[i] = K ? __ldcg(reinterpret_cast<const uint32_t *>(vscales + i * 8 * NB)) : 0u;
            }
        } else {
            // in place of rows that no row of the tile sees the nearest that one does, with scale 0
#pragma unroll
            for (int i = 0; i < WT; ++i) {
                const int key = first + 8 * i + r8;
                const size_t row = row0 + min(max(key, lo), pos_last);
                const uint32_t in = key >= lo && key <= pos_last ? ~0u : 0u;
                x.w[i] = __ldcg(reinterpret_cast<const uint2 *>(codes + row * (HD / 2)));
                x.d[i] = __ldcg(reinterpret_cast<const uint32_t *>(scales + row * NB)) & in;
                x.dv[i] = K ? __ldcg(reinterpret_cast<const uint32_t *>(vscales + row * NB)) & in : 0u;
            }
        }
    }
    template <bool K>
    __device__ __forceinline__ bool put(int idx, bool more, Share &x) const {
        const int part = lane >> 3, r8 = lane & 7, slot = idx % NU, use = idx / NU;
        if (use > 0 && !warp_wait(bar + 8u * ((K ? B_K_EMPTY : B_V_EMPTY) + slot), (use - 1) & 1, abort, err)) return false;
        uint32_t over = 0;
#pragma unroll
        for (int i = 0; i < WT; ++i) over |= beyond(x.d[i]) | beyond(x.dv[i]);
        const bool odd = __any_sync(0xffffffffu, over != 0);
        if (!K && odd) {
#pragma unroll
            for (int i = 0; i < WT; ++i)
                if (beyond(x.d[i])) x.d[i] = 0u;
        }
        int kr, f;
        place<K>(idx % NBX, kr, f);
        const uint32_t row = NBX == 1 || K ? (uint32_t)(kr + r8) * 128u : (uint32_t)f * C::VBOX + (uint32_t)((kr & 63) + r8) * 128u;
        const uint32_t unit = base + (K ? C::K_OFF : C::V_OFF) + (uint32_t)slot * UNIT + row;
        const uint32_t c0 = unit + (uint32_t)((part ^ r8) << 4), c1 = unit + (uint32_t)(((4 + part) ^ r8) << 4);
#pragma unroll
        for (int i = 0; i < WT; ++i) {
            uint4 h0, l0, h1, l1;
            split_word(wd, x.w[i].x, dup_lo(x.d[i]), h0, l0);
            split_word(wd, x.w[i].y, dup_hi(x.d[i]), h1, l1);
            st_shared(c0 + 1024u * i, h0);
            st_shared(c0 + 1024u * i + QBOX, l0);
            st_shared(c1 + 1024u * i, h1);
            st_shared(c1 + 1024u * i + QBOX, l1);
        }
        if (K && odd) {
#pragma unroll
            for (int i = 0; i < WT; ++i)
                if (beyond(x.d[i]) | beyond(x.dv[i])) st_shared(c0 + 1024u * i, make_uint4(0x7FFF7FFFu, 0u, 0u, 0u));
        }
        // the next unit is asked for once this one's registers are read, and no earlier: a wait for older loads is one
        // for these too
        if (more) load<K>(idx + 1, x);
        fence_proxy_async();                             // the MMAs read through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + 8u * ((K ? B_K_FULL : B_V_FULL) + slot));
        return true;
    }
    // the units of K's tiles or of V's
    template <bool K>
    __device__ __forceinline__ void run(int units) const {
        Share x;
        load<K>(0, x);
        for (int u = 0; u < units; ++u)
            if (!put<K>(u, u + 1 < units, x)) break;
    }
};

template <int HD, bool WIN>
__global__ void __launch_bounds__(TC_THREADS, 1)
attn_prefill_q4_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const AttnPrefillArgs a,
                          const __grid_constant__ KvRuns runs, const int n_runs) {
    using C = Q4Cfg<HD>;
    constexpr int NBX = C::NBX;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // the swizzle wants 1024-byte boundaries; there is no room to round up
    const uint32_t base = smem_u32(smem_raw);
    int *const state = reinterpret_cast<int *>(smem_raw + C::BAR_OFF + 8 * B_COUNT);       // abort flag, tensor-memory address
    float *const xch = reinterpret_cast<float *>(smem_raw + C::X_OFF);                     // [2][half][row]
    const uint32_t bar = base + C::BAR_OFF;
    const uint32_t q_full = bar + 8u * B_Q;
    auto s_full = [&](int b) { return bar + 8u * (B_S_FULL + b); };
    auto p_full = [&](int b) { return bar + 8u * (B_P_FULL + b); };       // P_t written
    auto pv_done = [&](int b) { return bar + 8u * (B_PV_DONE + b); };     // O += P_t V_t done
    auto k_full = [&](int s) { return bar + 8u * (B_K_FULL + s); };
    auto k_empty = [&](int s) { return bar + 8u * (B_K_EMPTY + s); };
    auto v_full = [&](int s) { return bar + 8u * (B_V_FULL + s); };
    auto v_empty = [&](int s) { return bar + 8u * (B_V_EMPTY + s); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = state;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        for (int b = 0; b < NS; ++b) {
            mbar_init(s_full(b), 1);
            mbar_init(p_full(b), SM_WARPS);
            mbar_init(pv_done(b), 1);
        }
        for (int s = 0; s < NU; ++s) {
            mbar_init(k_full(s), W_WARPS);
            mbar_init(k_empty(s), 1);
            mbar_init(v_full(s), W_WARPS);
            mbar_init(v_empty(s), 1);
        }
        state[0] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&tmQ)) : "memory");
    }
    if (warp == S_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(state + 1)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)state[1];
    pdl_wait();                                          // q, the cache and the tiles come from the kernels before
    pdl_trigger();

    // longest tiles (latest positions) first
    const AttnTile tl = tile_of(a, runs, n_runs, BQ, a.n_tiles - 1 - (int)blockIdx.x);
    const int h = blockIdx.y, Hkv = a.kv.n_kv_head, j = h / (a.H / Hkv);
    const bool bad = tile_bad(tl, a.kv, BQ) || (base & 1023u) != 0;
    if (bad && threadIdx.x == 0) raise_error(a.err, ERRF_BAD_INDEX);
    const int pos_last = tl.pos0 + tl.n_rows - 1;
    const int W = WIN ? a.window : 0;
    const int lo = W > 0 && tl.pos0 + 1 > W ? tl.pos0 + 1 - W : 0;      // the first key any row sees
    const int kt0 = lo / BKEY, nt = bad ? 0 : pos_last / BKEY + 1 - kt0;

    if (warp < SM_WARPS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(SM_REGS));
    else if (warp < W_WARP + 2 * W_WARPS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(W_REGS));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(I_REGS));
    if (nt == 0) {
        // nothing to do: on to the end
    } else if (warp < SM_WARPS) {
        // ---- softmax: thread row r of the query tile, keys [64 hf, 64 hf + 64) of each tile
        constexpr int HK = BKEY / 2;
        const int quarter = warp & 3, hf = warp >> 2;
        const int r = quarter * 32 + lane, qpos = tl.pos0 + r;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t o_col = C::O_COL + hf * (HD / 2);     // this half's O columns
        const float c = 1.4426950408889634f / sqrtf((float)HD);
        // the other half's value of the same row; two buffers in turn, so that a half one tile ahead does not overwrite
        // what the other has not read
        auto exchange = [&](int turn, float v) {
            float *x = xch + (turn & 1) * 2 * BQ + r;
            x[hf * BQ] = v;
            named_sync(1, SM_WARPS * 32);
            return x[(hf ^ 1) * BQ];
        };
        float m_run = -INFINITY, l_run = 0.f;
        // ok stays uniform over each warp, and every softmax thread runs all nt
        // iterations, so the named barriers (which have no time limit) are always
        // reached by all 256 threads; after a timeout the iterations only pass them
        bool ok = true;
        int b = 0, round = 0;                                // t % NS, t / NS
        for (int t = 0; t < nt; ++t, b = b + 1 == NS ? 0 : b + 1, round += b == 0) {
            const int key0 = (kt0 + t) * BKEY + hf * HK;
            const uint32_t s_col = lane_base + b * BKEY + hf * HK;
            ok = ok && warp_wait(s_full(b), round & 1, abort, a.err);
            float s[HK];
            float mx = -INFINITY;
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int q = 0; q < HK / 32; ++q) {
                    uint32_t v[32];
                    tmem_ld32(s_col + q * 32, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[q * 32 + i] = __uint_as_float(v[i]);
                }
                // causal (and window) mask: key k is visible iff k <= qpos (and qpos - k < W)
                if (key0 + HK - 1 > qpos || (WIN && qpos - key0 >= W)) {
#pragma unroll
                    for (int i = 0; i < HK; ++i) {
                        const int k = key0 + i;
                        if (k > qpos || (WIN && qpos - k >= W)) s[i] = -INFINITY;
                    }
                }
                float m8[8];                                 // half-row maximum as a tree of 8 chains
#pragma unroll
                for (int i = 0; i < 8; ++i) m8[i] = s[i];
#pragma unroll
                for (int i = 8; i < HK; ++i) m8[i & 7] = fmaxf(m8[i & 7], s[i]);
                mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
            }
            mx = fmaxf(mx, exchange(t, mx));
            if (!ok) continue;
            float factor = 1.f;
            const bool raise = mx != -INFINITY && (m_run == -INFINITY || (mx - m_run) * c > RESCALE_LOG2);
            if (raise) {
                factor = m_run == -INFINITY ? 0.f : ex2((m_run - mx) * c);
                m_run = mx;
            }
            const float m0 = m_run == -INFINITY ? 0.f : m_run;
            // a raised maximum rescales O, which P_{t-1} V_{t-1} must have finished
            if (t >= 1 && __any_sync(0xffffffffu, raise)) {
                ok = warp_wait(pv_done(b == 0 ? NS - 1 : b - 1), (b == 0 ? round - 1 : round) & 1, abort, a.err);
                if (!ok) continue;
                tc_fence_after();
#pragma unroll 1
                for (int q = 0; q < HD / 64; ++q) {
                    uint32_t v[32];
                    tmem_ld32(lane_base + o_col + q * 32, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * factor);
                    tmem_st32(lane_base + o_col + q * 32, v);
                }
            }
            // the weights of 32 keys over the columns of S they came from: 16 of hi pairs, 16 of lo pairs
            float rs8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) rs8[i] = 0.f;
#pragma unroll
            for (int q = 0; q < HK / 32; ++q) {
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p0 = ex2(fmaf(s[32 * q + 2 * i] - m0, c, LIFT)), p1 = ex2(fmaf(s[32 * q + 2 * i + 1] - m0, c, LIFT));
                    rs8[(2 * i) & 7] += p0;
                    rs8[(2 * i + 1) & 7] += p1;
                    split_pair(p0, p1, p[i], p[16 + i]);
                }
                tmem_st32(s_col + 32 * q, p);
            }
            l_run = l_run * factor + (((rs8[0] + rs8[1]) + (rs8[2] + rs8[3])) + ((rs8[4] + rs8[5]) + (rs8[6] + rs8[7])));
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(b));
        }
        const float l_row = l_run + exchange(nt, l_run);
        if (ok && warp_wait(pv_done((nt - 1) % NS), (nt - 1) / NS & 1, abort, a.err)) {
            tc_fence_after();
            const float inv = l_row > 0.f ? 1.f / l_row : 0.f;
            f16 *dst = a.o + ((size_t)(tl.row0 + r) * a.H + h) * HD + hf * (HD / 2);
#pragma unroll 1
            for (int q = 0; q < HD / 64; ++q) {
                uint32_t v[32];
                tmem_ld32(lane_base + o_col + q * 32, v);
                if (r < tl.n_rows) {
                    uint4 *d4 = reinterpret_cast<uint4 *>(dst + q * 32);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        d4[i] = make_uint4(pack_h2(__uint_as_float(v[8 * i]) * inv, __uint_as_float(v[8 * i + 1]) * inv),
                                           pack_h2(__uint_as_float(v[8 * i + 2]) * inv, __uint_as_float(v[8 * i + 3]) * inv),
                                           pack_h2(__uint_as_float(v[8 * i + 4]) * inv, __uint_as_float(v[8 * i + 5]) * inv),
                                           pack_h2(__uint_as_float(v[8 * i + 6]) * inv, __uint_as_float(v[8 * i + 7]) * inv));
                }
            }
        }
    } else if (warp < W_WARP + 2 * W_WARPS) {
        // ---- widening: K and V by warps of their own, so that neither ring waits behind the other
        Widener<HD> wide{a.kv, ((size_t)tl.seq * a.kv.seq_stride + (size_t)j * a.kv.n_ctx * HD) / HD, kt0, lo, pos_last,
                         (warp - W_WARP) % W_WARPS, lane, base, bar, abort, a.err};
        if (warp < W_WARP + W_WARPS) wide.template run<true>(nt * NBX);
        else wide.template run<false>(nt * NBX);
    } else if (warp == S_WARP) {
        // ---- S_t = q K_t^T into buffer t % NS, once the P that took the place of the S before has been read.  The whole warp walks
        // the loop, so that addresses and descriptors stay uniform; the elected lane issues.
        const bool leader = elect_one();
        if (leader) {
            mbar_expect_tx(q_full, NBX * QBOX);
            for (int i = 0; i < NBX; ++i) tma_load_2d(base + i * QBOX, &tmQ, q_full, h * HD + i * 64, tl.row0);
        }
        bool ok = warp_wait(q_full, 0, abort, a.err);
        const uint64_t q_desc = sdesc(base), k_desc = sdesc(base + C::K_OFF);
        uint32_t slot = 0, use = 0;
        for (int t = 0; ok && t < nt; ++t) {
            const int b = t % NS;
            if (t >= NS && !warp_wait(pv_done(b), (t / NS - 1) & 1, abort, a.err)) break;
            const uint32_t s_acc = tmem + b * BKEY;
            for (int f = 0; f < NBX; ++f) {
                ok = warp_wait(k_full(slot), use & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint64_t qd = q_desc + (uint32_t)f * (QBOX >> 4), kd = k_desc + slot * (UNIT >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        mma1(s_acc, qd + 2 * kk, kd + 2 * kk, C::IDESC_S, (f | kk) != 0);
                        mma1(s_acc, qd + 2 * kk, kd + (QBOX >> 4) + 2 * kk, C::IDESC_S, 1);
                    }
                    commit1(k_empty(slot));
                    if (f == NBX - 1) commit1(s_full(b));
                }
                __syncwarp();
                if (++slot == NU) { slot = 0; ++use; }
            }
        }
    } else if (warp == PV_WARP) {
        // ---- O (+)= P_t V_t once the softmax has written P_t (and rescaled O)
        const bool leader = elect_one();
        const uint32_t o_acc = tmem + C::O_COL;
        const uint64_t v_desc = sdesc_mn(base + C::V_OFF, C::VBOX);
        uint32_t slot = 0, use = 0;
        bool ok = true;
        for (int t = 0; ok && t < nt; ++t) {
            const int b = t % NS;
            if (!warp_wait(p_full(b), t / NS & 1, abort, a.err)) break;
            for (int f = 0; f < NBX; ++f) {
                ok = warp_wait(v_full(slot), use & 1, abort, a.err);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint64_t vd = v_desc + slot * (UNIT >> 4);
                    const uint32_t p0 = tmem + b * BKEY + f * C::VKEYS;
#pragma unroll
                    for (int kk = 0; kk < C::VKEYS / 16; ++kk) {
                        // 16 keys: 8 columns of P's hi pairs, 16 on their lo pairs, among the 32 of their 32 keys
                        const uint32_t p = p0 + kk / 2 * 32 + kk % 2 * 8;
                        mma1_ts(o_acc, p, vd + kk * (2048 >> 4), C::IDESC_O, (t | f | kk) != 0);
                        mma1_ts(o_acc, p + 16, vd + kk * (2048 >> 4), C::IDESC_O, 1);
                        mma1_ts(o_acc, p, vd + (QBOX >> 4) + kk * (2048 >> 4), C::IDESC_O, 1);
                    }
                    commit1(v_empty(slot));
                    if (f == NBX - 1) commit1(pv_done(b));
                }
                __syncwarp();
                if (++slot == NU) { slot = 0; ++use; }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // after a timeout: wait (bounded) for q's copy before the memory is released
    if (*abort && warp == S_WARP && lane == 0)
        for (uint32_t i = 0; i < WAIT_LIMIT && !mbar_try_wait(q_full, 0); ++i) {
        }
    __syncthreads();
    if (warp == S_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

// ---------------------------------------------------------------- mma.sync

constexpr int MQ = 64, MKEY = 64, M_THREADS = 128;

template <int HD, bool WIN>
__global__ void __launch_bounds__(M_THREADS) attn_prefill_q4_kernel(const AttnPrefillArgs a,
                                                                    const __grid_constant__ KvRuns runs, const int n_runs) {
    constexpr int NB = HD / 32, TASKS = MKEY * 4 / M_THREADS;     // (row, word part) tasks of a thread and tile
    extern __shared__ __align__(128) uint8_t smem_mma[];
    f16 *Qs = reinterpret_cast<f16 *>(smem_mma);
    f16 *Kh = Qs + MQ * HD, *Kl = Kh + MKEY * HD, *Vh = Kl + MKEY * HD, *Vl = Vh + MKEY * HD;

    pdl_wait();
    pdl_trigger();
    const AttnTile tl = tile_of(a, runs, n_runs, MQ, a.n_tiles - 1 - (int)blockIdx.x);
    const int h = blockIdx.y, j = h / (a.H / a.kv.n_kv_head);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    if (tile_bad(tl, a.kv, MQ)) {
        if (tid == 0) raise_error(a.err, ERRF_BAD_INDEX);
        return;
    }
    const int n_keys = tl.pos0 + tl.n_rows, W = WIN ? a.window : 0;
    const int lo = W > 0 && tl.pos0 + 1 > W ? tl.pos0 + 1 - W : 0;
    const int kt0 = lo / MKEY, n_kt = (n_keys + MKEY - 1) / MKEY;
    const size_t row0 = ((size_t)tl.seq * a.kv.seq_stride + (size_t)j * a.kv.n_ctx * HD) / HD;

    // Q tile (rows past n_rows are zero)
    for (int i = tid; i < MQ * (HD / 8); i += M_THREADS) {
        const int r = i / (HD / 8), c = i - r * (HD / 8);
        const bool pv = r < tl.n_rows;
        cp_async16(Qs + Swz<HD>::off(r, c), a.q + ((size_t)(tl.row0 + (pv ? r : 0)) * a.H + h) * HD + c * 8, pv);
    }
    cp_async_commit();

    // a thread's codes and scales of a tile: row task % 64, word part task / 64
    uint32_t kw[TASKS][NB], vw[TASKS][NB];
    uint16_t kd[TASKS][NB], vd[TASKS][NB];
    auto load = [&](int kt) {
#pragma unroll
        for (int i = 0; i < TASKS; ++i) {
            const int x = tid + i * M_THREADS, key = kt * MKEY + x % MKEY, part = x / MKEY;
            const bool in = key >= lo && key < n_keys;
            const size_t row = row0 + (in ? key : lo);
            const uint32_t *pk = reinterpret_cast<const uint32_t *>(a.kv.k4 + row * (HD / 2)) + part * NB;
            const uint32_t *pv = reinterpret_cast<const uint32_t *>(a.kv.v4 + row * (HD / 2)) + part * NB;
            const unsigned short *sk = reinterpret_cast<const unsigned short *>(a.kv.kd + row * NB);
            const unsigned short *sv = reinterpret_cast<const unsigned short *>(a.kv.vd + row * NB);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                kw[i][b] = __ldcg(pk + b);
                vw[i][b] = __ldcg(pv + b);
                kd[i][b] = in ? __ldcg(sk + b) : (unsigned short)0;
                vd[i][b] = in ? __ldcg(sv + b) : (unsigned short)0;
            }
        }
    };
    const q4::Widen wd;
    auto put = [&]() {
#pragma unroll
        for (int i = 0; i < TASKS; ++i) {
            const int x = tid + i * M_THREADS, r = x % MKEY, part = x / MKEY;
            uint32_t nan = 0;
#pragma unroll
            for (int b = 0; b < NB; ++b) nan |= beyond(kd[i][b]) | beyond(vd[i][b]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                uint4 hi, lw;
                const int at = Swz<HD>::off(r, 4 * b + part);
                split_word(wd, kw[i][b], dup_lo(kd[i][b]), hi, lw);
                if (nan && b == 0) hi.x = 0x7FFF7FFFu;
                *reinterpret_cast<uint4 *>(Kh + at) = hi;
                *reinterpret_cast<uint4 *>(Kl + at) = lw;
                split_word(wd, vw[i][b], dup_lo(beyond(vd[i][b]) ? 0u : vd[i][b]), hi, lw);
                *reinterpret_cast<uint4 *>(Vh + at) = hi;
                *reinterpret_cast<uint4 *>(Vl + at) = lw;
            }
        }
    };

    float o[HD / 8][4];
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float mrow[2] = {-INFINITY, -INFINITY}, lrow[2] = {0.f, 0.f};
    const float sl2 = 1.4426950408889634f / sqrtf((float)HD);
    const int qp0 = tl.pos0 + warp * 16 + g;       // position of this thread's first row
    uint32_t qf[HD / 16][4];

    load(kt0);
    for (int kt = kt0; kt < n_kt; ++kt) {
        __syncthreads();                           // the tile before is read
        put();
        if (kt + 1 < n_kt) load(kt + 1);
        if (kt == kt0) cp_async_wait<0>();
        __syncthreads();
        if (kt == kt0) {
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
                const int r = warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
                ldmatrix_x4(qf[kk], smem_u32(Qs + Swz<HD>::off(r, kk * 2 + (lane >> 4))));
            }
        }
        // S = Q K^T for 16 rows x 64 keys
        float s[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
#pragma unroll
            for (int np = 0; np < 4; ++np) {       // pairs of 8-key tiles
                const int at = Swz<HD>::off(np * 16 + (lane & 7) + (lane >> 4) * 8, kk * 2 + ((lane >> 3) & 1));
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    uint32_t kf[4];
                    ldmatrix_x4(kf, smem_u32((part ? Kl : Kh) + at));
                    const uint32_t b0[2] = {kf[0], kf[1]}, b1[2] = {kf[2], kf[3]};
                    mma_f16_16816(s[2 * np], qf[kk], b0);
                    mma_f16_16816(s[2 * np + 1], qf[kk], b1);
                }
            }
        }
        // mask + online softmax (rows qp0 and qp0 + 8)
        const int key0 = kt * MKEY;
        const bool need_mask = key0 + MKEY - 1 > tl.pos0 + warp * 16 || WIN;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = key0 + nt * 8 + 2 * t4 + (e & 1), qp = qp0 + (e >> 1) * 8;
                float v = s[nt][e];
                if (need_mask && (key > qp || (WIN && qp - key >= W))) v = -INFINITY;
                s[nt][e] = v;
                mx[e >> 1] = fmaxf(mx[e >> 1], v);
            }
        }
        float corr[2], m0[2], rs[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            const float mn = fmaxf(mrow[r], mx[r]);
            corr[r] = mn == -INFINITY ? 1.f : ex2((mrow[r] - mn) * sl2);
            mrow[r] = mn;
            m0[r] = mn == -INFINITY ? 0.f : mn;
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nt][e] = ex2(fmaf(s[nt][e] - m0[e >> 1], sl2, LIFT));
                rs[e >> 1] += s[nt][e];
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            rs[r] += __shfl_xor_sync(0xffffffffu, rs[r], 1);
            rs[r] += __shfl_xor_sync(0xffffffffu, rs[r], 2);
            lrow[r] = lrow[r] * corr[r] + rs[r];
        }
#pragma unroll
        for (int dt = 0; dt < HD / 8; ++dt) {
            o[dt][0] *= corr[0]; o[dt][1] *= corr[0];
            o[dt][2] *= corr[1]; o[dt][3] *= corr[1];
        }
        // O += P V
#pragma unroll
        for (int kk = 0; kk < MKEY / 16; ++kk) {
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split_pair(s[2 * kk + (i >> 1)][2 * (i & 1)], s[2 * kk + (i >> 1)][2 * (i & 1) + 1], ph[i], pl[i]);
#pragma unroll
            for (int dp = 0; dp < HD / 16; ++dp) {
                const int at = Swz<HD>::off(kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, dp * 2 + (lane >> 4));
                uint32_t vf[4];
                ldmatrix_x4_trans(vf, smem_u32(Vh + at));
                const uint32_t b0[2] = {vf[0], vf[1]}, b1[2] = {vf[2], vf[3]};
                mma_f16_16816(o[2 * dp], ph, b0);
                mma_f16_16816(o[2 * dp + 1], ph, b1);
                mma_f16_16816(o[2 * dp], pl, b0);
                mma_f16_16816(o[2 * dp + 1], pl, b1);
                ldmatrix_x4_trans(vf, smem_u32(Vl + at));
                const uint32_t l0[2] = {vf[0], vf[1]}, l1[2] = {vf[2], vf[3]};
                mma_f16_16816(o[2 * dp], ph, l0);
                mma_f16_16816(o[2 * dp + 1], ph, l1);
            }
        }
    }

    // normalise and store
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = warp * 16 + g + r * 8;
        if (row >= tl.n_rows) continue;
        const float inv = lrow[r] > 0.f ? 1.f / lrow[r] : 0.f;
        f16 *dst = a.o + ((size_t)(tl.row0 + row) * a.H + h) * HD;
#pragma unroll
        for (int dt = 0; dt < HD / 8; ++dt)
            *reinterpret_cast<uint32_t *>(dst + dt * 8 + 2 * t4) = pack_h2(o[dt][2 * r] * inv, o[dt][2 * r + 1] * inv);
    }
}

template <int HD>
constexpr size_t mma_smem() { return (size_t)(MQ + 4 * MKEY) * HD * sizeof(f16); }

}  // namespace

bool attn_prefill_q4_tc_ok(int head_dim) { return head_dim == 64 || head_dim == 128; }

int attn_prefill_q4_rows(bool tc) { return tc ? BQ : MQ; }

cudaError_t launch_attn_prefill_q4(const AttnPrefillArgs &a, const KvRuns *runs, int n_runs, const TmaMap *mQ, const Launch &l) {
    if (a.n_tiles < 1) return cudaSuccess;
    const int hd = a.kv.head_dim, Hkv = a.kv.n_kv_head;
    if (Hkv < 1 || a.H % Hkv || a.H > 65535 || !a.kv.k4 || (!a.tiles && (!runs || n_runs < 1 || n_runs > KvRuns::MAX)))
        return cudaErrorInvalidValue;
    static const KvRuns none = {};
    const KvRuns &r = a.tiles ? none : *runs;
    const dim3 grid(a.n_tiles, a.H);
    const bool win = a.window > 0;
    if (mQ) {
        const CUtensorMap &q = *reinterpret_cast<const CUtensorMap *>(mQ);
        if (hd == 128)
            return launch_kernel(win ? attn_prefill_q4_tc_kernel<128, true> : attn_prefill_q4_tc_kernel<128, false>, grid,
                                 dim3(TC_THREADS), Q4Cfg<128>::SMEM, l, q, a, r, n_runs);
        if (hd == 64)
            return launch_kernel(win ? attn_prefill_q4_tc_kernel<64, true> : attn_prefill_q4_tc_kernel<64, false>, grid,
                                 dim3(TC_THREADS), Q4Cfg<64>::SMEM, l, q, a, r, n_runs);
        return cudaErrorInvalidValue;
    }
#define Q4_PRE_CASE(HDV)                                                                                                 \
    if (hd == HDV)                                                                                                       \
        return launch_kernel(win ? attn_prefill_q4_kernel<HDV, true> : attn_prefill_q4_kernel<HDV, false>, grid, dim3(M_THREADS), \
                             mma_smem<HDV>(), l, a, r, n_runs);
    Q4_PRE_CASE(32) Q4_PRE_CASE(64) Q4_PRE_CASE(128)
#undef Q4_PRE_CASE
    return cudaErrorInvalidValue;
}

cudaError_t init_attn_prefill_q4_attributes() {
    cudaError_t e = cudaSuccess;
#define Q4_PRE_ATTR(HDV)                                                                          \
    if (!e) e = allow_smem(attn_prefill_q4_kernel<HDV, false>, mma_smem<HDV>());                   \
    if (!e) e = allow_smem(attn_prefill_q4_kernel<HDV, true>, mma_smem<HDV>());
    Q4_PRE_ATTR(32) Q4_PRE_ATTR(64) Q4_PRE_ATTR(128)
#undef Q4_PRE_ATTR
#define Q4_PRE_ATTR(HDV)                                                                           \
    if (!e) e = allow_smem(attn_prefill_q4_tc_kernel<HDV, false>, Q4Cfg<HDV>::SMEM);                \
    if (!e) e = allow_smem(attn_prefill_q4_tc_kernel<HDV, true>, Q4Cfg<HDV>::SMEM);
    Q4_PRE_ATTR(64) Q4_PRE_ATTR(128)
#undef Q4_PRE_ATTR
    return e;
}

}  // namespace llm
