// Decode GEMV over Q4_0 weight rows for 1..8 rows of x: y[t][n] = sum over
// blocks b of d[n][b] * sum over k in b of (c[n][k] - 8) * x[t][k], the linear
// layers of a decode step whose weights are held in four bits.
//
// Bound by HBM: 9/16 byte a weight, each read once, leaves 10 weights a clock
// to an SM sub-partition at the copy bandwidth.  Widening codes on the CUDA
// cores costs more than two instructions a weight, over that; so the codes go
// to the tensor cores as they are.  On this GPU mma.sync m16n8k16 (f16, f32
// sums) takes 8 clocks of a sub-partition, logic and shift instructions 2,
// FFMA 1.  The M side is 16 weight rows, the N side the rows of x (the other
// columns are zero).  A word of eight codes becomes four fragment registers by
// four ANDs and one shift: the masked halves are fp16 subnormals, c * 2^-24
// (bits 0, 16) and 16 c * 2^-24 (bits 4, 20), which the tensor cores multiply
// exactly; x is divided by 16 for the latter (where x is not in shared memory
// their sums are kept apart and divided instead).  The offset 8 is taken off by starting a sum at -8 sum(x) of its block: from a
// table in shared memory where x is there too, else from the product of x with
// a constant fragment, shared by every row of a warp's tile.  Each block of
// 32 k is one sum of at most 32 exact products in fp32, scaled by d in fp32
// and added in fp32: x and the codes are never rounded.
//
// One CTA an SM owns a contiguous run of rows.  Its 16 warps are 16 / units
// row groups of `units` warps: a group takes every (16 / units)-th tile of 32
// rows (two m16 tiles), warp cu of it the 128-element groups cu, cu + units, ..
// of K.  A warp brings its codes and scales itself, with cp.async, through a
// ring of its own (2304 bytes a step; the first steps before the dependency
// wait where the launch overlaps the previous kernel: weights never depend on
// it).  The warps of a row group join their sums in shared memory, in a fixed
// order, so results do not depend on timing.  More units spread few rows over all
// warps, fewer meet less often: the launcher takes the split with the fewest
// steps a warp, counting a meeting as half a step (with 16 units throughout,
// 128256 x 4096 took 83 us, a quarter of it in meetings).
// (Bulk copies by a producer warp, one a row and step, took 26.7 us for
// 28672 x 4096: about 130 clocks a copy of 1152 bytes.)
#include "common.cuh"
#include "launch.cuh"
#include "q4.cuh"

namespace llm {

namespace {

constexpr int CW = 16;                       // warps
constexpr int THREADS = CW * 32;
constexpr int RG = 32;                       // rows of a warp's tile (two m16 tiles)
constexpr int CODES = RG * 64;               // bytes of a step's codes in a warp's ring
constexpr int STAGE = CODES + RG * 8;        // ... and its scales
constexpr int RED_COL = 36;                  // floats between columns of a warp's sums (bank-conflict free)
constexpr size_t SMEM_CAP = 224 * 1024;
constexpr int X_PAD = 32;                    // elements between rows of x in shared memory beyond K

struct Plan {
    int units;           // warps that share a row tile's K
    int nst;             // ring stages of a warp
    bool x_smem;         // x is staged in shared memory
    int red_warp;        // floats of a warp's sums of one row tile (two tiles' sums alternate)
    size_t smem;
};

// false: K is not a positive multiple of 256
bool make_plan(int N, int K, int T, int ctas, Plan *p) {
    if (K < q4::CHUNK || K % q4::CHUNK) return false;
    const int groups = K / 128, rows = (N + ctas - 1) / ctas, tiles = (rows + RG - 1) / RG;
    long long best = 0;
    for (int u = CW; u >= 2; u /= 2) {
        const long long mine = (tiles + CW / u - 1) / (CW / u), cost = mine * (2LL * ((groups + u - 1) / u) + 1);
        if (u == CW || cost < best) { best = cost; p->units = u; }
    }
    // x and the table of its block sums (16 bytes a block and column pair)
    p->red_warp = (T + 1) / 2 * 2 * RED_COL;
    const size_t red = (size_t)2 * CW * p->red_warp * sizeof(float);
    const size_t x = (size_t)T * (K + X_PAD) * sizeof(f16) + (size_t)K * 2;
    // beside four ring stages, or three (74 KB in flight on an SM, still above
    // what the copy bandwidth needs at 1 us), where it fits, and a row tile
    // reads x from shared memory; else each warp reads its fragments from L2 a
    // step ahead: with so long a K a CTA has few row tiles to read x again for
    const size_t ring = (size_t)CW * STAGE;
    p->x_smem = x + red + 3 * ring <= SMEM_CAP;
    p->nst = !p->x_smem || x + red + 4 * ring <= SMEM_CAP ? 4 : 3;
    p->smem = p->nst * ring + red + (p->x_smem ? x : 0);
    return true;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, const float (&c)[4]) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// The power of two that brings an fp16 number of these bits (no sign) to
// 2^14 .. 2^15, 0 for zero; subnormals count by their leading bit.
__device__ __forceinline__ int row_shift(uint32_t bits) {
    return bits == 0u ? 0 : bits < 0x400u ? 14 + 24 - (31 - __clz(bits)) : bits >= 0x7C00u ? 0 : 14 - ((int)(bits >> 10) - 15);
}

// XS: x in shared memory; NST: ring stages of a warp
template <bool XS, int NST>
__global__ void __launch_bounds__(THREADS, 1) gemv_q4_kernel(const GemvQ4Args a, const Plan p, const int early) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ uint32_t s_top[8];                    // the rows' largest |x|, as fp16 bits
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int r0 = (int)((long long)blockIdx.x * a.N / gridDim.x);
    const int nrows = (int)((long long)(blockIdx.x + 1) * a.N / gridDim.x) - r0;
    const int groups = a.K / 128;
    const int units = p.units, cu = warp % units, rg = warp / units, TR = RG * CW / units;
    float *red = reinterpret_cast<float *>(smem_raw + (size_t)NST * CW * STAGE);
    f16 *xs = reinterpret_cast<f16 *>(red + 2 * CW * p.red_warp);

    // ---- this warp's ring: rows r0 + (tile * ngroups + rg) * 32 .., group kc * units + cu
    const int my_kc = cu < groups ? (groups - cu + units - 1) / units : 0;          // this warp's steps of a row tile
    const int ntiles = nrows > rg * RG ? (nrows - rg * RG + TR - 1) / TR : 0;       // its row group's tiles
    const int nsteps = my_kc * ntiles;
    uint8_t *ring = smem_raw + (size_t)warp * NST * STAGE;
    const uint32_t row_bytes = (uint32_t)groups / 2 * q4::CHUNK_BYTES;
    // sources of this lane's chunk of row g and of the scales of row `lane`, in the next step to request
    const uint8_t *csrc = a.W + (size_t)(r0 + rg * RG) * row_bytes + (size_t)(cu >> 1) * q4::CHUNK_BYTES;
    const uint8_t *ssrc = csrc + 128 + 8 * (cu & 1) + (size_t)lane * row_bytes;
    csrc += 64 * (cu & 1) + 16 * t4 + (size_t)g * row_bytes;
    const uint32_t cdst = smem_u32(ring) + g * 64 + ((t4 ^ ((g >> 1) & 3)) << 4);   // rows 8 apart have the same swizzle
    const uint32_t sdst = smem_u32(ring) + CODES + lane * 8;
    const size_t row8 = 8 * (size_t)row_bytes;
    const int kc_step = units / 2 * q4::CHUNK_BYTES;
    const long long tile_step = (long long)TR * row_bytes - (long long)(my_kc - 1) * kc_step;
    int want = nsteps, want_kc = my_kc, want_left = nrows - rg * RG;   // steps, steps of the tile and rows not requested
    uint32_t want_off = 0;                           // ring offset of the next step's slot
    auto request = [&]() {
        if (want > 0) {
            const uint32_t d = cdst + want_off;
            if (want_left >= RG) {
                const uint8_t *q = csrc;
#pragma unroll
                for (int i = 0; i < RG / 8; ++i) {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(d + i * 512), "l"(q));
                    q += row8;
                }
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" :: "r"(sdst + want_off), "l"(ssrc));
            } else {
                // rows past the CTA's repeat its last: their sums are not stored
                const int last = want_left - 1;
#pragma unroll
                for (int i = 0; i < RG / 8; ++i)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                 :: "r"(d + i * 512), "l"(csrc + (long long)(min(g + 8 * i, last) - g) * row_bytes));
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;"
                             :: "r"(sdst + want_off), "l"(ssrc + (long long)(min(lane, last) - lane) * row_bytes));
            }
            --want;
            want_off = want_off == (NST - 1) * STAGE ? 0 : want_off + STAGE;
            long long step = kc_step;
            if (--want_kc == 0) {
                want_kc = my_kc;
                want_left -= TR;
                step = tile_step;
            }
            csrc += step;
            ssrc += step;
        }
        cp_async_commit();
    };
    if (early)                                       // beside the previous kernel: weights never depend on it
        for (int j = 0; j < NST - 1; ++j) request();
    pdl_wait();
    pdl_trigger();

    // ---- x: column g of the N side is row g of x (columns from T on repeat row 0, their sums are not stored)
    float4 *tab = reinterpret_cast<float4 *>(xs + (size_t)a.T * (a.K + X_PAD));     // [K / 32][4]: {u, v, u, v}
    const f16 *xp = a.x;
    int ldx = a.ldx;
    if (XS) {
        // Into shared memory, as the fragments want it: pieces of 8 elements,
        // (0,1) (4,5) | (2,3) (6,7), the second half divided by 16 for the
        // nibbles that stand four bits higher.  So that the division rounds
        // nothing that counts, a row is first multiplied by the power of two
        // that brings its largest element to 2^14 .. 2^15, which is exact;
        // what is then rounded off is 2^-35 of that element at most.
        ldx = a.K + X_PAD;
        xp = xs;
        const int per = a.K / 8, n = a.T * per;      // pieces, a multiple of 32 a row
        if (tid < 8) s_top[tid] = 0u;
        __syncthreads();
        constexpr int HOLD = 4;                      // pieces a thread keeps between the two passes
        uint4 held[HOLD];
        auto piece = [&](int i) { return *reinterpret_cast<const uint4 *>(a.x + (size_t)(i / per) * a.ldx + (i % per) * 8); };
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (tid + j * THREADS < n) held[j] = piece(tid + j * THREADS);
        auto top = [&](int i, const uint4 &u) {      // of a warp's pieces, all of one row
            const uint32_t m = 0x7FFF7FFFu;
            const uint32_t v = __vmaxu2(__vmaxu2(u.x & m, u.y & m), __vmaxu2(u.z & m, u.w & m));
            const uint32_t w = __reduce_max_sync(0xffffffffu, max(v & 0xFFFFu, v >> 16));
            if (lane == 0) atomicMax(&s_top[i / per], w);
        };
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (tid + j * THREADS < n) top(tid + j * THREADS, held[j]);      // whole warps: n % 32 == 0
        for (int i = tid + HOLD * THREADS; i < n; i += THREADS) top(i, piece(i));
        __syncthreads();
        auto put = [&](int i, const uint4 &u) {
            const int t = i / per, c = i - t * per;
            const float up = __uint_as_float((uint32_t)(127 + row_shift(s_top[t])) << 23);
            const float e[8] = {h2lo(u.x) * up, h2hi(u.x) * up, h2lo(u.y) * up, h2hi(u.y) * up,
                                h2lo(u.z) * up, h2hi(u.z) * up, h2lo(u.w) * up, h2hi(u.w) * up};
            *reinterpret_cast<uint4 *>(xs + (size_t)t * ldx + c * 8) =
                make_uint4(pack_h2(e[0], e[1]), pack_h2(e[4], e[5]), pack_h2(e[2] * 0.0625f, e[3] * 0.0625f),
                           pack_h2(e[6] * 0.0625f, e[7] * 0.0625f));
            // -8 * 2^-24 * sum(x) of the block, where the lanes that sum x's column pair t / 2 look for it
            float v = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            if ((lane & 3) < 2) reinterpret_cast<float *>(tab + 4 * (c >> 2) + (t >> 1))[(t & 1) + 2 * (lane & 3)] = v * (-8.f / 16777216.f);
        };
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (tid + j * THREADS < n) put(tid + j * THREADS, held[j]);
        for (int i = tid + HOLD * THREADS; i < n; i += THREADS) put(i, piece(i));
    }
    if (!early)                                      // x was asked for first: it is not behind the weights' burst
        for (int j = 0; j < NST - 1; ++j) request();
    if (XS) __syncthreads();
    xp += (size_t)(g < a.T ? g : 0) * ldx + cu * 128 + 8 * t4;
    const float4 *tp = tab + (size_t)cu * 16 + t4;
    uint4 bx[4];                                     // !XS: the next step's x
    auto load_x = [&](int kc) {
#pragma unroll
        for (int b = 0; b < 4; ++b) bx[b] = *reinterpret_cast<const uint4 *>(xp + (size_t)kc * units * 128 + 32 * b);
    };
    if (!XS && nsteps > 0) load_x(0);

    uint32_t slot = 0;
    const uint8_t *wr = ring + g * 64 + ((t4 ^ ((g >> 1) & 3)) << 4), *dr = ring + CODES + g * 8;
    for (int tile = 0; tile < ntiles; ++tile) {
        float y[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
        for (int kc = 0; kc < my_kc; ++kc) {
            cp_async_wait<NST - 2>();
            __syncwarp();
            request();                           // into the slot read in the step before
            uint4 xv[4];
#pragma unroll
            for (int b = 0; b < 4; ++b)
                xv[b] = XS ? *reinterpret_cast<const uint4 *>(xp + kc * units * 128 + 32 * b) : bx[b];
            if (!XS) load_x(kc + 1 < my_kc ? kc + 1 : 0);
            uint4 w[2][2];                       // words of rows g and g + 8 of each m16 tile
            uint2 dd[2][2];                      // and their scales
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    w[i][h] = *reinterpret_cast<const uint4 *>(wr + slot + (16 * i + 8 * h) * 64);
                    dd[i][h] = *reinterpret_cast<const uint2 *>(dr + slot + (16 * i + 8 * h) * 8);
                }
            slot = slot + STAGE == NST * STAGE ? 0 : slot + STAGE;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint4 x = xv[b];
                float off1[4], off16[4] = {0.f, 0.f, 0.f, 0.f};
                if (XS) {
                    const float4 f = tp[kc * units * 16 + 4 * b];
                    off1[0] = f.x; off1[1] = f.y; off1[2] = f.z; off1[3] = f.w;
                } else {
                    mma(off1, 0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u, x.x, x.z, off16);
                    mma(off16, 0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u, x.y, x.w, off16);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t wg = b == 0 ? w[i][0].x : b == 1 ? w[i][0].y : b == 2 ? w[i][0].z : w[i][0].w;
                    const uint32_t wh = b == 0 ? w[i][1].x : b == 1 ? w[i][1].y : b == 2 ? w[i][1].z : w[i][1].w;
                    const uint32_t sg = wg >> 8, sh = wh >> 8;
                    const uint32_t pg = b < 2 ? dd[i][0].x : dd[i][0].y, ph = b < 2 ? dd[i][1].x : dd[i][1].y;
                    const float dg = b & 1 ? h2hi(pg) : h2lo(pg), dh = b & 1 ? h2hi(ph) : h2lo(ph);
                    float s1[4], s16[4];
                    mma(s1, wg & 0x000F000Fu, wh & 0x000F000Fu, sg & 0x000F000Fu, sh & 0x000F000Fu, x.x, XS ? x.y : x.z, off1);
                    if (XS) {
                        mma(s16, wg & 0x00F000F0u, wh & 0x00F000F0u, sg & 0x00F000F0u, sh & 0x00F000F0u, x.z, x.w, s1);
                    } else {
                        mma(s16, wg & 0x00F000F0u, wh & 0x00F000F0u, sg & 0x00F000F0u, sh & 0x00F000F0u, x.y, x.w, off16);
#pragma unroll
                        for (int e = 0; e < 4; ++e) s16[e] = fmaf(s16[e], 0.0625f, s1[e]);
                    }
                    y[i][0] = fmaf(dg, s16[0], y[i][0]);
                    y[i][1] = fmaf(dg, s16[1], y[i][1]);
                    y[i][2] = fmaf(dh, s16[2], y[i][2]);
                    y[i][3] = fmaf(dh, s16[3], y[i][3]);
                }
            }
        }
        // ---- the row tile is done: join the group's sums, in a fixed order
        float *sums = red + ((tile & 1) * CW + rg * units) * p.red_warp;
        if (2 * t4 < a.T) {
            float *mine = sums + cu * p.red_warp + 2 * t4 * RED_COL + g;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mine[16 * i] = y[i][0]; mine[16 * i + RED_COL] = y[i][1];
                mine[16 * i + 8] = y[i][2]; mine[16 * i + 8 + RED_COL] = y[i][3];
            }
        }
        // once a tile: the readers of these sums are done before the next but one overwrites them
        asm volatile("bar.sync %0, %1;" :: "r"(rg + 1), "r"(units * 32) : "memory");
        const int row = (tile * (CW / units) + rg) * RG + lane;
        for (int t = cu; t < a.T; t += units) {
            float v = 0.f;
            for (int c = 0; c < units; ++c) v += sums[c * p.red_warp + t * RED_COL + lane];
            const int sh = XS ? row_shift(s_top[t]) : 0;
            if (row < nrows) a.out[(size_t)t * a.ldo + r0 + row] = v * __uint_as_float((uint32_t)(127 + 24 - sh) << 23);
        }
    }
    cp_async_wait<0>();
}

}  // namespace

// early: with l.pdl, weights may be read before the previous kernel is done
cudaError_t launch_gemv_q4(const GemvQ4Args &a, int num_sms, const Launch &l, bool early) {
    Plan p;
    const int ctas = a.N < num_sms ? a.N : num_sms;
    if (a.T < 1 || a.T > 8 || ctas < 1 || !make_plan(a.N, a.K, a.T, ctas, &p)) return cudaErrorInvalidValue;
    const dim3 grid(ctas), block(THREADS);
    return !p.x_smem      ? launch_kernel(gemv_q4_kernel<false, 4>, grid, block, p.smem, l, a, p, (int)early)
           : p.nst == 4   ? launch_kernel(gemv_q4_kernel<true, 4>, grid, block, p.smem, l, a, p, (int)early)
                          : launch_kernel(gemv_q4_kernel<true, 3>, grid, block, p.smem, l, a, p, (int)early);
}

cudaError_t init_gemv_q4_attributes() {
    cudaError_t e = allow_smem(gemv_q4_kernel<true, 4>, SMEM_CAP);
    if (!e) e = allow_smem(gemv_q4_kernel<true, 3>, SMEM_CAP);
    if (!e) e = allow_smem(gemv_q4_kernel<false, 4>, SMEM_CAP);
    return e;
}

}  // namespace llm
