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
// exactly.  The two scales of 16 are summed apart and joined in fp32.  The
// offset 8 is taken off by starting a sum at -8 sum(x) of its block: from a
// table in shared memory where x is there too, else from the product of x with
// a constant fragment, shared by every row of a warp's tile.  Each block of
// 32 k is one sum of at most 32 exact products in fp32, scaled by d in fp32
// and added in fp32: x and the codes are never rounded.
//
// One CTA an SM owns a contiguous run of rows, cut into steps of TR rows by C
// chunks of 256 k.  Warp w takes the 128-element group w % 2C of the 32 rows
// (two m16 tiles) of row group w / 2C in every step and brings them itself,
// with cp.async, through a ring of its own: 2304 bytes a step, the ring's first
// steps before the dependency wait (weights never depend on the previous
// kernel).  Warps meet only where a row tile is done and the 2C warps of a row
// group join their sums in shared memory, in order of k, so results do not
// depend on timing.  (Bulk copies by a producer warp, one a row and step, took
// 26.7 us for 28672 x 4096: about 130 clocks a copy of 1152 bytes.)  C is 8
// from K = 1280 on; below, a step takes more rows so that every warp has work.
#include <type_traits>

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
    int C;               // chunks of a step
    int TR;              // rows of a step, RG * CW / 2C
    int nkc;             // steps along K
    int nst;             // ring stages of a warp
    bool x_smem;         // x is staged in shared memory
    int red_warp;        // floats of a warp's sums of one row tile (two tiles' sums alternate)
    size_t smem;
};

// false: K is not a positive multiple of 256
bool make_plan(int K, int T, Plan *p) {
    if (K < q4::CHUNK || K % q4::CHUNK) return false;
    const int chunks = K / q4::CHUNK;
    p->C = chunks >= 5 ? 8 : chunks >= 3 ? 4 : chunks;
    p->TR = RG * CW / (2 * p->C);
    p->nkc = (chunks + p->C - 1) / p->C;
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

// XS: x in shared memory; NST: ring stages of a warp
template <bool XS, int NST>
__global__ void __launch_bounds__(THREADS, 1) gemv_q4_kernel(const GemvQ4Args a, const Plan p, const int early) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int r0 = (int)((long long)blockIdx.x * a.N / gridDim.x);
    const int nrows = (int)((long long)(blockIdx.x + 1) * a.N / gridDim.x) - r0;
    const int ntiles = (nrows + p.TR - 1) / p.TR;
    const int groups = a.K / 128;
    const int units = 2 * p.C, cu = warp % units, rg = warp / units, ngroups = CW / units;
    float *red = reinterpret_cast<float *>(smem_raw + (size_t)NST * CW * STAGE);
    f16 *xs = reinterpret_cast<f16 *>(red + 2 * CW * p.red_warp);

    // ---- this warp's ring: rows r0 + tile * TR + rg * 32 .., group kc * units + cu
    const int my_kc = cu < groups ? (groups - cu + units - 1) / units : 0;          // this warp's steps of a row tile
    const int my_tiles = nrows > rg * RG ? (nrows - rg * RG + p.TR - 1) / p.TR : 0;
    const int nsteps = my_kc * my_tiles;
    uint8_t *ring = smem_raw + (size_t)warp * NST * STAGE;
    const uint32_t row_bytes = (uint32_t)groups / 2 * q4::CHUNK_BYTES;
    // sources of this lane's chunk of row g and of the scales of row `lane`, in the next step to request
    const uint8_t *csrc = a.W + (size_t)(r0 + rg * RG) * row_bytes + (size_t)(cu >> 1) * q4::CHUNK_BYTES + 64 * (cu & 1);
    const uint32_t cdst = smem_u32(ring) + g * 64 + ((t4 ^ ((g >> 1) & 3)) << 4);   // rows 8 apart have the same swizzle
    const uint32_t sdst = smem_u32(ring) + CODES + lane * 8;
    const uint32_t tile_step = (uint32_t)p.TR * row_bytes - (uint32_t)(my_kc - 1) * p.C * q4::CHUNK_BYTES;
    int want = 0, want_kc = 0, want_left = nrows - rg * RG;
    uint32_t want_off = 0;                           // ring offset of its slot
    auto request = [&]() {
        if (want < nsteps) {
            // rows past the CTA's repeat its last: their sums are not stored
            const int last = want_left - 1;
            const uint8_t *rows = csrc + 16 * t4;
            const uint32_t d = cdst + want_off;
#pragma unroll
            for (int i = 0; i < RG / 8; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                             :: "r"(d + i * 512), "l"(rows + (size_t)((uint32_t)min(g + 8 * i, last) * (unsigned long long)row_bytes)));
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;"
                         :: "r"(sdst + want_off), "l"(csrc + 128 - 56 * (cu & 1) + (size_t)((uint32_t)min(lane, last) * (unsigned long long)row_bytes)));
            ++want;
            want_off = want_off + STAGE == NST * STAGE ? 0 : want_off + STAGE;
            if (++want_kc == my_kc) {
                want_kc = 0;
                want_left -= p.TR;
                csrc += tile_step;
            } else {
                csrc += p.C * q4::CHUNK_BYTES;
            }
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
        ldx = a.K + X_PAD;
        xp = xs;
        const int per = a.K / 8, n = a.T * per;      // 8-element pieces, a multiple of 32 a row
        for (int i = tid; i < n; i += THREADS) {     // whole warps take part: n % 32 == 0
            const int t = i / per, c = i - t * per;
            const uint4 u = *reinterpret_cast<const uint4 *>(a.x + (size_t)t * a.ldx + c * 8);
            *reinterpret_cast<uint4 *>(xs + (size_t)t * ldx + c * 8) = u;
            // -8 * 2^-24 * sum(x) of the block, where the lanes that sum x's column pair t / 2 look for it
            float v = ((h2lo(u.x) + h2hi(u.x)) + (h2lo(u.y) + h2hi(u.y))) + ((h2lo(u.z) + h2hi(u.z)) + (h2lo(u.w) + h2hi(u.w)));
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            if ((lane & 3) < 2) reinterpret_cast<float *>(tab + 4 * (c >> 2) + (t >> 1))[(t & 1) + 2 * (lane & 3)] = v * (-8.f / 16777216.f);
        }
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
        if (tile < my_tiles) {
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
                    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                    float off1[4], off16[4] = {0.f, 0.f, 0.f, 0.f};
                    if (XS) {
                        const float4 f = tp[kc * units * 16 + 4 * b];
                        off1[0] = f.x; off1[1] = f.y; off1[2] = f.z; off1[3] = f.w;
                    } else {
                        mma(off1, 0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u, x.x, x.z, zero);
                        mma(off16, 0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u, x.y, x.w, zero);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t wg = b == 0 ? w[i][0].x : b == 1 ? w[i][0].y : b == 2 ? w[i][0].z : w[i][0].w;
                        const uint32_t wh = b == 0 ? w[i][1].x : b == 1 ? w[i][1].y : b == 2 ? w[i][1].z : w[i][1].w;
                        const uint32_t sg = wg >> 8, sh = wh >> 8;
                        float s1[4], s16[4];
                        mma(s1, wg & 0x000F000Fu, wh & 0x000F000Fu, sg & 0x000F000Fu, sh & 0x000F000Fu, x.x, x.z, off1);
                        mma(s16, wg & 0x00F000F0u, wh & 0x00F000F0u, sg & 0x00F000F0u, sh & 0x00F000F0u, x.y, x.w, off16);
                        const uint32_t pg = b < 2 ? dd[i][0].x : dd[i][0].y, ph = b < 2 ? dd[i][1].x : dd[i][1].y;
                        const float dg = b & 1 ? h2hi(pg) : h2lo(pg), dh = b & 1 ? h2hi(ph) : h2lo(ph);
                        y[i][0] = fmaf(dg, fmaf(s16[0], 0.0625f, s1[0]), y[i][0]);
                        y[i][1] = fmaf(dg, fmaf(s16[1], 0.0625f, s1[1]), y[i][1]);
                        y[i][2] = fmaf(dh, fmaf(s16[2], 0.0625f, s1[2]), y[i][2]);
                        y[i][3] = fmaf(dh, fmaf(s16[3], 0.0625f, s1[3]), y[i][3]);
                    }
                }
            }
        }
        // ---- the row tile is done: join the 2C warps' sums in order of k
        float *sums = red + (tile & 1) * CW * p.red_warp;
        if (2 * t4 < a.T) {
            float *mine = sums + warp * p.red_warp + 2 * t4 * RED_COL + g;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mine[16 * i] = y[i][0]; mine[16 * i + RED_COL] = y[i][1];
                mine[16 * i + 8] = y[i][2]; mine[16 * i + 8 + RED_COL] = y[i][3];
            }
        }
        __syncthreads();                              // once a tile: its readers are done before the next but one is written
        const int left = nrows - tile * p.TR;
        for (int u = warp; u < ngroups * a.T; u += CW) {
            const int og = u / a.T, t = u - og * a.T, row = og * RG + lane;
            float v = 0.f;
            for (int c = 0; c < units; ++c) v += sums[(og * units + c) * p.red_warp + t * RED_COL + lane];
            if (row < left) a.out[(size_t)t * a.ldo + r0 + tile * p.TR + row] = v * 16777216.f;
        }
    }
    cp_async_wait<0>();
}

}  // namespace

cudaError_t launch_gemv_q4(const GemvQ4Args &a, int num_sms, const Launch &l) {
    Plan p;
    if (a.T < 1 || a.T > 8 || a.N < 1 || num_sms < 1 || !make_plan(a.K, a.T, &p)) return cudaErrorInvalidValue;
    const dim3 grid(a.N < num_sms ? a.N : num_sms), block(THREADS);
    return !p.x_smem      ? launch_kernel(gemv_q4_kernel<false, 4>, grid, block, p.smem, l, a, p, (int)l.pdl)
           : p.nst == 4   ? launch_kernel(gemv_q4_kernel<true, 4>, grid, block, p.smem, l, a, p, (int)l.pdl)
                          : launch_kernel(gemv_q4_kernel<true, 3>, grid, block, p.smem, l, a, p, (int)l.pdl);
}

cudaError_t init_gemv_q4_attributes() {
    cudaError_t e = allow_smem(gemv_q4_kernel<true, 4>, SMEM_CAP);
    if (!e) e = allow_smem(gemv_q4_kernel<true, 3>, SMEM_CAP);
    if (!e) e = allow_smem(gemv_q4_kernel<false, 4>, SMEM_CAP);
    return e;
}

}  // namespace llm
