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
// offset 8 is taken off by starting both sums at -8 sum(x), the product of x
// with a constant fragment, shared by every row of a warp's tile.  Each block
// of 32 k is one sum of at most 32 exact products in fp32, scaled by d in fp32
// and added in fp32: x and the codes are never rounded.
//
// One CTA an SM owns a contiguous run of rows.  Its producer warp streams them
// through a ring of stages, TR rows by C chunks of 256 k, one bulk copy a row
// and stage, each lane its rows, before the dependency wait (weights never
// depend on the previous kernel).  Consumer warp w takes chunk w % C of the 32
// rows (two m16 tiles) of group w / C; the C warps of a group join their sums
// in shared memory in order, so results do not depend on timing.  C is 8 from
// K = 2048 on; below, the stage takes more rows instead so that every warp has
// work.  A row's stage pitch is 64 bytes off a multiple of 128, which spreads
// two rows' 64-byte groups over all banks.
// Every mbarrier wait is bounded (ERRF_WAIT_TIMEOUT, then the CTA winds down).
#include "common.cuh"
#include "launch.cuh"
#include "q4.cuh"
#include "tma.cuh"

namespace llm {

namespace {

constexpr int CW = 8;                        // consumer warps
constexpr int THREADS = (CW + 1) * 32;       // + one producer warp
constexpr int RG = 32;                       // rows of a warp's tile (two m16 tiles)
constexpr int RED_COL = 36;                  // floats between columns of a warp's sums (bank-conflict free)
constexpr int RED_WARP = 8 * RED_COL;
constexpr size_t RED_BYTES = (size_t)2 * CW * RED_WARP * sizeof(float);
constexpr size_t SMEM_CAP = 224 * 1024;
constexpr int X_PAD = 32;                    // elements between rows of x in shared memory beyond K

struct Plan {
    int C;               // chunks of a stage row
    int TR;              // rows of a stage, RG * CW / C
    int nkc;             // stages along K
    int nst;             // ring stages
    uint32_t pitch;      // bytes of a stage row
    uint32_t stage;      // bytes of a stage
    int x_smem;          // x is staged in shared memory
    size_t smem;
};

// false: K is not a positive multiple of 256
bool make_plan(int K, int T, Plan *p) {
    if (K < q4::CHUNK || K % q4::CHUNK) return false;
    const int chunks = K / q4::CHUNK;
    p->C = chunks >= 5 ? 8 : chunks >= 3 ? 4 : chunks;
    p->TR = RG * CW / p->C;
    p->nkc = (chunks + p->C - 1) / p->C;
    p->pitch = (uint32_t)(p->C * q4::CHUNK_BYTES + 63) / 128 * 128 + 64;
    p->stage = p->pitch * (uint32_t)p->TR;
    const size_t x = (size_t)T * (K + X_PAD) * sizeof(f16);
    // x beside three stages or more where it fits (a row tile then reads it
    // from shared memory); else each warp reads its fragments from L2 a stage
    // ahead: with so long a K a CTA has few row tiles to read x again for
    p->x_smem = x + RED_BYTES + 3 * (size_t)p->stage <= SMEM_CAP;
    const size_t room = SMEM_CAP - RED_BYTES - (p->x_smem ? x : 0);
    p->nst = (int)(room / p->stage);
    if (p->nst > 5) p->nst = 5;
    p->smem = (size_t)p->nst * p->stage + RED_BYTES + (p->x_smem ? x : 0);
    return p->nst >= 2;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, const float (&c)[4]) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// XS: x in shared memory
template <bool XS>
__global__ void __launch_bounds__(THREADS, 1) gemv_q4_kernel(const GemvQ4Args a, const Plan p) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    __shared__ uint64_t bars[16];                 // full[8], empty[8]
    __shared__ int s_abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r0 = (int)((long long)blockIdx.x * a.N / gridDim.x);
    const int nrows = (int)((long long)(blockIdx.x + 1) * a.N / gridDim.x) - r0;
    const int ntiles = (nrows + p.TR - 1) / p.TR, nstages = ntiles * p.nkc;
    const int chunks = a.K / q4::CHUNK;
    const size_t row_bytes = (size_t)chunks * q4::CHUNK_BYTES;
    float *red = reinterpret_cast<float *>(smem_raw + (size_t)p.nst * p.stage);
    f16 *xs = reinterpret_cast<f16 *>(smem_raw + (size_t)p.nst * p.stage + RED_BYTES);
    const uint32_t full0 = smem_u32(&bars[0]), empty0 = smem_u32(&bars[8]);
    volatile int *abort = &s_abort;

    if (tid == 0) {
        for (int s = 0; s < p.nst; ++s) {
            mbar_init(full0 + 8u * s, 1);
            mbar_init(empty0 + 8u * s, CW);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_trigger();

    if (warp == CW) {
        // ---- producer
        int issued = 0;
        for (int j = 0; j < nstages; ++j) {
            const int s = j % p.nst, tile = j / p.nkc, kc = j - tile * p.nkc;
            const int rows = min(p.TR, nrows - tile * p.TR);
            const uint32_t bytes = (uint32_t)min(p.C, chunks - kc * p.C) * q4::CHUNK_BYTES;
            bool go = true;
            if (lane == 0) {
                go = j < p.nst || mbar_wait(empty0 + 8u * s, ((j / p.nst) & 1) ^ 1, abort, a.err);
                if (go) mbar_expect_tx(full0 + 8u * s, bytes * (uint32_t)rows);
            }
            if (!__shfl_sync(0xffffffffu, go, 0)) break;
            const uint8_t *src = a.W + (size_t)(r0 + tile * p.TR) * row_bytes + (size_t)kc * p.C * q4::CHUNK_BYTES;
            const uint32_t dst = smem_u32(smem_raw) + (uint32_t)s * p.stage;
            for (int r = lane; r < rows; r += 32)
                bulk_load(dst + (uint32_t)r * p.pitch, src + (size_t)r * row_bytes, bytes, full0 + 8u * s);
            issued = j + 1;
        }
        if (*abort && lane == 0) {
            // let every issued copy land before the shared memory goes away
            for (int j = issued > p.nst ? issued - p.nst : 0; j < issued; ++j)
                for (uint32_t i = 0; i < WAIT_LIMIT && !mbar_try_wait(full0 + 8u * (j % p.nst), (j / p.nst) & 1); ++i) {
                }
        }
        __syncwarp();
    } else {
        // ---- consumers
        const int ci = warp % p.C, rg = warp / p.C, ngroups = CW / p.C;
        const int g = lane >> 2, t4 = lane & 3;
        pdl_wait();
        const f16 *xp = a.x;
        size_t ldx = a.ldx;
        if (XS) {
            for (int i = tid; i < a.T * (a.K / 8); i += CW * 32) {
                const int t = i / (a.K / 8), c = i - t * (a.K / 8);
                cp_async16(xs + (size_t)t * (a.K + X_PAD) + c * 8, a.x + (size_t)t * a.ldx + c * 8, true);
            }
            cp_async_commit();
            cp_async_wait<0>();
            named_sync(1, CW * 32);
            xp = xs;
            ldx = a.K + X_PAD;
        }
        // column g of the N side is row g of x; this lane's eight elements of a block
        const bool col = g < a.T;
        xp += (size_t)(col ? g : 0) * ldx + ci * q4::CHUNK + 8 * t4;
        uint4 bx[8];
        auto load_x = [&](int kc) {
            const bool in = col && kc * p.C + ci < chunks;
#pragma unroll
            for (int b = 0; b < 8; ++b)
                bx[b] = in ? *reinterpret_cast<const uint4 *>(xp + (size_t)kc * p.C * q4::CHUNK + 32 * b)
                           : make_uint4(0u, 0u, 0u, 0u);
        };
        float y[2][4];
        bool alive = true;                        // after a timed-out wait the rest runs without waiting
        if (!XS && nstages > 0) load_x(0);
        for (int j = 0; j < nstages; ++j) {
            const int s = j % p.nst, tile = j / p.nkc, kc = j - tile * p.nkc;
            if (kc == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i) y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
            }
            if (XS) load_x(kc);
            alive = alive && mbar_wait(full0 + 8u * s, (j / p.nst) & 1, abort, a.err);
            const int rows = min(p.TR, nrows - tile * p.TR) - rg * RG;       // of this warp's group
            if (alive && rows > 0 && kc * p.C + ci < chunks) {
                const uint8_t *base = smem_raw + (size_t)s * p.stage + (size_t)(rg * RG + g) * p.pitch + ci * q4::CHUNK_BYTES;
                const bool two = rows > 16;
#pragma unroll
                for (int grp = 0; grp < 2; ++grp) {
                    uint4 w[2][2];                // words of rows g and g + 8 of each tile, blocks 4 grp ..
                    uint2 dd[2][2];               // and their scales
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint8_t *rp = base + (size_t)(16 * i + 8 * h) * p.pitch;
                            w[i][h] = *reinterpret_cast<const uint4 *>(rp + 64 * grp + 16 * t4);
                            dd[i][h] = *reinterpret_cast<const uint2 *>(rp + 128 + 8 * grp);
                        }
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint4 x = bx[4 * grp + b];
                        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                        float off1[4], off16[4];
                        mma(off1, 0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u, x.x, x.z, zero);
                        mma(off16, 0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u, x.y, x.w, zero);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (i == 1 && !two) continue;
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
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8u * s);
            if (!XS && j + 1 < nstages) load_x(kc + 1 == p.nkc ? 0 : kc + 1);
            if (kc + 1 < p.nkc) continue;
            // ---- the row tile is done: join the C warps' sums in chunk order
            float *rw = red + (tile & 1) * CW * RED_WARP;
            if (2 * t4 < a.T) {
                float *mine = rw + warp * RED_WARP + 2 * t4 * RED_COL + g;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mine[16 * i] = y[i][0]; mine[16 * i + RED_COL] = y[i][1];
                    mine[16 * i + 8] = y[i][2]; mine[16 * i + 8 + RED_COL] = y[i][3];
                }
            }
            named_sync(1, CW * 32);
            const int left = nrows - tile * p.TR;
            for (int u = warp; u < ngroups * a.T; u += CW) {
                const int og = u / a.T, t = u - og * a.T, row = og * RG + lane;
                float v = 0.f;
                for (int c = 0; c < p.C; ++c) v += rw[(og * p.C + c) * RED_WARP + t * RED_COL + lane];
                if (row < left && !*abort) a.out[(size_t)t * a.ldo + r0 + tile * p.TR + row] = v * 16777216.f;
            }
        }
    }
    __syncthreads();
}

}  // namespace

cudaError_t launch_gemv_q4(const GemvQ4Args &a, int num_sms, const Launch &l) {
    Plan p;
    if (a.T < 1 || a.T > 8 || a.N < 1 || num_sms < 1 || !make_plan(a.K, a.T, &p)) return cudaErrorInvalidValue;
    const dim3 grid(a.N < num_sms ? a.N : num_sms), block(THREADS);
    return p.x_smem ? launch_kernel(gemv_q4_kernel<true>, grid, block, p.smem, l, a, p)
                    : launch_kernel(gemv_q4_kernel<false>, grid, block, p.smem, l, a, p);
}

cudaError_t init_gemv_q4_attributes() {
    cudaError_t e = allow_smem(gemv_q4_kernel<true>, SMEM_CAP);
    if (!e) e = allow_smem(gemv_q4_kernel<false>, SMEM_CAP);
    return e;
}

}  // namespace llm
