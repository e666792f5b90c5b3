// Decode GEMV over Q4_0 weight rows for 1..8 rows of x: y[t][n] = sum over
// blocks b of d[n][b] * sum over k in b of (c[n][k] - 8) * x[t][k], the linear
// layers of a decode step whose weights are held in four bits.
//
// Bound by HBM: 9/16 byte a weight, each read once, leaves 10 weights a clock
// to an SM sub-partition at the copy bandwidth, for which scalar products on
// the CUDA cores are too many instructions.  So they run on mma.sync m16n8k16
// (f16, f32 sums; 8 clocks of a sub-partition on this GPU, where logic, shift
// and fp16-pair instructions take 2 and FFMA 1): 16 weight rows are the M side,
// the rows of x the N side (its other columns are not used).  A word of eight
// codes becomes four fragment registers by one shift and, for each, one logic
// instruction and one exact fp16 subtraction, which leave c - 8 (q4::Widen).
// Each block of 32 k is one sum of 32 exact products in fp32, scaled by d in
// fp32 and added in fp32: x and the codes are never rounded.  (Codes as fp16 subnormals c * 2^-24, with
// 8 sum(x) taken off a block's sum, save the subtractions, but the tensor
// cores truncate their addends to the largest one's exponent: y was 9e-7 off
// instead of 1e-7, and x needed scaling and a table of sums before the first
// product.)
//
// One CTA an SM owns a contiguous run of rows.  Its 16 warps are 16 / units
// row groups of `units` warps: a group takes every (16 / units)-th tile of 32
// rows (two m16 tiles), warp cu of it the 256-element chunks cu, cu + units, ..
// of K, each in two steps of 128.  A warp brings its codes and scales itself,
// with cp.async, through a ring of its own (2 KB of codes a step, the scales of
// a chunk with its first; the first steps before the dependency wait where the
// launch overlaps the previous kernel: weights never depend on it).  The warps
// of a row group join their sums in shared memory, in a fixed order, so results
// do not depend on timing.  More units spread few rows over all warps, fewer
// meet less often: the launcher takes the split with the fewest chunks a warp,
// counting a meeting as a quarter of one (with 16 units throughout,
// 128256 x 4096 took 83 us, a quarter of it in meetings).
//
// The QKV epilogue rotates pairs of rows and appends to the cache.  Its rows are
// handed out in blocks of 32, one tile each, so the warp that joins a tile holds
// one Q4_0 block of the cache, an element a lane, and encodes it there: in a
// decode step of the 8B shape that is 2.3 us a layer less than a kernel of its
// own, and whole tiles alone are worth 2%.
//
// Measured, calls in a row in a captured graph, one row of x where not said
// otherwise, and the time the bytes take at the copy bandwidth (6.79 TB/s): 4096 x
// 4096 4.3 us (1.4), 28672 x 4096 14.8 (9.7), 4096 x 14336 with 8 rows 10.5 (4.9),
// 128256 x 4096 55.5 (43.5; 5.3 TB/s).  2.5 us of each go by before the first
// product and after the last; in between (128256 x 4096) the schedulers issue in
// 60% of their clocks (ALU 47%, FMA 40%, tensor 27% of theirs) with four warps
// each, which wait for the pipes and the shared-memory queue and hardly for memory.
//
// What was slower or no faster: bulk copies by a producer warp, one a row and
// step (28672 x 4096 26.7 us: 130 clocks a copy of 1152 bytes); the columns that a
// single row of x leaves unused taking other blocks (57.1 us for 128256 x 4096, as
// without the odd columns' sums, 57.2); two CTAs of half the warps an SM; steps of
// 16 rows and whole chunks, whose copies run along the rows (64 lines a chunk
// instead of 112; with four stages each 55.9 instead of 57.3 us for 128256 x 4096,
// but 16.8 instead of 16.1 for 28672 x 4096 and 11.9 instead of 11.2 for 4096 x
// 14336 with the early requests); the chunks that 16 warps share unevenly (56 of a
// K of 14336) cut into halves (11.8 instead of 11.0: a step that may be either half
// is scheduled worse than the two of a chunk); one kernel for all epilogues, its
// products kept in the instruction cache (8B decode 662 tok/s instead of 676); one
// m16 tile where the second has no rows (663).
#include "common.cuh"
#include "launch.cuh"
#include "q4.cuh"

namespace llm {

namespace {

constexpr int CW = 16;                       // warps
constexpr int THREADS = CW * 32;
constexpr int RG = 32;                       // rows of a warp's tile (two m16 tiles)
constexpr int CODES = RG * 64;               // bytes of a step's codes in a warp's ring
constexpr int SCALES = RG * 16;              // bytes of a chunk's scales
// Ring stages of a warp: 64 KB of codes ahead on an SM.  A fourth delays x,
// which queues behind the weights requested before it (4096 x 14336 11.6 us
// instead of 11.0, 28672 x 4096 17.6 instead of 17.1, 8B decode 568 tok/s
// instead of 577).
constexpr int NST = 3;
constexpr int SC_SLOTS = 3;                  // chunks whose scales are held: NST - 1 steps ahead touch at most three
constexpr size_t RING_BYTES = (size_t)CW * (NST * CODES + SC_SLOTS * SCALES);
constexpr int RED_COL = 36;                  // floats between columns of a warp's sums (bank-conflict free)
constexpr size_t SMEM_CAP = 224 * 1024;
constexpr int X_PAD = 32;                    // elements between rows of x in shared memory beyond K

struct Plan {
    int log_units;       // units = 2^log_units warps share a row tile's K
    int run, longer;     // a CTA's rows: run row units, one more for the first `longer` CTAs
    bool x_smem;         // x is staged in shared memory
    int red_warp;        // floats of a warp's sums of one row tile (two tiles' sums alternate)
    size_t smem;
};

// false: K is not a positive multiple of 256
bool make_plan(int N, int K, int T, int ctas, int unit, Plan *p) {
    if (K < q4::CHUNK || K % q4::CHUNK) return false;
    p->run = N / unit / ctas;
    p->longer = N / unit % ctas;
    const int chunks = K / q4::CHUNK, rows = (p->run + (p->longer > 0)) * unit, tiles = (rows + RG - 1) / RG;
    long long best = 0;
    for (int lu = 4; lu >= 0; --lu) {
        const int u = 1 << lu;
        const long long mine = (tiles + CW / u - 1) / (CW / u), cost = mine * (4LL * ((chunks + u - 1) / u) + 1);
        if (u == CW || cost < best) { best = cost; p->log_units = lu; }
    }
    p->red_warp = (T + 1) / 2 * 2 * RED_COL;
    const size_t red = (size_t)2 * CW * p->red_warp * sizeof(float);
    const size_t x = (size_t)T * (K + X_PAD) * sizeof(f16);
    // x beside the rings where it fits; else each warp reads its fragments from
    // L2 a step ahead: with so long a K a CTA has few row tiles to read x again for
    p->x_smem = x + red + RING_BYTES <= SMEM_CAP;
    p->smem = RING_BYTES + red + (p->x_smem ? x : 0);
    return true;
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma0(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

constexpr int row_unit(int epi) { return epi == EPI_SWIGLU ? 2 * GU_GROUP : epi == EPI_QKV ? q4::BLOCK : 1; }

// XS: x in shared memory; ONE: one row of x, so the
// odd columns' sums are not kept (28672 x 4096 17.7 us, with them 18.2)
template <int EPI, bool XS, bool ONE>
__global__ void __launch_bounds__(THREADS, 1) gemv_q4_kernel(const GemvQ4Args a, const Plan p, const int early) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    // the warp's number from a shuffle: what follows from it is then known to be the same for its lanes
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    constexpr int UNIT = row_unit(EPI);              // rows kept together
    // no divisions here: a CTA that starts when its SM falls free has all this ahead of its first product
    const int bx0 = (int)blockIdx.x, r0 = (bx0 * p.run + min(bx0, p.longer)) * UNIT;
    const int nrows = (p.run + (bx0 < p.longer)) * UNIT;
    __shared__ float s_r[8];                         // the rows' RMSNorm factors
    __shared__ int s_pos[8], s_seq[8];               // QKV: their cells, -1 where outside the cache
    __shared__ float s_sq[EPI == EPI_RESID ? CW : 1][8];   // sums of h^2 by row group
    const int chunks = a.K / q4::CHUNK;
    const int lu = p.log_units, units = 1 << lu, cu = warp & (units - 1), rg = warp >> lu, TR = RG * CW >> lu;
    static_assert(RG * CW == 512, "TR = 2^(9 - lu)");
    float *red = reinterpret_cast<float *>(smem_raw + RING_BYTES);
    f16 *xs = reinterpret_cast<f16 *>(red + 2 * CW * p.red_warp);

    // ---- this warp's ring: rows r0 + (tile * ngroups + rg) * 32 .., chunk kc * units + cu
    const int my_kc = (chunks - cu + units - 1) >> lu;                                // this warp's chunks of a row tile
    const int ntiles = nrows > rg * RG ? (nrows - rg * RG + TR - 1) >> (9 - lu) : 0;   // its row group's tiles
    uint8_t *ring = smem_raw + (size_t)warp * (NST * CODES + SC_SLOTS * SCALES);
    const uint32_t row_bytes = (uint32_t)chunks * q4::CHUNK_BYTES;
    // source of the next chunk to request (the warp's) and this lane's offsets from it: rows g, g + 8, .. of the codes
    // and row `lane` of the scales
    const uint8_t *src = a.W + (size_t)(r0 + rg * RG) * row_bytes + (size_t)cu * q4::CHUNK_BYTES;
    uint32_t coff[RG / 8];
#pragma unroll
    for (int i = 0; i < RG / 8; ++i) coff[i] = (uint32_t)(g + 8 * i) * row_bytes + 16 * t4;
    const uint32_t soff = (uint32_t)lane * row_bytes + 128;
    const uint32_t cdst = smem_u32(ring) + g * 64 + ((t4 ^ ((g >> 1) & 3)) << 4);   // rows 8 apart have the same swizzle
    const uint32_t sdst = smem_u32(ring) + NST * CODES + lane * 16;
    const int kc_step = units * q4::CHUNK_BYTES;
    const long long tile_step = (long long)TR * row_bytes - (long long)(my_kc - 1) * kc_step;
    int want = my_kc * ntiles, want_kc = my_kc, want_left = nrows - rg * RG;   // chunks, chunks of the tile and rows not requested
    uint32_t want_c = 0, want_s = 0;                 // ring offsets of the next step's codes and the next chunk's scales
    auto request = [&](int half) {
        if (want > 0) {
            if (want_left >= RG) {
#pragma unroll
                for (int i = 0; i < RG / 8; ++i)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                 :: "r"(cdst + want_c + i * 512), "l"(src + 64 * half + coff[i]));
                if (half == 0) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(sdst + want_s), "l"(src + soff));
            } else {
                // rows past the CTA's repeat its last: their sums are not stored
                const uint32_t last = (uint32_t)(want_left - 1) * row_bytes;
#pragma unroll
                for (int i = 0; i < RG / 8; ++i)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                 :: "r"(cdst + want_c + i * 512), "l"(src + 64 * half + min(coff[i], last + 16 * t4)));
                if (half == 0)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(sdst + want_s), "l"(src + min(soff, last + 128)));
            }
            want_c = want_c == (NST - 1) * CODES ? 0 : want_c + CODES;
            if (half == 1) {
                --want;
                want_s = want_s == (SC_SLOTS - 1) * SCALES ? 0 : want_s + SCALES;
                if (--want_kc == 0) {
                    want_kc = my_kc;
                    want_left -= TR;
                    src += tile_step;
                } else {
                    src += kc_step;
                }
            }
        }
        cp_async_commit();
    };
    if (early)                                       // beside the previous kernel: weights never depend on it
#pragma unroll
        for (int j = 0; j < NST - 1; ++j) request(j & 1);
    pdl_wait();
    pdl_trigger();

    // ---- x: column g of the N side is row g of x (columns from T on repeat row 0, their sums are not stored)
    const f16 *xp = a.x;
    int ldx = a.ldx;
    // a row's sums of squares and cell are asked for at once, x right behind them, and all are waited for together
    constexpr int SSQ = 8;
    float part[SSQ];
    int ps = 0, sq = 0;
    const bool stats = warp < a.T;
    if (stats) {
        if (EPI == EPI_QKV) { ps = a.pos[warp]; sq = a.seq[warp]; }
#pragma unroll
        for (int j = 0; j < SSQ; ++j) {
            const int i = lane + 32 * j;
            part[j] = a.ss_in && i < a.n_ss_in ? a.ss_in[(size_t)warp * a.n_ss_in + i] : 0.f;
        }
    }
    auto finish_stats = [&]() {
        if (!stats) return;
        float r = 1.f;
        if (a.ss_in) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < SSQ; ++j) ss += part[j];
            for (int i = lane + 32 * SSQ; i < a.n_ss_in; i += 32) ss += a.ss_in[(size_t)warp * a.n_ss_in + i];
            r = 1.f / sqrtf(warp_sum(ss) / (float)a.K + a.eps);
        }
        if (lane == 0) s_r[warp] = r;
        if (EPI == EPI_QKV && lane == 0) {
            const bool ok = ps >= 0 && ps < a.kv.n_ctx && sq >= 0 && sq < a.kv.n_seq;
            if (!ok && blockIdx.x == 0) raise_error(a.err, ERRF_BAD_INDEX);
            s_pos[warp] = ok ? ps : -1;
            s_seq[warp] = sq;
        }
    };
    if (XS) {
        const int per = a.K / 8, n = a.T * per;      // 16-byte pieces of x
        constexpr int HOLD = 4;                      // pieces a thread asks for before the ring's first steps
        uint4 held[HOLD];
        auto piece = [&](int i) {
            return *reinterpret_cast<const uint4 *>(ONE ? a.x + 8 * i : a.x + (size_t)(i / per) * a.ldx + (i % per) * 8);
        };
        auto put = [&](int i, const uint4 &u) {
            *reinterpret_cast<uint4 *>(ONE ? xs + 8 * i : xs + (size_t)(i / per) * (a.K + X_PAD) + (i % per) * 8) = u;
        };
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (tid + j * THREADS < n) held[j] = piece(tid + j * THREADS);
        if (!early)                                  // behind x in the queue, before x is waited for
            for (int j = 0; j < NST - 1; ++j) request(j & 1);
#pragma unroll
        for (int j = 0; j < HOLD; ++j)
            if (tid + j * THREADS < n) put(tid + j * THREADS, held[j]);
#pragma unroll 4
        for (int i = tid + HOLD * THREADS; i < n; i += THREADS) put(i, piece(i));
        ldx = a.K + X_PAD;
        xp = xs;
    } else if (!early) {
        for (int j = 0; j < NST - 1; ++j) request(j & 1);
    }
    finish_stats();
    __syncthreads();
    xp += (size_t)(g < a.T ? g : 0) * ldx + cu * q4::CHUNK + 8 * t4;
    uint4 bx[4];                                     // !XS: the next step's x
    auto load_x = [&](int k) {
#pragma unroll
        for (int b = 0; b < 4; ++b) bx[b] = *reinterpret_cast<const uint4 *>(xp + (size_t)k + 32 * b);
    };
    if (!XS && my_kc * ntiles > 0) load_x(0);

    const q4::Widen wd;
    float ssq[EPI == EPI_RESID ? 8 : 1];             // RESID: this warp's sums of h^2, by its rows of x in turn
#pragma unroll
    for (float &v : ssq) v = 0.f;
    uint32_t cslot = 0, sslot = 0;
    const uint8_t *wr = ring + g * 64 + ((t4 ^ ((g >> 1) & 3)) << 4), *dr = ring + NST * CODES + g * 16;
    for (int tile = 0; tile < ntiles; ++tile) {
        // what the epilogue adds to this lane's row, for the warp's first row of x, is asked for ahead of the products
        const int row = (tile * (CW >> lu) + rg) * RG + lane, n = r0 + row;
        const bool in = row < nrows;
        auto turn = [&](int t) {                     // QKV: the row pair's rotation
            const int hd = a.kv.head_dim;
            return EPI == EPI_QKV && in && s_pos[t] >= 0 && n < a.n_q + a.n_kv
                       ? a.rope[(size_t)s_pos[t] * (hd / 2) + (n < a.n_q ? n : n - a.n_q) % hd / 2]
                       : make_float2(1.f, 0.f);
        };
        float2 cs = make_float2(1.f, 0.f);
        float h0 = 0.f, gain = 0.f;
        if (cu < a.T) {
            if (EPI == EPI_QKV) cs = turn(cu);
            if (EPI == EPI_RESID && in) {
                h0 = a.hres[(size_t)cu * a.ldh + n];
                if (a.xg_out) gain = a.gain_next[n];
            }
        }
        float y[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
        for (int kc = 0; kc < my_kc; ++kc) {
            const int k0 = kc * units * q4::CHUNK;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                cp_async_wait<NST - 2>();
                __syncwarp();
                request((half + NST - 1) & 1);       // NST - 1 steps on, into the slot read in the step before
                uint4 xv[4];
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    xv[b] = XS ? *reinterpret_cast<const uint4 *>(xp + k0 + 128 * half + 32 * b) : bx[b];
                if (!XS) load_x(half == 0 ? k0 + 128 : kc + 1 < my_kc ? k0 + units * q4::CHUNK : 0);
                uint4 w[2][2];                       // words of rows g and g + 8 of each m16 tile
                uint2 dd[2][2];                      // and their scales
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        w[i][h] = *reinterpret_cast<const uint4 *>(wr + cslot + (16 * i + 8 * h) * 64);
                        dd[i][h] = *reinterpret_cast<const uint2 *>(dr + sslot + (16 * i + 8 * h) * 16 + 8 * half);
                    }
                cslot = cslot == (NST - 1) * CODES ? 0 : cslot + CODES;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint4 x = xv[b];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t wg = b == 0 ? w[i][0].x : b == 1 ? w[i][0].y : b == 2 ? w[i][0].z : w[i][0].w;
                        const uint32_t wh = b == 0 ? w[i][1].x : b == 1 ? w[i][1].y : b == 2 ? w[i][1].z : w[i][1].w;
                        const uint32_t sg = wg >> 8, sh = wh >> 8;
                        const uint32_t pg = b < 2 ? dd[i][0].x : dd[i][0].y, ph = b < 2 ? dd[i][1].x : dd[i][1].y;
                        const float dg = b & 1 ? h2hi(pg) : h2lo(pg), dh = b & 1 ? h2hi(ph) : h2lo(ph);
                        float s[4];
                        mma0(s, wd.low(wg), wd.low(wh), wd.low(sg), wd.low(sh), x.x, x.z);
                        mma(s, wd.high(wg), wd.high(wh), wd.high(sg), wd.high(sh), x.y, x.w);
                        y[i][0] = fmaf(dg, s[0], y[i][0]);
                        if (!ONE) y[i][1] = fmaf(dg, s[1], y[i][1]);
                        y[i][2] = fmaf(dh, s[2], y[i][2]);
                        if (!ONE) y[i][3] = fmaf(dh, s[3], y[i][3]);
                    }
                }
            }
            sslot = sslot == (SC_SLOTS - 1) * SCALES ? 0 : sslot + SCALES;
        }
        // ---- the row tile is done: join the group's sums, in a fixed order
        float *sums = red + ((tile & 1) * CW + rg * units) * p.red_warp;
        if (2 * t4 < a.T) {
            float *mine = sums + cu * p.red_warp + 2 * t4 * RED_COL + g;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mine[16 * i] = y[i][0];
                mine[16 * i + 8] = y[i][2];
                if (!ONE) { mine[16 * i + RED_COL] = y[i][1]; mine[16 * i + 8 + RED_COL] = y[i][3]; }
            }
        }
        // once a tile: the readers of these sums are done before the next but one overwrites them
        if (units > 1) asm volatile("bar.sync %0, %1;" :: "r"(rg + 1), "r"(units * 32) : "memory");
        else __syncwarp();
        int q = 0;
        for (int t = cu; t < a.T; t += units, ++q) {
            if (t != cu) {
                if (EPI == EPI_QKV) cs = turn(t);
                if (EPI == EPI_RESID && in) h0 = a.hres[(size_t)t * a.ldh + n];
            }
            float v = 0.f;
            if (units >= 4) {
                float v4[4] = {0.f, 0.f, 0.f, 0.f};
                for (int c = 0; c < units; c += 4)
#pragma unroll
                    for (int k = 0; k < 4; ++k) v4[k] += sums[(c + k) * p.red_warp + t * RED_COL + lane];
                v = (v4[0] + v4[1]) + (v4[2] + v4[3]);
            } else {
                for (int c = 0; c < units; ++c) v += sums[c * p.red_warp + t * RED_COL + lane];
            }
            v *= s_r[t];
            if (EPI == EPI_QKV) {
                // lane pairs hold the elements of a rotation, 2i and 2i + 1
                const float w = __shfl_xor_sync(0xffffffffu, v, 1), x = v;
                if (n < a.n_q + a.n_kv) v = lane & 1 ? fmaf(v, cs.x, w * cs.y) : fmaf(v, cs.x, -w * cs.y);
                const float up = __shfl_down_sync(0xffffffffu, v, 1);
                if (a.kv.k4 && n >= a.n_q) {         // the warp's 32 rows are one block: whole blocks are kept together
                    const bool is_k = n < a.n_q + a.n_kv;
                    float d;
                    int code;
                    if (__any_sync(0xffffffffu, q4::encode_lane(v, d, code))) {
                        // next to a border: from the exact products (a value is exact as it is)
                        const float up = fabsf(d) > q4::TINY ? 1.f : q4::RAISE, xs = x * up, ws = (lane & 1 ? w : -w) * up;
                        q4::encode_lane(is_k ? q4::two_prod(xs, cs.x) + q4::two_prod(ws, cs.y) : q4::Pair{xs, 0.f}, d, code);
                        d /= up;
                    }
                    uint32_t word = (uint32_t)code << q4::shift_of(lane & 7);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
                    if (s_pos[t] >= 0) {
                        if (f16_bad(v)) raise_error(a.err, ERRF_F16_RANGE);
                        const int hd = a.kv.head_dim, c = n - a.n_q - (is_k ? 0 : a.n_kv), head = c / hd, blk = (c - head * hd) / 32;
                        const size_t row = (size_t)s_seq[t] * a.kv.seq_stride + ((size_t)head * a.kv.n_ctx + s_pos[t]) * hd;
                        if ((lane & 7) == 0)
                            reinterpret_cast<uint32_t *>((is_k ? a.kv.k4 : a.kv.v4) + row / 2)[(lane >> 3) * (hd / 32) + blk] = word;
                        if (lane == 0) (is_k ? a.kv.kd : a.kv.vd)[row / 32 + blk] = f2h(d);
                    }
                } else if (in && s_pos[t] >= 0) {
                    if (n < a.n_q) {
                        a.q_out[(size_t)t * a.n_q + n] = v;
                    } else if (!(lane & 1)) {
                        const bool is_k = n < a.n_q + a.n_kv;
                        const int hd = a.kv.head_dim, c = n - a.n_q - (is_k ? 0 : a.n_kv), head = c / hd;
                        const size_t off = (size_t)s_seq[t] * a.kv.seq_stride + ((size_t)head * a.kv.n_ctx + s_pos[t]) * hd + (c - head * hd);
                        if (a.kv.k8) {
                            *reinterpret_cast<uint16_t *>((is_k ? a.kv.k8 : a.kv.v8) + off) = pack_e4m3x2(v, up);
                        } else {
                            if (f16_bad(v) || f16_bad(up)) raise_error(a.err, ERRF_F16_RANGE);
                            *reinterpret_cast<uint32_t *>((is_k ? a.kv.k : a.kv.v) + off) = pack_h2(v, up);
                        }
                    }
                }
            } else if (EPI == EPI_STORE) {
                if (in) a.out[(size_t)t * a.ldo + n] = v;
            } else if (EPI == EPI_RESID) {
                float h = 0.f;
                if (in) {
                    h = h0 + v;
                    a.hres[(size_t)t * a.ldh + n] = h;
                    if (a.xg_out) {
                        const float xg = h * gain;
                        if (f16_bad(xg)) raise_error(a.err, ERRF_F16_RANGE);
                        a.xg_out[(size_t)t * a.ldxg + n] = f2h(xg);
                    }
                }
                const float sq = warp_sum(h * h);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k == q) ssq[k] += sq;
            } else {
                // a gate row's lane takes its up row from the lane GU_GROUP on
                const float up = __shfl_down_sync(0xffffffffu, v, GU_GROUP);
                if (in && !(lane & GU_GROUP)) {
                    const float u = silu(v) * up;
                    if (f16_bad(u)) raise_error(a.err, ERRF_F16_RANGE);
                    a.u_out[(size_t)t * a.ldu + n / (2 * GU_GROUP) * GU_GROUP + (lane & (GU_GROUP - 1))] = f2h(u);
                }
            }
        }
    }
    if (EPI == EPI_RESID && a.xg_out && units == CW) {
        // one row group: the warp of a row of x holds the CTA's sum
        if (cu < a.T && lane == 0) a.ss_out[(size_t)cu * gridDim.x + blockIdx.x] = ssq[0];
    } else if (EPI == EPI_RESID && a.xg_out) {
        // this CTA's sums of squares of the new h, in a fixed order
        int q = 0;
        for (int t = cu; t < a.T; t += units, ++q) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k == q) v = ssq[k];
            if (lane == 0) s_sq[rg][t] = v;
        }
        __syncthreads();
        if (tid < a.T) {
            float v = 0.f;
            for (int k = 0; k < CW >> lu; ++k) v += s_sq[k][tid];
            a.ss_out[(size_t)tid * gridDim.x + blockIdx.x] = v;
        }
    }
    cp_async_wait<0>();
}

}  // namespace

int gemv_q4_ctas(int epi, int N, int num_sms) {
    const int units = N / row_unit(epi);
    return units < num_sms ? units : num_sms;
}

// early: with l.pdl, weights may be read before the previous kernel is done
cudaError_t launch_gemv_q4(int epi, const GemvQ4Args &a, int num_sms, const Launch &l, bool early) {
    Plan p;
    const int ctas = gemv_q4_ctas(epi, a.N, num_sms);
    if (a.T < 1 || a.T > 8 || ctas < 1 || a.N % row_unit(epi) || !make_plan(a.N, a.K, a.T, ctas, row_unit(epi), &p))
        return cudaErrorInvalidValue;
    const dim3 grid(ctas), block(THREADS);
#define Q4_GEMV1(E, XS)                                                                              \
    return a.T == 1 ? launch_kernel(gemv_q4_kernel<E, XS, true>, grid, block, p.smem, l, a, p, (int)early) \
                    : launch_kernel(gemv_q4_kernel<E, XS, false>, grid, block, p.smem, l, a, p, (int)early);
#define Q4_GEMV(E)                       \
    if (epi == E) {                      \
        if (p.x_smem) Q4_GEMV1(E, true)  \
        Q4_GEMV1(E, false)               \
    }
    Q4_GEMV(EPI_STORE) Q4_GEMV(EPI_RESID) Q4_GEMV(EPI_QKV) Q4_GEMV(EPI_SWIGLU)
#undef Q4_GEMV
#undef Q4_GEMV1
    return cudaErrorInvalidValue;
}

cudaError_t init_gemv_q4_attributes() {
    cudaError_t e = cudaSuccess;
#define Q4_GEMV_ATTR1(E, XS)                                      \
    if (!e) e = allow_smem(gemv_q4_kernel<E, XS, true>, SMEM_CAP); \
    if (!e) e = allow_smem(gemv_q4_kernel<E, XS, false>, SMEM_CAP);
#define Q4_GEMV_ATTR(E) Q4_GEMV_ATTR1(E, true) Q4_GEMV_ATTR1(E, false)
    Q4_GEMV_ATTR(EPI_STORE) Q4_GEMV_ATTR(EPI_RESID) Q4_GEMV_ATTR(EPI_QKV) Q4_GEMV_ATTR(EPI_SWIGLU)
#undef Q4_GEMV_ATTR
#undef Q4_GEMV_ATTR1
    return e;
}

}  // namespace llm
