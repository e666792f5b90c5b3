// Decode GEMV over Q4_0 weight rows, 1..8 rows of x: y[t][n] = sum over blocks
// b of d[n][b] * sum over k in b of (c[n][k] - 8) * x[t][k], fp32 sums.
// One warp a weight row: lane w of a 256-element chunk takes its word w, the
// eight elements 128 (w / 16) + 32 (w % 4) + 8 (w / 4 % 4) + {0..7}.
#include "common.cuh"
#include "launch.cuh"
#include "q4.cuh"

namespace llm {

namespace {

constexpr int WARPS = 8;

template <int T>
__global__ void __launch_bounds__(WARPS * 32) gemv_q4_kernel(const GemvQ4Args a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long n = (long long)blockIdx.x * WARPS + warp;
    if (n >= a.N) return;
    const uint8_t *row = a.W + (size_t)n * (a.K / q4::CHUNK * q4::CHUNK_BYTES);
    const int off = 128 * (lane >> 4) + 32 * (lane & 3) + 8 * ((lane >> 2) & 3);
    float acc[T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = 0.f;
    for (int ch = 0; ch < a.K / q4::CHUNK; ++ch) {
        const uint8_t *c = row + (size_t)ch * q4::CHUNK_BYTES;
        const uint32_t word = reinterpret_cast<const uint32_t *>(c)[lane];
        const float d = __half2float(reinterpret_cast<const __half *>(c + 128)[off >> 5]);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint4 xv = *reinterpret_cast<const uint4 *>(a.x + (size_t)t * a.ldx + ch * q4::CHUNK + off);
            const __half *xh = reinterpret_cast<const __half *>(&xv);
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += (float)((int)((word >> q4::shift_of(e)) & 15u) - 8) * __half2float(xh[e]);
            acc[t] += d * s;
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const float y = warp_sum(acc[t]);
        if (lane == 0) a.out[(size_t)t * a.ldo + n] = y;
    }
}

}  // namespace

cudaError_t launch_gemv_q4(const GemvQ4Args &a, int num_sms, const Launch &l) {
    if (a.T < 1 || a.T > 8 || a.N < 1 || a.K < q4::CHUNK || a.K % q4::CHUNK) return cudaErrorInvalidValue;
    const dim3 grid((a.N + WARPS - 1) / WARPS), block(WARPS * 32);
    switch (a.T) {
#define Q4_CASE(TV) case TV: return launch_kernel(gemv_q4_kernel<TV>, grid, block, 0, l, a);
        Q4_CASE(1) Q4_CASE(2) Q4_CASE(3) Q4_CASE(4) Q4_CASE(5) Q4_CASE(6) Q4_CASE(7) Q4_CASE(8)
#undef Q4_CASE
    }
    return cudaErrorInvalidValue;
}

}  // namespace llm
