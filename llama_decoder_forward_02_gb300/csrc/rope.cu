// Rotary position tables: cos and sin of position times frequency, the
// frequencies scaled for contexts beyond the trained one ("LLama.cpp — how it
// works", "Context creation": the rope_freq_base, rope_freq_scale and YaRN
// parameters of llama_context).
//
// Angles are kept as fractions of a turn in 64-bit fixed point, where a position's
// angle is one integer product that drops whole turns by itself.  A frequency is
// float64's, rounded to 2^-64 of a turn, so an angle is off by 2^-53 of it and by
// 2^-65 of a turn times the position (2^-35 of a turn at position 2^30).  Only for a pair
// slower than 2^-41 of a turn a position (theta times factor above 10^11) does that
// leave small sines with fewer bits than a float's.
// The nearest of 512 directions e^(ia), kept as pairs of floats,
// is turned by the rest |d| <= pi / 512, whose sine and cosine - 1 are two terms of
// their series (the next is below 2^-50):
//   cos(a + d) = cos a + (cos a (cos d - 1) - sin a sin d),  and sin alike.
// The bracket is at most 0.0062, so its float32 error adds 2^-30 to the one rounding
// of the result.
//
// Bound by the writing of 8 bytes a pair: 131072 positions of 64 pairs take 12.9 us,
// 78% of the copy bandwidth, 4096 of 32 pairs 2.0 us, a launch.  With sincos in float64,
// which this GPU does at 1/60 of float32's rate, the first took 677 us.
#include <cmath>

#include "common.cuh"
#include "launch.cuh"

namespace llm {

namespace {

constexpr int MAX_PAIRS = 64, THREADS = 256, DIRS = 512;
constexpr double PI = 3.14159265358979323846;

// cos and sin of k / 512 turns as pairs of floats.
struct alignas(16) Direction { float c, cl, s, sl; };
struct Directions { Direction d[DIRS]; };

constexpr double series(double x, bool sine) {       // |x| <= pi / 4
    double term = sine ? x : 1.0, sum = term;
    for (int n = sine ? 2 : 1; n < 24; n += 2) {
        term *= -x * x / (n * (n + 1.0));
        sum += term;
    }
    return sum;
}
constexpr Directions make_directions() {
    Directions t{};
    for (int k = 0; k < DIRS; ++k) {
        const int quarter = k / (DIRS / 4), r = k % (DIRS / 4);
        const bool swap = r > DIRS / 8;              // above an eighth of a turn: from the other axis
        const double x = (swap ? DIRS / 4 - r : r) * (2 * PI / DIRS);
        const double c0 = series(x, swap), s0 = series(x, !swap);
        const double c = quarter == 0 ? c0 : quarter == 1 ? -s0 : quarter == 2 ? -c0 : s0;
        const double s = quarter == 0 ? s0 : quarter == 1 ? c0 : quarter == 2 ? -s0 : -c0;
        t.d[k].c = (float)c;
        t.d[k].cl = (float)(c - (double)(float)c);
        t.d[k].s = (float)s;
        t.d[k].sl = (float)(s - (double)(float)s);
    }
    return t;
}
__device__ const Directions directions = make_directions();

struct Frequencies {
    unsigned long long f[MAX_PAIRS];                 // turns a position, in 2^-64
    float scale, scale_lo;                           // the factor as a pair
};

// The angle phase / 2^64 turns.
__device__ __forceinline__ float2 turn_of(const Direction *dirs, unsigned long long phase, float scale, float scale_lo) {
    constexpr int LOW = 55;                          // bits below a direction
    const unsigned long long at = phase + (1ull << (LOW - 1));
    const Direction t = dirs[at >> LOW];
    // the rest in [-2^54, 2^54): 23 bits and sign, then 23 of the 32 below (each exact as a float by its bits)
    const long long rest = (long long)(at & ((1ull << LOW) - 1)) - (1ll << (LOW - 1));
    const float hi = __int_as_float(0x4B400000 + (int)(rest >> 32)) - 12582912.f;
    const float lo = __uint_as_float(0x4B000000u | ((unsigned)rest >> 9)) - 8388608.f;
    const float d = fmaf(hi, (float)(2 * PI / 4294967296.0), lo * (float)(2 * PI / 36028797018963968.0));
    const float d2 = d * d;
    const float sd = fmaf(d * d2, fmaf(d2, (float)(1.0 / 120), (float)(-1.0 / 6)), d), cd = d2 * fmaf(d2, (float)(1.0 / 24), -0.5f);
    const float c = t.cl + fmaf(t.c, cd, -t.s * sd), s = t.sl + fmaf(t.s, cd, t.c * sd);
    // times the factor, the large product exact in the sum
    return make_float2(fmaf(t.c, scale, fmaf(scale, c, t.c * scale_lo)), fmaf(t.s, scale, fmaf(scale, s, t.s * scale_lo)));
}

// Rows of `width` pairs (even), of which those from `pairs` on do not turn; a thread
// takes two pairs of every step'th row.  T: also out_t[j * n_pos + i] = out[i][j].
template <bool T>
__global__ void __launch_bounds__(THREADS) rope_table_kernel(const __grid_constant__ Frequencies fr, int pairs, int width, int pos0,
                                                             int n_pos, float4 *out, float2 *out_t) {
    __shared__ Direction dirs[DIRS];
    for (int i = threadIdx.x; i < DIRS; i += THREADS) dirs[i] = directions.d[i];
    const int units = width / 2, u = threadIdx.x % units, per = THREADS / units, j = 2 * u;
    const int step = gridDim.x * per;
    int row = blockIdx.x * per + threadIdx.x / units;
    const bool turns = j < pairs;                    // pairs is even
    const unsigned long long f0 = turns ? fr.f[j] : 0ull, f1 = turns ? fr.f[j + 1] : 0ull;
    const float scale = turns ? fr.scale : 1.f, scale_lo = turns ? fr.scale_lo : 0.f;
    unsigned long long a0 = (unsigned long long)(pos0 + row) * f0, a1 = (unsigned long long)(pos0 + row) * f1;
    const unsigned long long s0 = step * f0, s1 = step * f1;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x >= per * units) return;
    for (; row < n_pos; row += step, a0 += s0, a1 += s1) {
        const float2 x = turn_of(dirs, a0, scale, scale_lo), y = turn_of(dirs, a1, scale, scale_lo);
        out[(size_t)row * units + u] = make_float4(x.x, x.y, y.x, y.y);
        if (T) {
            out_t[(size_t)j * n_pos + row] = x;
            out_t[(size_t)(j + 1) * n_pos + row] = y;
        }
    }
}

}  // namespace

// A pair that turns `turns` times in n positions has index
// n_rot ln(n / (2 pi turns)) / (2 ln theta).
void rope_frequencies(const RopeSpec &r, double *f, double *scale) {
    const int n = r.n_rot;
    const double pi2 = 6.283185307179586476925, s = r.factor;
    *scale = r.attn_factor > 0.f ? r.attn_factor : r.scaling == ROPE_RAMP ? 0.1 * std::log(s) + 1.0 : 1.0;
    auto pair_of = [&](double turns) { return n * std::log(r.n_ctx_orig / (turns * pi2)) / (2.0 * std::log((double)r.theta)); };
    double lo = 0, hi = 0;
    if (r.scaling == ROPE_RAMP) {
        lo = std::fmax(std::floor(pair_of(r.fast)), 0.0);
        hi = std::fmin(std::ceil(pair_of(r.slow)), n - 1.0);
    }
    for (int i = 0; i < n / 2; ++i) {
        double x = std::pow((double)r.theta, -2.0 * i / n);
        double keep = 1.0;                            // share of the unscaled frequency
        if (r.scaling == ROPE_LINEAR) keep = 0.0;
        if (r.scaling == ROPE_BANDS) keep = (r.n_ctx_orig * x / pi2 - r.slow) / ((double)r.fast - r.slow);
        if (r.scaling == ROPE_RAMP) keep = 1.0 - (i - lo) / std::fmax(hi - lo, 0.001);
        keep = std::fmin(std::fmax(keep, 0.0), 1.0);
        f[i] = x * keep + x / s * (1.0 - keep);
    }
}

cudaError_t launch_rope_table(const RopeSpec &r, int pos0, int n_pos, int width, float2 *out, float2 *out_t, const Launch &l) {
    const int pairs = r.n_rot / 2;
    if (pairs < 2 || pairs % 2 || pairs > width || width % 2 || width > MAX_PAIRS || n_pos < 1) return cudaErrorInvalidValue;
    double f[MAX_PAIRS], scale;
    rope_frequencies(r, f, &scale);
    Frequencies fr;
    for (int i = 0; i < pairs; ++i) fr.f[i] = (unsigned long long)std::llrint(f[i] / (2 * PI) * 18446744073709551616.0);      // at most 2^62
    fr.scale = (float)scale;
    fr.scale_lo = (float)(scale - (double)fr.scale);
    // four CTAs an SM: each fetches the directions once
    const int per = THREADS / (width / 2), want = (n_pos + per - 1) / per;
    const dim3 grid(want < 4 * 152 ? want : 4 * 152), block(THREADS);
    return launch_kernel(out_t ? rope_table_kernel<true> : rope_table_kernel<false>, grid, block, 0, l, fr, pairs, width, pos0, n_pos,
                         reinterpret_cast<float4 *>(out), out_t);
}

}  // namespace llm
