// Rotary position tables: cos and sin of position times frequency, the
// frequencies scaled for contexts beyond the trained one ("LLama.cpp — how it
// works", "Context creation": the rope_freq_base, rope_freq_scale and YaRN
// parameters of llama_context).
#include <cmath>

#include "common.cuh"
#include "launch.cuh"

namespace llm {

namespace {

constexpr int MAX_PAIRS = 64, THREADS = 256;

struct Frequencies {
    double f[MAX_PAIRS];      // radians a position
    double scale;
};

__global__ void __launch_bounds__(THREADS) rope_table_kernel(const __grid_constant__ Frequencies fr, int pairs, int pos0,
                                                             int n_pos, float2 *out) {
    pdl_wait();
    pdl_trigger();
    const long long i = (long long)blockIdx.x * THREADS + threadIdx.x;
    if (i >= (long long)n_pos * pairs) return;
    const int p = (int)(i / pairs), j = (int)(i % pairs);
    const double a = (double)(pos0 + p) * fr.f[j];
    out[i] = make_float2((float)(cos(a) * fr.scale), (float)(sin(a) * fr.scale));
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

cudaError_t launch_rope_table(const RopeSpec &r, int pos0, int n_pos, float2 *out, const Launch &l) {
    if (r.n_rot < 2 || r.n_rot > 2 * MAX_PAIRS || n_pos < 1) return cudaErrorInvalidValue;
    Frequencies fr;
    rope_frequencies(r, fr.f, &fr.scale);
    const long long n = (long long)n_pos * (r.n_rot / 2);
    return launch_kernel(rope_table_kernel, dim3((unsigned)((n + THREADS - 1) / THREADS)), dim3(THREADS), 0, l, fr, r.n_rot / 2,
                         pos0, n_pos, out);
}

}  // namespace llm
