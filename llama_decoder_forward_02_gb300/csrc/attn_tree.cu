// Attention of the nodes of trees of drafted tokens over a cache ("Inside the
// inference engine: model architectures and forward pass", section "KV Cache:
// memory for causal attention"; the mask of a node is its sequence's earlier
// cells and the path to it): for row t of tree i and query head h
//   o[t][h] = softmax_c(q[t][h] . K[c] / sqrt(hd)) V[c]
// over the cells c < base[i] (with a window those c > pos[t] - window) and the
// cells base[i] + j whose bit j of mask[t] is set.  A row that sees nothing is zero.
//
// One warp takes a row and query head, a lane a key of 32.
#include "common.cuh"
#include "launch.cuh"

namespace llm {

namespace {

constexpr int WARPS = 4;

template <int HD, bool F8>
__global__ void __launch_bounds__(WARPS * 32) attn_tree_kernel(const AttnTreeArgs a) {
    __shared__ float qs[WARPS][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int tree = blockIdx.y, Hkv = a.kv.n_kv_head;
    const int r0 = a.row0[tree], n = a.row0[tree + 1] - r0, seq = a.seq[tree], base = a.base[tree];
    const bool ok = r0 >= 0 && n >= 0 && n <= a.max_nodes && r0 <= a.T - n && seq >= 0 && seq < a.kv.n_seq && base >= 0 &&
                    base <= a.kv.n_ctx - n;
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0) raise_error(a.err, ERRF_BAD_INDEX);
    const int item = blockIdx.x * WARPS + warp, node = item / a.H, h = item % a.H, t = r0 + node;
    if (node >= min(n, a.max_nodes) || t < 0 || t >= a.T) return;
    f16 *o = a.o + ((size_t)t * a.H + h) * HD;
    if (!ok) {
        for (int d = lane; d < HD; d += 32) o[d] = f2h(0.f);
        return;
    }
    const float c = 1.4426950408889634f / sqrtf((float)HD);
    for (int d = lane; d < HD; d += 32) qs[warp][d] = hf(a.q[((size_t)t * a.H + h) * HD + d]) * c;
    __syncwarp();
    const size_t row = (size_t)seq * a.kv.seq_stride + (size_t)(h / (a.H / Hkv)) * a.kv.n_ctx * HD;
    auto value = [&](const f16 *p, const uint8_t *p8, size_t e) {
        return F8 ? h2lo(e4m3x2_to_h2(p8[e])) : hf(p[e]);
    };
    const int lo = a.window > 0 ? max(0, min(a.pos[t] - a.window + 1, base)) : 0;
    float m = -INFINITY, l = 0.f, acc[HD / 32] = {0.f};
    for (int k0 = lo; k0 < base + n; k0 += 32) {
        const int k = k0 + lane, j = k - base;
        const bool seen = k < base + n && (j < 0 || (a.mask[(size_t)t * a.words + j / 32] >> (j & 31) & 1u));
        float s = -INFINITY;
        if (seen) {
            s = 0.f;
            for (int d = 0; d < HD; ++d) s = fmaf(qs[warp][d], value(a.kv.k, a.kv.k8, row + (size_t)k * HD + d), s);
        }
        const float mn = fmaxf(m, warp_max(s)), f = mn == -INFINITY ? 1.f : exp2f(m - mn);
        const float p = seen ? exp2f(s - mn) : 0.f;
        l = l * f + warp_sum(p);
        m = mn;
        for (int i = 0; i < HD / 32; ++i) acc[i] *= f;
        for (int q = 0; q < 32; ++q) {
            const float pq = __shfl_sync(0xffffffffu, p, q);
            if (!__shfl_sync(0xffffffffu, (int)seen, q)) continue;
            for (int i = 0; i < HD / 32; ++i)
                acc[i] = fmaf(pq, value(a.kv.v, a.kv.v8, row + (size_t)(k0 + q) * HD + lane + 32 * i), acc[i]);
        }
    }
    for (int i = 0; i < HD / 32; ++i) o[lane + 32 * i] = f2h(l == 0.f ? 0.f : acc[i] / l);
}

}  // namespace

size_t attn_tree_scratch_bytes(int, int, int, int, int, int) { return 16; }

cudaError_t launch_attn_tree(const AttnTreeArgs &a, const TmaMap *, const TmaMap *, const Launch &l) {
    const dim3 grid((a.max_nodes * a.H + WARPS - 1) / WARPS, a.n_tree), block(WARPS * 32);
    const bool f8 = a.kv.k8;
    switch (a.kv.head_dim) {
        case 32: return launch_kernel(f8 ? attn_tree_kernel<32, true> : attn_tree_kernel<32, false>, grid, block, 0, l, a);
        case 64: return launch_kernel(f8 ? attn_tree_kernel<64, true> : attn_tree_kernel<64, false>, grid, block, 0, l, a);
        case 128: return launch_kernel(f8 ? attn_tree_kernel<128, true> : attn_tree_kernel<128, false>, grid, block, 0, l, a);
    }
    return cudaErrorInvalidValue;
}

}  // namespace llm
