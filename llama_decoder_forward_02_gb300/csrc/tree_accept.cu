// Acceptance of a tree of drafted tokens, and the move of the accepted cells.
//
// After a step over a tree, target[i] is the token that the model picks after
// node i.  Node 0 stands; from a node that stands its child whose token is the
// node's target stands too (the lowest of several).  That path's keys and values
// move from cells base + path[j] to base + j, of every layer, and the target of
// its last node is the sequence's next token.  Drawing every node's target from the
// model's distribution and keeping what agrees leaves the distribution of tokens
// as it is without drafts ("LLama.cpp — how it works", "Steps 14–15", has the
// sampler that draws them).
//
// path[j] >= j and grows with j, so rows that are written in ascending order,
// each group read whole before it is written, never overwrite one still to be
// read.  Every CTA walks its tree itself (a few hundred bytes).
//
// Bound by latency: row numbers, then parents, then their targets, the walk, then the
// rows, each a load that waits for the one before.  One tree of 16 nodes, 5 accepted, of
// 32 layers of 8 kv heads of 128: 2.7 us back to back, eight trees of 64 6.2 us, where
// the bytes would take 1.5.  Fewer CTAs with several planes each take about the same
// (6.0 us), eight units of a thread in flight more (8.3).
#include "common.cuh"
#include "launch.cuh"

namespace llm {

namespace {

constexpr int THREADS = 128;

// Moves rows of `units` units U from base + path[j] to base + j, j = 1 .. count - 1.
template <typename U>
__device__ __forceinline__ void move_rows(U *rows, int units, const int *path, int count) {
    const int n = count * units;
    for (int i0 = 0; i0 < n; i0 += THREADS) {
        const int i = i0 + threadIdx.x, j = i / units, at = i - j * units;
        U v;
        if (i < n) v = rows[(size_t)path[j] * units + at];
        __syncthreads();
        if (i < n && path[j] != j) rows[(size_t)j * units + at] = v;
    }
}

// grid (tree, layer * head, K or V)
__global__ void __launch_bounds__(THREADS) tree_accept_kernel(const TreeAcceptArgs a) {
    __shared__ int first_child[TREE_MAX_NODES], path[TREE_MAX_NODES], sh_count;
    const int tree = blockIdx.x, block = blockIdx.y, tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int r0 = a.row0[tree], n = a.row0[tree + 1] - r0, seq = a.seq[tree], base = a.base[tree];
    const bool ok = r0 >= 0 && n >= 0 && n <= a.max_nodes && r0 <= a.T - n && seq >= 0 && seq < a.n_seq && base >= 0 &&
                    base <= a.n_ctx - n;
    const bool writes = block == 0 && blockIdx.z == 0;        // the CTA that reports
    if (!ok && writes && tid == 0) raise_error(a.err, ERRF_BAD_INDEX);
    const int nodes = ok ? n : 0;
    for (int i = tid; i < nodes; i += THREADS) first_child[i] = nodes;
    if (tid == 0) sh_count = 0;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < nodes; i += THREADS) {
        const int p = a.parent[r0 + i];
        if (i == 0 ? p != -1 : p < 0 || p >= i) bad = true;
        else if (i > 0 && a.token[r0 + i] == a.target[r0 + p]) atomicMin(&first_child[p], i);
    }
    const bool broken = __syncthreads_or(bad);
    if (broken && writes && tid == 0) raise_error(a.err, ERRF_BAD_INDEX);
    if (tid == 0 && !broken) {
        int c = 0;
        for (int cur = 0; cur < nodes; cur = first_child[cur]) path[c++] = cur;
        sh_count = c;
    }
    __syncthreads();
    const int count = sh_count;
    if (writes) {
        for (int i = tid; i < a.max_nodes; i += THREADS) a.path[(size_t)tree * a.max_nodes + i] = i < count ? path[i] : -1;
        if (tid == 0) {
            a.n_accept[tree] = count;
            a.next[tree] = count ? a.target[r0 + path[count - 1]] : -1;
        }
    }
    if (count < 2) return;
    // row (seq, layer, head, base) of the planes
    const size_t row = ((size_t)seq * a.heads + block) * a.n_ctx + base;
    const int hd = a.head_dim;
    uint8_t *cache = (uint8_t *)(blockIdx.z ? a.v : a.k);
    if (a.kv_type == TREE_KV_F16) move_rows((uint4 *)(cache + row * hd * 2), hd / 8, path, count);
    else if (a.kv_type == TREE_KV_E4M3) move_rows((uint4 *)(cache + row * hd), hd / 16, path, count);
    else {
        move_rows((uint4 *)(cache + row * (hd / 2)), hd / 32, path, count);
        const size_t rows = (size_t)a.n_seq * a.heads * a.n_ctx;
        move_rows((f16 *)(cache + rows * (hd / 2)) + row * (hd / 32), hd / 32, path, count);
    }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptArgs &a, const Launch &l) {
    if (a.n_tree < 1 || a.heads < 1 || a.heads > 65535 || a.max_nodes < 1 || a.max_nodes > TREE_MAX_NODES)
        return cudaErrorInvalidValue;
    return launch_kernel(tree_accept_kernel, dim3(a.n_tree, a.heads, 2), dim3(THREADS), 0, l, a);
}

}  // namespace llm
