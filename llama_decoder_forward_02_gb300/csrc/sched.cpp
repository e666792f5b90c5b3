#include "sched.h"

#include <cstdio>
#include <new>

namespace llm {

int plan_batch(const llm_batch &b, int n_vocab, int n_ctx, int n_seq_max, int n_ubatch,
               const std::vector<int32_t> &seq_next, BatchPlan &p) {
    char buf[160];
    p = BatchPlan();
    if (b.n_tokens <= 0) { p.error = "batch has no tokens"; return LLM_ERR_INVALID; }
    if (!b.token) { p.error = "batch has no token array"; return LLM_ERR_INVALID; }
    const int n = b.n_tokens;
    p.n = n;
    if (!(b.flags & LLM_BATCH_TOKENS_ON_DEVICE)) {
        p.tok.assign(b.token, b.token + n);
        for (int i = 0; i < n; ++i)
            if (p.tok[i] < 0 || p.tok[i] >= n_vocab) {
                snprintf(buf, sizeof buf, "invalid token[%d] = %d", i, p.tok[i]);
                p.error = buf;
                return LLM_ERR_INVALID;
            }
    }
    p.seq.assign(n, 0);
    if (b.seq_id) p.seq.assign(b.seq_id, b.seq_id + n);
    for (int i = 0; i < n; ++i)
        if (p.seq[i] < 0 || p.seq[i] >= n_seq_max) {
            snprintf(buf, sizeof buf, "invalid seq_id[%d] = %d (n_seq_max %d)", i, p.seq[i], n_seq_max);
            p.error = buf;
            return LLM_ERR_INVALID;
        }
    std::vector<int32_t> nxt = seq_next;
    p.pos.resize(n);
    for (int i = 0; i < n; ++i) {
        const int s = p.seq[i];
        if (b.pos && b.pos[i] != nxt[s]) {
            snprintf(buf, sizeof buf, "pos[%d] = %d but sequence %d continues at %d", i, b.pos[i], s, nxt[s]);
            p.error = buf;
            return LLM_ERR_INVALID;
        }
        p.pos[i] = nxt[s]++;
    }
    p.out.assign(n, 0);
    if (b.output) {
        for (int i = 0; i < n; ++i) p.out[i] = b.output[i] ? 1 : 0;
    } else {
        p.out[n - 1] = 1;
    }
    for (int i = 0; i < n; ++i)
        if (p.pos[i] >= n_ctx) {
            snprintf(buf, sizeof buf, "position %d of sequence %d does not fit n_ctx %d", p.pos[i], p.seq[i], n_ctx);
            p.error = buf;
            return LLM_NO_KV_ROOM;
        }
    p.out_index.assign(n, -1);
    for (int i = 0; i < n; ++i)
        if (p.out[i]) p.out_index[i] = p.n_outputs++;
    for (int s = 0; s < n; s += n_ubatch) p.ub_start.push_back(s);
    p.ub_start.push_back(n);
    return LLM_OK;
}

int plan_tree(const llm_tree_batch &b, int n_vocab, int n_ctx, int n_seq_max, int n_ubatch, int window,
              const std::vector<int32_t> &seq_next, TreePlan &p) {
    char buf[160];
    p = TreePlan();
    if (b.n_trees < 1 || !b.n_nodes || !b.token || !b.parent) { p.error = "the batch has no trees, nodes, tokens or parents"; return LLM_ERR_INVALID; }
    if (b.n_trees > n_seq_max) { p.error = "more trees than sequences"; return LLM_ERR_INVALID; }
    long long n = 0;
    for (int i = 0; i < b.n_trees; ++i) {
        if (b.n_nodes[i] < 1 || b.n_nodes[i] > TREE_PLAN_MAX_NODES) {
            snprintf(buf, sizeof buf, "tree %d has %d nodes (1..%d)", i, b.n_nodes[i], TREE_PLAN_MAX_NODES);
            p.error = buf;
            return LLM_ERR_INVALID;
        }
        n += b.n_nodes[i];
    }
    if (n > n_ubatch) { p.error = "the trees have more nodes than a ubatch has rows"; return LLM_ERR_INVALID; }
    std::vector<int8_t> taken(n_seq_max, 0);
    p.row0.push_back(0);
    for (int i = 0; i < b.n_trees; ++i) {
        const int s = b.seq_id ? b.seq_id[i] : i;
        if (s < 0 || s >= n_seq_max || taken[s]) {
            snprintf(buf, sizeof buf, "seq_id[%d] = %d is outside [0, %d) or has a tree already", i, s, n_seq_max);
            p.error = buf;
            return LLM_ERR_INVALID;
        }
        taken[s] = 1;
        p.seq_of.push_back(s);
        p.base.push_back(seq_next[s]);
        p.row0.push_back(p.row0.back() + b.n_nodes[i]);
        if (b.n_nodes[i] > p.max_nodes) p.max_nodes = b.n_nodes[i];
    }
    p.token.assign(b.token, b.token + n);
    p.parent.assign(b.parent, b.parent + n);
    p.words = (p.max_nodes + 31) / 32;
    p.mask.assign((size_t)n * p.words, 0u);
    for (int i = 0; i < b.n_trees; ++i) {
        const int r0 = p.row0[i], s = p.seq_of[i];
        for (int j = 0; j < b.n_nodes[i]; ++j) {
            const int r = r0 + j, par = p.parent[r];
            if (p.token[r] < 0 || p.token[r] >= n_vocab) {
                snprintf(buf, sizeof buf, "invalid token[%d] = %d", r, p.token[r]);
                p.error = buf;
                return LLM_ERR_INVALID;
            }
            if (j == 0 ? par != -1 : par < 0 || par >= j) {
                snprintf(buf, sizeof buf, "parent[%d] = %d of node %d is not a lower node of its tree (-1 for node 0)", r, par, j);
                p.error = buf;
                return LLM_ERR_INVALID;
            }
            p.pos.push_back(j ? p.pos[r0 + par] + 1 : p.base[i]);
            p.seq.push_back(s);
            p.cell.push_back(p.base[i] + j);
            uint32_t *m = &p.mask[(size_t)r * p.words];
            for (int w = 0; j && w < p.words; ++w) m[w] = p.mask[(size_t)(r0 + par) * p.words + w];
            m[j / 32] |= 1u << (j % 32);
            if (window > 0) {
                int up = j;                       // the ancestor `window` levels up
                for (int w = 0; up >= 0 && w < window; ++w) up = p.parent[r0 + up];
                if (up >= 0) m[up / 32] &= ~(1u << (up % 32));
            }
        }
    }
    for (int i = 0; i < b.n_trees; ++i)
        if (p.base[i] + b.n_nodes[i] > n_ctx) {
            snprintf(buf, sizeof buf, "%d nodes behind position %d of sequence %d do not fit n_ctx %d", b.n_nodes[i], p.base[i] - 1,
                     p.seq_of[i], n_ctx);
            p.error = buf;
            return LLM_NO_KV_ROOM;
        }
    p.n = (int)n;
    return LLM_OK;
}

void accept_path(const TreePlan &p, const int32_t *target, std::vector<int32_t> &stand, std::vector<int32_t> &count) {
    stand.assign(p.n, -1);
    count.clear();
    for (size_t i = 0; i + 1 < p.row0.size(); ++i) {
        const int r0 = p.row0[i], n = p.row0[i + 1] - r0;
        int cur = 0, c = 0;
        stand[r0 + c++] = 0;
        // children have higher numbers than their parent
        for (int j = 1; j < n; ++j)
            if (p.parent[r0 + j] == cur && p.token[r0 + j] == target[r0 + cur]) stand[r0 + c++] = cur = j;
        count.push_back(c);
    }
}

}  // namespace llm

extern "C" int32_t llm_tree_check(int32_t n_vocab, int32_t n_ctx, int32_t n_seq_max, int32_t n_ubatch,
                                  const int32_t *seq_pos_max, const llm_tree_batch *b, int32_t *pos_out, int32_t *cell_out) {
    if (!b || !seq_pos_max || n_seq_max < 1 || n_ubatch < 1) return LLM_ERR_INVALID;
    try {
        std::vector<int32_t> nxt(n_seq_max);
        for (int s = 0; s < n_seq_max; ++s) nxt[s] = seq_pos_max[s] + 1;
        llm::TreePlan p;
        const int rc = llm::plan_tree(*b, n_vocab, n_ctx, n_seq_max, n_ubatch, 0, nxt, p);
        if (rc != LLM_OK) return rc;
        for (int i = 0; i < p.n; ++i) {
            if (pos_out) pos_out[i] = p.pos[i];
            if (cell_out) cell_out[i] = p.cell[i];
        }
    } catch (const std::bad_alloc &) {
        return LLM_ERR_ALLOC;
    }
    return LLM_OK;
}

extern "C" int32_t llm_batch_check(int32_t n_vocab, int32_t n_ctx, int32_t n_seq_max, int32_t n_ubatch,
                                   const int32_t *seq_pos_max, const llm_batch *b, int32_t *pos_out,
                                   int32_t *out_index, int32_t *ubatch_starts, int32_t *n_ubatches) {
    if (!b || !seq_pos_max || n_seq_max < 1 || n_ubatch < 1) return LLM_ERR_INVALID;
    std::vector<int32_t> nxt(n_seq_max);
    for (int s = 0; s < n_seq_max; ++s) nxt[s] = seq_pos_max[s] + 1;
    llm::BatchPlan p;
    const int rc = llm::plan_batch(*b, n_vocab, n_ctx, n_seq_max, n_ubatch, nxt, p);
    if (rc != LLM_OK) return rc;
    for (int i = 0; i < p.n; ++i) {
        if (pos_out) pos_out[i] = p.pos[i];
        if (out_index) out_index[i] = p.out_index[i];
    }
    const int nub = (int)p.ub_start.size() - 1;
    if (ubatch_starts)
        for (int i = 0; i < nub; ++i) ubatch_starts[i] = p.ub_start[i];
    if (n_ubatches) *n_ubatches = nub;
    return LLM_OK;
}
