// Host-side batch scheduler: the rules of "LLama.cpp — how it works",
// "Step 10" (llama_batch_allocr::init fills missing seq ids, positions and
// output flags, and rejects bad token ids) and "Steps 11–12" (init_batch cuts
// the batch into consecutive ubatches of at most n_ubatch tokens).  Pure C++,
// no CUDA, so it runs and is tested without a GPU.
#pragma once
#include <stdint.h>
#include <string>
#include <vector>

#include "../../include/llm.h"

namespace llm {

struct BatchPlan {
    int n = 0;
    std::vector<int32_t> tok;        // host copy of the token ids (empty if on device)
    std::vector<int32_t> pos, seq;
    std::vector<int8_t> out;
    std::vector<int32_t> out_index;  // batch index -> logits row, or -1
    int n_outputs = 0;
    std::vector<int32_t> ub_start;   // ubatch i covers [ub_start[i], ub_start[i+1])
    std::string error;
};

// Validates `b` against the cache state `seq_next` (next free position of
// every sequence, i.e. seq_pos_max + 1) and fills `p`.  Returns LLM_OK,
// LLM_NO_KV_ROOM or LLM_ERR_INVALID (with p.error set).
int plan_batch(const llm_batch &b, int n_vocab, int n_ctx, int n_seq_max, int n_ubatch,
               const std::vector<int32_t> &seq_next, BatchPlan &p);

// The trees of a llm_decode_tree call, rows in batch order.
struct TreePlan {
    int n = 0;                                    // rows
    int max_nodes = 0, words = 0;
    std::vector<int32_t> token, parent, pos, seq, cell;      // [n]
    std::vector<int32_t> row0, seq_of, base;                 // [trees + 1], [trees], [trees]
    std::vector<uint32_t> mask;                   // [n][words]: bit j of row t = it sees node j of its tree
    std::string error;
};
constexpr int TREE_PLAN_MAX_NODES = 256;
// As plan_batch; with window > 0 a node sees the window - 1 nearest of its ancestors.
int plan_tree(const llm_tree_batch &b, int n_vocab, int n_ctx, int n_seq_max, int n_ubatch, int window,
              const std::vector<int32_t> &seq_next, TreePlan &p);
// The nodes of each tree that target accepts (stand, rows of the tree from row0 on,
// the rest -1) and their number.
void accept_path(const TreePlan &p, const int32_t *target, std::vector<int32_t> &stand, std::vector<int32_t> &count);

}  // namespace llm
