// How kv8_attention divides its work: decided from the host's sizes alone, the same for the
// workspace's size and for the launch.
#pragma once

#include <stdint.h>

namespace w4a8 {

struct AttentionPlan {
    bool prompt;              // many query rows a sequence: blocks of 128 rows, else of 16
    bool deal;                // equal shares of all steps, parts joined afterwards
    int64_t blocks, join_blocks;
    int64_t part_rows;        // rows of partial results
};
AttentionPlan attention_plan(int64_t B, int64_t max_new, int64_t max_kv, int q_heads, int kv_heads, int head_dim);
int64_t attention_workspace(const AttentionPlan& p, int head_dim);

}  // namespace w4a8
