// How kv8_attention divides its work: decided from the host's sizes alone, the same for the
// workspace's size and for the launch.
#pragma once

#include <stdint.h>

namespace w4a8 {

struct AttentionPlan {
    int rows;                 // query rows of a block: 128 or 64 (many), or 16
    bool prompt;              // many query rows a sequence
    int64_t tiles;            // row tiles of a sequence
    bool halves;              // 64 rows: blocks of 8 waves, every second tile each half
    bool wide;                // few rows, short contexts: blocks of 8 waves, a context each
    bool parts;               // blocks leave partial results, joined by a second launch
    int chunks, chunk_steps;  // many rows: most chunks of a context, steps of 64 keys in one
    int64_t blocks, join_blocks;
    int64_t part_rows;        // rows of partial results
};
AttentionPlan attention_plan(int64_t B, int64_t max_new, int64_t max_kv, int q_heads, int kv_heads, int head_dim);
int64_t attention_workspace(const AttentionPlan& p, int head_dim);

}  // namespace w4a8
