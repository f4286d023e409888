// pd_prefix.h -- what the host side, the shared-prefix pass and the merge of
// pd_decode_attn_prefix agree on.
#pragma once

#include "pd_internal.h"

namespace pd {
namespace prefix {

constexpr int kMaxGroups = 256;   // PD_MAX_PREFIX_GROUPS
constexpr int kMaxTeams = 76;     // teams of two CTAs of the prefix pass at most (sizes the workspace)

// Keys of a tile: 128, or 64 where a tile of 128 would leave no ring (D > 128).
__host__ __device__ constexpr int tile_tokens(int dpad) { return dpad > 128 ? 64 : 128; }
// Query rows of an item: two 128-row tiles, or one where its O fills TMEM.
__host__ __device__ constexpr int block_rows(int dpad) { return dpad > 128 ? 128 : 256; }

// Teams that share W units: all there are, but each at least kMinUnits (a team
// more is a partial more of each of its rows to write and fold).
constexpr int kMinUnits = 1;
__host__ __device__ inline int teams_of(long long W, int most) {
    const long long n = (W + kMinUnits - 1) / kMinUnits;
    return n < most ? static_cast<int>(n) : most;
}

// One group on the line of work units.  An item is two row blocks of a KV head,
// which a team's CTAs work on side by side (a unit is a tile), or a block left
// over, whose tiles they take in turn (a unit is two tiles); per KV head the pairs
// come first.
struct GroupPlan {
    long long first_unit;
    int first_item;
    int tiles;      // of the prefix; 0: nothing to do
    int first_seq;
    int rows;       // sequences x query heads of a KV head
    int blocks;     // row blocks
    int tokens;     // of the prefix
};

struct PrefixParams {
    const __nv_bfloat16 *q;
    const int32_t *prefix_table, *prefix_lens, *group_starts;
    int num_groups, max_prefix_blocks, num_blocks;
    int num_seqs, num_q_heads, num_kv_heads, group, head_dim;
    FastDiv block_size, fd_group;
    int tok_dim;
    int box_tokens;     // tokens of a TMA box: a power of two from 16 that divides the block and the tile
    float scale_log2;   // |scale| log2(e) (times k_scale), above 0
    int negative;       // the scale is negative: q changes sign instead
    int max_items;
    float *part_ml;     // [slot][block rows] (m, l); a team's item has two slots, one for each CTA
    float *part_o;      // [slot][dpad / 8][block rows][8]
    GroupPlan *plan_groups;
    long long *plan_total;
    unsigned int *status;
};

struct MergeParams {
    const GroupPlan *plan_groups;
    const long long *plan_total;
    const float *part_ml, *part_o;   // the prefix pass's
    const float *own_o, *own_ml;     // [rows, N, D] and [rows, N, 2]: the own-token pass's
    const int32_t *context_lens;
    __nv_bfloat16 *out;
    int num_groups, num_seqs, num_q_heads, num_kv_heads, group, head_dim, dpad;
    int num_splits, min_kv_per_split, max_tokens, teams;
    float v_scale;      // of the prefix partials (an FP8 cache; the own-token pass applies its own)
    FastDiv fd_hq, fd_group, fd_split, fd_bs;
};

template <int DPAD, bool KV8>
cudaError_t launch_prefix(const CUtensorMap *tk, const CUtensorMap *tv, const PrefixParams &p, int teams,
                          cudaStream_t stream);

}  // namespace prefix
}  // namespace pd
