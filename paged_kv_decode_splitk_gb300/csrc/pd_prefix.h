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
// Query rows a CTA takes at most: two 128-row tiles, or one where its O fills TMEM.
__host__ __device__ constexpr int block_rows(int dpad) { return dpad > 128 ? 128 : 256; }
// Query rows of an item at most: a block for each CTA of a team.
__host__ __device__ constexpr int item_rows(int dpad) { return 2 * block_rows(dpad); }

// How an item's rows go to the two CTAs of a team: as many as one CTA can take go
// to both, which take the tiles in turn; more, half to each, with every tile for
// both.  In turn a tile is copied (and over an FP8 cache converted) once, but there
// are twice as many partials.  Measured (8 KV heads of 128 columns, us a step, in turn
// and by halves): 32768 tokens, 128 rows 34.8 and 44.0, 256 rows 40.2 and 45.4, over
// FP8 37.6 and 53.0, 44.7 and 54.6; 8192 tokens, 128 rows 20.5 and 22.6, 256 rows
// 24.2 and 24.1.
__host__ __device__ constexpr bool is_pair(int rows, int of_item) { return rows > of_item / 2; }

// What the prefix pass found the work to be: units in all, the teams that share
// them, and whether every item has whole teams.
struct PlanTotal {
    long long units;
    int teams;
    int whole;
};

// One group on the line of work units.  Its items are, for each KV head, the
// item_rows-row pieces of its query rows; a unit of a pair item is a tile, of one
// whose tiles are taken in turn, two.
struct GroupPlan {
    long long first_unit;
    int first_item;
    int tiles;      // of the prefix; 0: nothing to do
    int first_seq;
    int rows;       // sequences x query heads of a KV head
    int items;      // of a KV head
    int tokens;     // of the prefix
    int first_team, teams, last_teams;  // whole teams: of an item, and of a KV head's last

    // units of a KV head, and of its last item, which alone may have few rows
    __host__ __device__ int last_units(int of_item) const {
        return is_pair(rows - (items - 1) * of_item, of_item) ? tiles : (tiles + 1) >> 1;
    }
    __host__ __device__ long long head_units(int of_item) const {
        return static_cast<long long>(items - 1) * tiles + last_units(of_item);
    }
};

struct PrefixParams {
    const __nv_bfloat16 *q;
    const int32_t *prefix_table, *prefix_lens, *group_starts;
    int num_groups, max_prefix_blocks, num_blocks;
    const int32_t *context_lens;   // of the own tokens, with the most a table holds
    int max_own_tokens;
    int num_seqs, num_q_heads, num_kv_heads, group, head_dim;
    FastDiv block_size, fd_group;
    int tok_dim;
    int box_tokens;     // tokens of a TMA box: a power of two from 16 that divides the block and the tile
    float scale_log2;   // |scale| log2(e) (times k_scale), above 0
    int negative;       // the scale is negative: q changes sign instead
    int max_items;
    float *part_ml;     // [slot][block rows] (m, l); a team's item has two slots, one for each CTA
    float *part_o;      // [slot][dpad / 32][block rows][32], 16-byte chunks swapped by row
    GroupPlan *plan_groups;
    PlanTotal *plan_total;
    unsigned int *status;
};

struct MergeParams {
    const GroupPlan *plan_groups;
    const PlanTotal *plan_total;
    const float *part_ml, *part_o;   // the prefix pass's
    const float *own_o, *own_ml;     // [rows, N, D] and [rows, N, 2]: the own-token pass's
    const int32_t *context_lens;
    __nv_bfloat16 *out;
    int num_groups, num_seqs, num_q_heads, num_kv_heads, group, head_dim, dpad;
    int num_splits, min_kv_per_split, max_tokens;
    int ways;           // lines of lanes a row has
    float v_scale;      // of the prefix partials (an FP8 cache; the own-token pass applies its own)
    FastDiv fd_hq, fd_group, fd_split, fd_bs;
};

template <int DPAD, bool KV8>
cudaError_t launch_prefix(const CUtensorMap *tk, const CUtensorMap *tv, const PrefixParams &p, int teams,
                          cudaStream_t stream);

}  // namespace prefix
}  // namespace pd
