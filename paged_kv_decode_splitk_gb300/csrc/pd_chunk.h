// pd_chunk.h -- what the host side, the kernel and the fold of pd_chunk_attn agree on.
#pragma once

#include "pd_chunk_plan.h"
#include "pd_internal.h"

namespace pd {
namespace chunk {

struct ChunkParams {
    Shape shape;
    const __nv_bfloat16 *q;
    long long q_tok;               // elements from a token's queries to the next's
    __nv_bfloat16 *out;
    float *lse;                    // or null
    const int32_t *block_table, *context_lens, *token_starts;
    int max_blocks, num_blocks;
    int num_tokens, num_seqs, num_q_heads, head_dim;
    int max_tokens;                // a table holds
    FastDiv block_size, fd_heads;  // fd_heads: item_heads
    int tok_dim, box_tokens;       // of the caches' maps (tokens of a box divide block and tile)
    int query_box;                 // tokens of a box of q
    float scale_log2;              // |scale| log2(e) (times k_scale), above 0
    int negative;                  // the scale is negative: q changes sign instead
    float v_scale;
    FastDiv ctas;                  // of the launch
    int most_units;                // that sequences without a row in common can make
    int slot_rows;                 // rows of a slot: a block's at most, a multiple of 32
    CutItem *cut;                  // [CTAs]
    float *part_ml;                // [slot][slot_rows] (m, l); CTA c has slots 2 c (it begins inside
    float *part_o;                 // [slot][dpad / 4][item's rows][4]  an item) and 2 c + 1 (it ends inside one)
    unsigned int *status;
};

// Rows of an item's partials.
__device__ __forceinline__ int partial_rows(int rows) { return (rows + 7) & ~7; }

struct FoldParams {
    const CutItem *cut;
    const float *part_ml, *part_o;
    __nv_bfloat16 *out;
    float *lse;
    int num_q_heads, head_dim, slot_rows;
    FastDiv fd_heads;
    int item_heads;
    float v_scale;
};

template <int DPAD, bool KV8>
cudaError_t launch_chunk(const CUtensorMap *tk, const CUtensorMap *tv, const CUtensorMap *tq, const ChunkParams &p, int ctas,
                         cudaStream_t stream);

}  // namespace chunk
}  // namespace pd
