// pd_chunk_plan.h -- how pd_chunk_attn divides its work, by functions that the
// kernel, the host side and the CPU tests share.
//
// An item is a block of a sequence's new tokens with the query heads of one KV
// head: up to block_rows query rows that meet the same keys, from the first that
// any of them sees to the last.  Items lie in one line, by sequence, head and block;
// an item has one unit for each key tile and kItemUnits in front of them for what
// it costs besides.  Every CTA takes the same number of units that follow one
// another, so every SM gets the same work whatever the shapes; an item that a border
// cuts leaves partials, which a second kernel folds, all others leave results.  Units
// before a block are a sum of rounded-up quotients, which floor_sum gives without a
// walk over the blocks.
#pragma once

#include <stdint.h>

#include "pd_internal.h"

namespace pd {
namespace chunk {

constexpr int kRowTile = 128;   // query rows of one product
constexpr int kMaxCtas = 152;   // CTAs of a launch at most (sizes the workspace)

// Keys of a tile: 128, or 64 where a tile of 128 would leave no ring (D > 128).
__host__ __device__ constexpr int tile_tokens(int dpad) { return dpad > 128 ? 64 : 128; }
// Query rows a CTA takes at most: two 128-row tiles, or one where its O fills TMEM.
__host__ __device__ constexpr int block_rows(int dpad) { return dpad > 128 ? 128 : 256; }

// What an item costs besides its tiles, in units: its queries, the first scores and
// the way out take about as long as two tiles.
constexpr int kItemUnits = 2;
// Units that are worth a CTA of their own.
constexpr int kCtaUnits = 5;
// Units of a launch are no more (they and their sums are 32-bit numbers).
constexpr int kMaxUnits = 0x3fffffff;

// Units of two parts of the batch, or more than kMaxUnits where they are more.  (Sequences
// whose rows overlap may pass any bound.)
__host__ __device__ inline int add_units(int a, int b) {
    const uint32_t sum = static_cast<uint32_t>(a) + static_cast<uint32_t>(b);
    return static_cast<int>(sum < kMaxUnits + 1u ? sum : kMaxUnits + 1u);
}

// What all items of a launch share.
struct Shape {
    int group;        // query heads of a KV head
    int item_heads;   // of them an item has (all, where they fit its rows)
    int head_parts;   // items that a token block's query heads make
    int kv_heads;
    int heads;        // KV heads x head_parts
    int block_tokens; // new tokens of a block
    FastDiv fd_block; // block_tokens
    int tile_log2;    // of the keys of a tile
    int period_log2;  // blocks after which their ends lie alike in their tiles
    int window;       // keys a token sees at most, itself among them; 0: all
};

inline Shape make_shape(int num_q_heads, int num_kv_heads, int dpad, int window) {
    Shape s;
    s.group = num_q_heads / num_kv_heads;
    s.head_parts = (s.group + block_rows(dpad) - 1) / block_rows(dpad);
    s.item_heads = (s.group + s.head_parts - 1) / s.head_parts;
    s.kv_heads = num_kv_heads;
    s.heads = num_kv_heads * s.head_parts;
    s.block_tokens = block_rows(dpad) / s.item_heads;
    if (s.block_tokens > 1) s.block_tokens &= ~1;  // (even, so that boxes of several tokens divide it)
    s.fd_block = make_fastdiv(s.block_tokens);
    s.tile_log2 = dpad > 128 ? 6 : 7;
    s.period_log2 = s.tile_log2;
    for (int t = s.block_tokens; s.period_log2 > 0 && t % 2 == 0; t /= 2) --s.period_log2;
    s.window = window;
    return s;
}

// Tokens of a box of queries: at most 32 rows, and boxes make up a block.
inline int query_box_tokens(const Shape &s) {
    int n = 1;
    while (2 * n * s.item_heads <= 32 && s.block_tokens % (2 * n) == 0) n *= 2;
    return n;
}

// The new tokens of a sequence: rows first to first + n - 1, at positions past to
// past + n - 1 = len - 1.  (past < 0: more new tokens than the sequence has; those
// before position 0 see nothing.)
struct Span {
    int first, n, past, len;
};

// sum over i < n of floor((a + i b) / 2^m), where b 2^p is a multiple of 2^m: after 2^p
// terms the quotients come again, all larger by b 2^p / 2^m.
__host__ __device__ inline int floor_sum(uint32_t n, uint32_t a, uint32_t b, int m, int p) {
    const uint32_t period = 1u << p, rest = n & (period - 1), whole = n >> p, step = (b << p) >> m;
    uint32_t all = 0, some = 0;  // of the first period's terms, and of its first `rest`
#pragma unroll 1
    for (uint32_t i = 0; i < (whole > 0 ? period : rest); ++i) {
        const uint32_t v = (a + i * b) >> m;
        all += v;
        some += i < rest ? v : 0;
    }
    // (the pairs of periods pass 32 bits for prompts of 2^24 tokens and more, which a window makes few units of)
    const uint32_t pairs = static_cast<uint32_t>(static_cast<uint64_t>(whole) * (whole - 1) / 2);
    return static_cast<int>(whole * all + step * (period * pairs + whole * rest) + some);
}

__host__ __device__ inline int blocks_of(const Shape &s, int n) { return fast_div(n + s.block_tokens - 1, s.fd_block); }

// Position that the first of a block's keys has, and one past its last.
__host__ __device__ inline int first_key(const Shape &s, int position) {
    return s.window > 0 && position >= s.window ? position + 1 - s.window : 0;
}
__host__ __device__ inline int end_key(const Shape &s, const Span &q, int block) {
    const int last = (block + 1) * s.block_tokens;
    const int end = q.past + (last < q.n ? last : q.n);
    return end > 0 ? end : 0;
}
__host__ __device__ inline int first_tile(const Shape &s, const Span &q, int block) {
    return first_key(s, q.past + block * s.block_tokens) >> s.tile_log2;
}
__host__ __device__ inline int tiles_of(const Shape &s, const Span &q, int block) {
    const int end = (end_key(s, q, block) + (1 << s.tile_log2) - 1) >> s.tile_log2;
    return end > 0 ? end - first_tile(s, q, block) : 0;
}

// Units of a block at most, in tables of max_tokens: a window and the block's tokens behind it touch a tile more at
// either end than they fill.
inline long long most_block_units(const Shape &s, int max_tokens) {
    const long long all = (max_tokens >> s.tile_log2) + 1ll;
    const long long seen = ((static_cast<long long>(s.window) + s.block_tokens) >> s.tile_log2) + 2;
    return kItemUnits + (s.window > 0 && seen < all ? seen : all);
}

// Units of the first `blocks` blocks of a head, all of them whole.
__host__ __device__ inline int units_before(const Shape &s, const Span &q, int blocks) {
    const int TB = s.block_tokens;
    uint32_t u = static_cast<uint32_t>(blocks) * kItemUnits;  // (what a window takes away again may pass 32 bits)
    // ends: blocks from i0 on end past position 0
    const int i0 = q.past >= 0 ? 0 : fast_div(-q.past, s.fd_block);
    if (blocks > i0)
        u += floor_sum(blocks - i0, q.past + (i0 + 1) * TB + (1 << s.tile_log2) - 1, TB, s.tile_log2, s.period_log2);
    if (s.window > 0) {
        // firsts: blocks from j0 on begin past key 0
        const long long before = static_cast<long long>(s.window) - 1 - q.past;
        const int j0 = before > 0 ? fast_div(static_cast<int>(before < 0x7ffffe00 ? before : 0x7ffffe00) + TB - 1, s.fd_block) : 0;
        if (blocks > j0) u -= floor_sum(blocks - j0, q.past + j0 * TB + 1 - s.window, TB, s.tile_log2, s.period_log2);
    }
    return static_cast<int>(u);
}
// Units of a head in all.
__host__ __device__ inline int head_units(const Shape &s, const Span &q) {
    if (q.n <= 0) return 0;
    const int last = blocks_of(s, q.n) - 1;
    return (last > 0 ? units_before(s, q, last) : 0) + kItemUnits + tiles_of(s, q, last);
}

// Units of a CTA, but for the last one's, which may be fewer: those of `most` CTAs that
// share W, and kCtaUnits at least.
__host__ __device__ inline int cta_units(int W, const FastDiv &most) {
    const int share = fast_div(W + static_cast<int>(most.d) - 1, most);
    return share > kCtaUnits ? share : kCtaUnits;
}

// What a CTA does at a time: an item, or the part of its tiles that the CTA has.
struct Segment {
    Span span;
    int seq, kvh, head;        // the sequence, the KV head, the first query head
    int token, tokens, heads;  // the first new token (a row of q), how many, query heads of each
    int pos;                   // of the first token
    int tile0, n;              // key tiles
    int of_item;               // tiles of the item
    int begins, whole;         // has the item's first tile; has all of them
    int item_last;             // unit, of the item
};

// A CTA's place in the line.
struct Walk {
    int u, end;                 // the next unit, and the one after the CTA's last
    int seq, kvh, part, block;  // part: of the KV head's query heads
    int skip;                   // units of the item before u
    Span span;
};

// The next segment (false: none is left).  spans(s) gives sequence s.
template <class Spans>
__host__ __device__ inline bool next_segment(const Shape &s, int num_seqs, const Spans &spans, Walk &w, Segment &g) {
#pragma unroll 1
    while (w.u < w.end) {
        const int tiles = tiles_of(s, w.span, w.block), units = kItemUnits + tiles;
        const int left = units - w.skip, mine = w.end - w.u < left ? w.end - w.u : left;
        const int from = w.skip > kItemUnits ? w.skip - kItemUnits : 0;
        const int to = w.skip + mine > kItemUnits ? w.skip + mine - kItemUnits : 0;
        const bool nothing = tiles == 0 && w.skip == 0;  // an item without keys: its rows are zeroed
        g.span = w.span;
        g.seq = w.seq;
        g.kvh = w.kvh;
        g.head = g.kvh * s.group + w.part * s.item_heads;
        g.heads = s.group - w.part * s.item_heads < s.item_heads ? s.group - w.part * s.item_heads : s.item_heads;
        g.token = w.span.first + w.block * s.block_tokens;
        g.tokens = w.span.n - w.block * s.block_tokens < s.block_tokens ? w.span.n - w.block * s.block_tokens : s.block_tokens;
        g.pos = w.span.past + w.block * s.block_tokens;
        g.tile0 = tiles > 0 ? first_tile(s, w.span, w.block) + from : 0;
        g.n = to - from;
        g.of_item = tiles;
        g.begins = from == 0;
        g.whole = g.n == tiles;
        g.item_last = w.u + left - 1;
        // on to the next item
        w.u += mine;
        w.skip = 0;
        if (w.u < w.end && (w.block + 1) * s.block_tokens < w.span.n) {
            ++w.block;
        } else if (w.u < w.end) {
            w.block = 0;
            if (++w.part == s.head_parts) {
                w.part = 0;
                ++w.kvh;
            }
            if (w.kvh == s.kv_heads) {
                w.kvh = 0;
                do {
                    if (++w.seq >= num_seqs) {
                        w.u = w.end;
                        break;
                    }
                    w.span = spans(w.seq);
                } while (w.span.n <= 0);
            }
        }
        if (g.n > 0 || nothing) return true;
    }
    return false;
}

// An item that several CTAs have, as the CTA with its first tile writes it down for
// the fold: query rows, and the CTAs from this one on that have a part.
struct CutItem {
    int token, head, tokens, heads;
    int parts;  // 0: no such item
};

}  // namespace chunk
}  // namespace pd
