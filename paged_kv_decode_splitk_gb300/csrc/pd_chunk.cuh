// pd_chunk.cuh -- attention of new tokens over the paged cache that holds them.
//
// What it computes.  For a new token at position p and each query head,
//   out = sum_j w_j V[j] / sum_j w_j,   w_j = 2^(x_j - m),   x_j = q.K[j] scale log2(e),
// over the keys j it sees, max(0, p + 1 - window) to p, in one pass over them: the
// reference m is the largest score of the first 64 columns that hold a key of the row's,
// raised by whole numbers when the weights of 64 keys sum past 2^15, so that no other
// maximum is taken and the sums are scaled exactly.
//
// GB300 mapping.
//   * An item is a block of new tokens with the query heads of a KV head, up to 256
//     rows (128 at head dims above 128), and the key tiles that any of its rows sees.
//     Items lie in one line of work units, of which every CTA (one an SM) takes the
//     same share (pd_chunk_plan.h).  What a border cuts leaves partials of (m, l, o).
//   * Warp 0 walks the CTA's part of the line and hands each segment to the other warps,
//     up to eight ahead; it loads K tiles, warp 2 V tiles, by TMA boxes of 64 columns x as
//     many tokens as lie together in a cache block, through the block table into a ring
//     (128-byte swizzle); warp 3 (over FP8 the first of the softmax) an item's queries,
//     whose rows are tokens by heads, as soon as the last item's scores are done.  One thread of warp 1 issues
//     tcgen05.mma: S (128 rows x a tile) into TMEM, then O += P V with P read from TMEM,
//     64 keys at a time, while the softmax is at the next 64.
//   * Two groups of four warps do the softmax, a thread a row.  With more than 128
//     rows each group has 128 of them and both meet every tile that their rows see;
//     with fewer the groups take the tiles in turn, each with an O of its own, folded
//     on the way out.  At head dims above 128 one O fills TMEM: one group, two S.
//   * Four warps take O out, to the results or the partials, while the softmax and the
//     products are at the next item.
//   * Only the 32 columns of a tile that hold a border of a row's keys are masked, in
//     TMEM, in front of the one code that weighs.  Code is what an SM's instruction cache
//     holds least of, so there is one copy of each part: at two thirds of its first room
//     single tokens took 100 us for 105 and FP8 chunks 306 for 341.  V rows past the
//     sequence, or before every row's window, are zeroed, so that whatever the cache's slots
//     hold there meets no product; boxes that lie there wholly are not read at all.
//   * P is rounded to BF16 (half a step: 2^-8 of each weight), the form the tensor
//     core multiplies with a BF16 V; l sums the unrounded weights in FP32, S, O, m and l
//     are FP32.  An FP8 cache is converted to f16 tiles (exactly) by warps 2 and 3, q
//     to f16 under a power of two for each row by the softmax warps, and P is f16
//     there (2^-11; weights below 2^-13 of the row's largest are off by up to 2^-24
//     of it).
//
// What bounds it.  Long prompts: the tensor core (a prompt of 8192 tokens, 32 heads of 128
// over 8: 327 to 340 us in a graph, 1620 to 1680 TFLOP/s, 85 to 89% of a library product's;
// call after call, at the card's power limit, 337 to 366), whose operands at D = 128 also fill
// shared memory: a tile of 256 rows takes 2048 cycles of products, 2048 of shared memory and
// 1075 of softmax, and 2300 in all.  D = 64: nothing is full (900 TFLOP/s, 2600 cycles a tile:
// products and shared memory 1024 each, softmax 1075); a stream's scores, softmax and values
// follow one another, since P lies over S.  D = 256: nor there (1150, 2150 cycles for 128 rows
// and 64 keys: products 1024, shared memory 1536); two S and one O of 128 rows fill TMEM, whose
// softmax one group of four warps does.  FP8: shared memory, 320 KB a tile, and its conversion
// (1330; four converting warps more take 5% longer).  Single tokens: HBM (a step of 256 behind 2048 tokens 6140 GB/s).  Small calls:
// the way to the first tile, 4 us of it code that is not in the caches yet, and the fold.
// Short items: the way out, 2500 cycles a stream, beside the next item's first tiles (eight
// prompts of 1024 tokens 76.5 us, 900 TFLOP/s).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <cfloat>

#include "pd.h"
#include "pd_chunk.h"
#include "pd_device.cuh"
#include "pd_tcgen05.cuh"
#include "pd_tile.cuh"

namespace pd {
namespace chunk {

using namespace tile;

struct ChunkMaps {
    CUtensorMap k, v, q;
};

// Scores of the columns below the first live one become -infinity.
template <int BN>
__device__ __forceinline__ void mask_columns_below(uint32_t (&x)[BN], int first) {
#pragma unroll
    for (int i = 0; i < BN; ++i)
        if (i < first) x[i] = 0xff800000u;
}

// Sequence s's new tokens; none where token_starts does not name rows of the batch.
__device__ __forceinline__ Span span_of(const ChunkParams &p, int s, bool flag) {
    Span q = {s, 1, 0, p.context_lens[s]};
    if (p.token_starts) {
        const int a = p.token_starts[s], b = p.token_starts[s + 1];
        const bool bad = a < 0 || b < a || b > p.num_tokens;
        if (bad && flag) dev::flag_status(p.status, PD_DEV_BAD_GROUPS);
        q.first = a;
        q.n = bad ? 0 : b - a;
    }
    if (q.len < 0 || q.len > p.max_tokens || (p.token_starts && q.n > q.len)) {
        if (flag) dev::flag_status(p.status, PD_DEV_BAD_CONTEXT_LEN);
        q.len = q.len < 0 ? 0 : (q.len > p.max_tokens ? p.max_tokens : q.len);
    }
    q.past = q.len - q.n;
    return q;
}

// (loads without a cache policy: items of the same head read the same tiles, from L2)
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// A segment as warp 0 hands it to the others.
struct Task {
    int n;                            // key tiles; -1: no more segments
    int tile0, two;                   // the first; more than 128 rows
    int end0, first1;                 // two: tiles that the first 128 rows see, [0, end0), and the others, [first1, n)
    int token, tokens, head, heads;   // rows of q and query heads
    int pos, low, len;                // of the first token; the first key any row sees; the sequence's tokens
    int seq, kvh;
    int begins, whole, parts;         // has the item's first tile, has all; CTAs from this one on that have a part
};
constexpr int kTasks = 8;

// With more than 128 rows each stream has 128 of them, and need not meet the tiles
// that only the other's rows see.
__device__ __forceinline__ Task task_of(const ChunkParams &p, const Segment &g, int dpad, int end, int share) {
    const Shape &s = p.shape;
    Task t;
    t.n = g.n;
    t.tile0 = g.tile0;
    t.two = dpad <= 128 && g.tokens * s.item_heads > kRowTile;
    const int last = g.pos + min(fast_div(kRowTile - 1, p.fd_heads), g.tokens - 1);  // the last position of the first 128 rows
    t.end0 = min(g.n, max(0, (last >= 0 ? (last >> s.tile_log2) + 1 : 0) - g.tile0));
    t.first1 = min(g.n, max(0, (first_key(s, g.pos + fast_div(kRowTile, p.fd_heads)) >> s.tile_log2) - g.tile0));
    t.token = g.token;
    t.tokens = g.tokens;
    t.head = g.head;
    t.heads = g.heads;
    t.pos = g.pos;
    t.low = first_key(s, g.pos);
    t.len = g.span.len;
    t.seq = g.seq;
    t.kvh = g.kvh;
    t.begins = g.begins;
    t.whole = g.whole;
    t.parts = 1;
#pragma unroll 1
    for (int u = end; g.begins && u <= g.item_last; u += share) ++t.parts;  // (once a CTA at most)
    return t;
}

// Shared-memory plan (bytes from the 1024-aligned base).
template <int DPAD, bool KV8>
struct Plan {
    static constexpr bool kOne = DPAD > 128;  // one stream, S double-buffered
    static constexpr int kTile = tile_tokens(DPAD);
    static constexpr int kBlock = block_rows(DPAD);
    static constexpr int kPart = 64;  // keys whose weights are handed on together
    static constexpr int kStageBytes = kTile * DPAD * 2;
    static constexpr int kStages = KV8 ? 3 : (DPAD == 64 ? 6 : 4);
    static constexpr int kRawBytes = KV8 ? kTile * DPAD : 0;
    static constexpr int kRawStages = KV8 ? 3 : 0;
    static constexpr int q = 0;             // [DPAD / 64][kBlock rows][128 bytes]
    static constexpr int ring = q + kBlock * DPAD * 2;
    static constexpr int raw = ring + kStages * kStageBytes;
    static constexpr int bars = raw + kRawStages * kRawBytes;
    static constexpr int misc = bars + 64 * 8;
    static constexpr int tasks = misc + 32 + 16 * 4;
    static constexpr int row_scale = tasks + (kTasks * static_cast<int>(sizeof(Task)) + 15) / 16 * 16;
    static constexpr int stream_ml = row_scale + (KV8 ? 2 * kBlock * 4 : 0);
    static constexpr int total = 1024 + stream_ml + 2 * 2 * kRowTile * 8;
    static constexpr int kThreads = 512;
};

template <int DPAD, bool KV8>
__global__ void __launch_bounds__(Plan<DPAD, KV8>::kThreads, 1)
    chunk_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkParams p) {
    using L = Plan<DPAD, KV8>;
    constexpr int BN = L::kTile;
    constexpr int BR = L::kBlock;
    constexpr int NST = L::kStages;
    constexpr int NT = L::kThreads;
    constexpr bool ONE = L::kOne;
    constexpr int HB = L::kPart, PARTS = BN / HB;
    constexpr int CHUNKS = DPAD / 8;  // 16-byte chunks of a 16-bit row
    constexpr uint32_t kDescS = tc::instr_desc(KV8 ? 0 : 1, kRowTile, BN, false);
    constexpr uint32_t kDescO = tc::instr_desc(KV8 ? 0 : 1, kRowTile, DPAD, true);
    const float kNegInf = -__int_as_float(0x7f800000);

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t base = dev::smem_addr(smem);
    // barriers: full[NST], empty[NST], raw_full[3], raw_empty[3], landed[NST], s[2],
    // p[4], o, half[2], q[2], q_free, tail, done[2], o_free[2], ml[4], task_full[8], task_free[8]
    const uint32_t bars = base + L::bars;
    const uint32_t bar_full = bars, bar_empty = bar_full + 8 * NST, bar_rfull = bar_empty + 8 * NST,
                   bar_rempty = bar_rfull + 24, bar_land = bar_rempty + 24, bar_s = bar_land + 8 * NST, bar_p = bar_s + 16,
                   bar_o = bar_p + 32, bar_h = bar_o + 8, bar_q = bar_h + 16, bar_qfree = bar_q + 16, bar_tail = bar_qfree + 8, bar_done = bar_tail + 8,
                   bar_ofree = bar_done + 16, bar_ml = bar_ofree + 16, bar_task = bar_ml + 32, bar_tfree = bar_task + 8 * kTasks,
                   bar_qraw = bar_land;  // (FP8: no tile lands apart)
    static_assert(3 * NST + 6 + 21 + 2 * kTasks <= 64, "barrier region");
    volatile int *gave_up = reinterpret_cast<int *>(smem + L::misc);
    uint32_t *tmem_s = reinterpret_cast<uint32_t *>(smem + L::misc + 4);
    int *start = reinterpret_cast<int *>(smem + L::misc + 8);  // the CTA's first sequence, its units before the CTA's first, a head's units
    int *sums = reinterpret_cast<int *>(smem + L::misc + 32);               // [NT / 32] of the warps

    // (the warp's number from one lane, so that the compiler knows it to be the
    // same on all: the product warp's operands then live in uniform registers)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    // ---- set-up that reads no global memory -----------------------------------
    if (warp == 0) {
        // (arrivals of each barrier, in the order above; the first set has 32 of them at most)
        constexpr int kReaders = 3 + (ONE ? 4 : 8) + 4;  // warps that read a task
        auto count = [](int i) {
            if (i < NST) return KV8 ? kConverters / 32 : 1;  // full
            if (i < 2 * NST + 3) return 1;                   // empty, raw_full
            if (i < 2 * NST + 6) return kConverters / 32;    // raw_empty
            i -= 3 * NST + 6;
            if (i < 2) return 1;    // landed, s
            if (i < 6) return 4;    // p
            if (i < 9) return 1;    // o, half
            if (i < 11) return KV8 ? 4 : 1;  // q
            if (i < 15) return 1;   // q_free, tail, done
            if (i < 21) return 4;   // o_free, ml
            return i < 21 + kTasks ? 1 : kReaders;  // task_full, task_free
        };
#pragma unroll
        for (int i = lane; i < 3 * NST + 6 + 21 + 2 * kTasks; i += 32) dev::mbar_init(bars + 8 * i, count(i));
        dev::fence_mbar_init();
    }
    if (tid == 0) {
        *gave_up = 0;
        dev::prefetch_tensormap(&maps.k);
        dev::prefetch_tensormap(&maps.v);
        dev::prefetch_tensormap(&maps.q);
    }
    if (warp == 1) tc::tmem_alloc_512(dev::smem_addr(tmem_s));
    dev::griddep_wait();  // q, the caches, tables and lengths are final

    // ---- the CTA's place in the line of units -----------------------------------
    // (the units of all sequences are summed by all threads, and those of the stripe of
    // sequences that has the CTA's first unit again; one warp finds the block)
    const auto spans = [&](int s) { return span_of(p, s, false); };
    Walk walk = {};
    int share = 0;
    {
        int all = 0;     // units of this thread's sequences
        int before = 0;  // of the stripes before
        const int stripes = (p.num_seqs + NT - 1) / NT;
        bool found = false;
        // the first round counts, the second looks for the place, which the first does
        // where there is one stripe alone
#pragma unroll 1
        for (int i = 0; i < 2 * stripes && !found; ++i) {
            const bool look = i >= stripes || stripes == 1;
            const int s = (i < stripes ? i : i - stripes) * NT + tid;
            const int of_head = s < p.num_seqs ? head_units(p.shape, span_of(p, s, blockIdx.x == 0 && i < stripes)) : 0;
            const int mine = p.shape.heads * of_head;
            all = add_units(all, mine);
            if (!look && i + 1 < stripes) continue;
            int upto = look ? mine : all;  // with those of the threads before it in the warp
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto = add_units(upto, o);
            }
            if (lane == 31) sums[warp] = upto;
            tc::fence_before();
            __syncthreads();
            tc::fence_after();
            // (the warps' sums added by one instruction, their upper bits to see whether that overflows)
            const int of_warp = lane < NT / 32 ? sums[lane] : 0;
            const bool over = __reduce_add_sync(0xffffffffu, of_warp >> 10) > kMaxUnits >> 10;
            const int stripe = over ? kMaxUnits + 1 : __reduce_add_sync(0xffffffffu, of_warp);
            const int from = before + upto - mine + __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0);
            if (i == stripes - 1) {  // all units
                share = cta_units(stripe, p.ctas);
                walk.u = blockIdx.x * share;
                walk.end = min(stripe, walk.u + share);
                if (stripe > p.most_units && tid == 0 && blockIdx.x == 0) dev::flag_status(p.status, PD_DEV_BAD_GROUPS);
                if (walk.u >= walk.end || stripe > p.most_units) walk.u = walk.end = 0;  // (too many: sequences overlap)
            }
            if (look) {
                if (from <= walk.u && walk.u < from + mine) {
                    start[0] = s;
                    start[1] = walk.u - from;
                    start[2] = of_head;
                }
                before += stripe;
                found = before > walk.u || walk.end == 0;
            }
            __syncthreads();
        }
        // Everything before this grid is done: the fold may come to wait for its end.
        dev::griddep_launch_dependents();
        if (warp == 0 && walk.end > 0) {
            walk.seq = start[0];
            walk.span = spans(walk.seq);
            const int of_head = start[2];
            int head = static_cast<int>(__fdividef(static_cast<float>(start[1]), static_cast<float>(of_head)));  // (or one beside it)
            int rest = start[1] - head * of_head;
            if (rest < 0) {
                --head;
                rest += of_head;
            } else if (rest >= of_head) {
                ++head;
                rest -= of_head;
            }
            walk.kvh = p.shape.head_parts == 1 ? head : head / p.shape.head_parts;
            walk.part = head - walk.kvh * p.shape.head_parts;
            walk.skip = rest;
#pragma unroll 1
            for (int n = blocks_of(p.shape, walk.span.n); n > 1;) {  // the last block that begins at or before the unit
                const int step = (n + 31) / 32, i = lane * step;
                const int at = units_before(p.shape, walk.span, walk.block + min(i, n - 1));
                const int pick = __popc(__ballot_sync(0xffffffffu, i < n && at <= rest)) - 1;
                walk.block += pick * step;
                n = min(step, n - pick * step);
                walk.skip = rest - __shfl_sync(0xffffffffu, at, pick);
            }
        }
    }
    constexpr uint32_t tmem = 0;  // all 512 columns: the allocation starts at the first
    const int bs = static_cast<int>(p.block_size.d);
    const int IH = p.shape.item_heads;
    // Warp 0 walks the line and hands each segment to the other warps, a few ahead.
    Task *const tasks = reinterpret_cast<Task *>(smem + L::tasks);
    int task = 0;           // the place of the next one
    uint32_t task_ph = 0;
    auto next_task = [&] {  // (the warp waits; false: there are no more)
        if (!wait_bar(bar_task + 8 * task, task_ph, gave_up)) return false;
        return tasks[task].n >= 0;
    };
    auto task_done = [&] {
        arrive_warp(bar_tfree + 8 * task, lane);
        if (++task == kTasks) {
            task = 0;
            task_ph ^= 1;
        }
    };
    // An item's queries into shared memory, by a warp.
    auto load_queries = [&](const Task &sg, uint32_t bar) {
        const int boxes = (sg.tokens + p.query_box - 1) / p.query_box, bytes = p.query_box * IH * 128;  // of 64 columns
        if (lane == 0) dev::mbar_arrive_expect_tx(bar, boxes * bytes * (DPAD / 64));
        __syncwarp();
#pragma unroll 1
        for (int b = lane; b < boxes * (DPAD / 64); b += 32) {
            const int c = b % (DPAD / 64), at = b / (DPAD / 64);
            tma_load_3d(base + L::q + c * (BR * 128) + at * bytes, &maps.q, bar, c * 64, sg.head, sg.token + at * p.query_box);
        }
    };
    // Registers: 512 threads were launched with 128 each, and 128 x 88 + 256 x 144 + 128 x
    // 136 is what all of them have.
    static_assert(NT == 512 && 88 + 2 * 144 + 136 <= 4 * 128, "the shares add up to the launch's registers");

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");

    if (warp == 0 || (!KV8 && warp == 2)) {
        // ---- loads: K and V tiles in the order the products take them ------------
        constexpr int COLS = KV8 ? (DPAD < 128 ? DPAD : 128) : kBoxCols;  // columns of a box
        const int CT = p.box_tokens;                         // tokens of a box
        const int NCH = BN / CT, NBOX = NCH * (DPAD / COLS);
        constexpr int DEPTH = KV8 ? L::kRawStages : NST;
        constexpr int BYTES = KV8 ? L::kRawBytes : L::kStageBytes;
        const uint32_t full = KV8 ? bar_rfull : bar_full, empty = KV8 ? bar_rempty : bar_empty;
        const uint32_t stage0 = base + (KV8 ? L::raw : L::ring);
        const int chunk = lane % NCH, col = lane / NCH;
        int st = 0;
        uint32_t ph = 0;       // phase of the stage about to be filled
        uint32_t land_ph = 0;  // of the landing barriers, a bit each
        bool ok = true;
        long long issued = 0;
        auto load_all = [&](const Task &sg) {
            const int32_t *ids = p.block_table + static_cast<long long>(sg.seq) * p.max_blocks;
            const int ahead = sg.two ? 1 : 2;
            const int low = sg.low, end = sg.pos + sg.tokens, len = sg.len;
            const bool mine = lane < NBOX;  // a box a lane
            // Block ids, 32 boxes' rows (chunks of CT tokens) at a time: lane l of `now`
            // has chunk 32 w + l of the segment, `then` the 32 after them, asked for a
            // window ahead.  Where no row sees a token of the chunk, and for a bad
            // id (-1), it is one outside the cache, which reads zeros.
            const int lg = 31 - __clz(NCH);
            auto ids_of = [&](int w) -> int {
                const int c = 32 * w + lane, j = c >> lg;
                const int tok = (sg.tile0 + j) * BN + (c & (NCH - 1)) * CT;
                if (j >= sg.n || tok >= end || tok + CT <= low) return p.num_blocks;
                const int id = __ldg(ids + fast_div(tok, p.block_size));
                return id >= 0 && id < p.num_blocks ? id : -1;
            };
            int w = 0, now = ids_of(0), then = ids_of(1), before = now;
            auto next_stage = [&] {
                ++issued;
                if (++st == DEPTH) {
                    st = 0;
                    ph ^= 1;
                }
                return true;
            };
            auto load = [&](bool is_v, int j) {
                if (!KV8 && is_v != (warp == 2)) return next_stage();  // the other warp's
                const int at = (sg.tile0 + j) * BN, tok = at + chunk * CT;
                const int wj = j << lg >> 5;
                if (wj > w) {
                    w = wj;
                    before = now;
                    now = then;
                    then = ids_of(w + 1);
                }
                int id = __shfl_sync(0xffffffffu, wj == w ? now : before, ((j << lg) + chunk) & 31);
                if (id < 0) {
                    if (mine) dev::flag_status(p.status, PD_DEV_BAD_BLOCK_ID);
                    id = p.num_blocks;
                }
                if (!wait_bar(empty + 8 * st, ph ^ 1, gave_up)) return false;
                const uint32_t dst = stage0 + st * BYTES;
                // A box of live and dead tokens holds whatever the cache's slots past the
                // sequence, or before every row's window, hold; a dead V row must not
                // reach the product (0 x NaN), so those rows are zeroed before the
                // tile is handed on.  It lands at a barrier of its stage.
                const int nl = max(0, low - at), nv = min(BN, len - at);
                const bool some = !KV8 && is_v && ((nl | nv) & (CT - 1));
                const uint32_t bar = (some ? bar_land : full) + 8 * st;
                if (lane == 0) dev::mbar_arrive_expect_tx(bar, BYTES);
                __syncwarp();
                if (mine) {
                    const int sub = tok - fast_div(tok, p.block_size) * bs;
                    const uint32_t to = dst + col * (BN * (KV8 ? COLS : 128)) + chunk * (CT * (KV8 ? COLS : 128));
                    const CUtensorMap *map = is_v ? &maps.v : &maps.k;
                    const int c1 = p.tok_dim == 1 ? sub : sg.kvh, c2 = p.tok_dim == 1 ? sg.kvh : sub;
                    tma_load_4d(to, map, bar, col * COLS, c1, c2, id);
                }
                if (some) {
                    const uint32_t lph = (land_ph >> st) & 1;
                    land_ph ^= 1u << st;
                    if (!wait_bar(bar, lph, gave_up)) {
                        if (lane == 0) dev::mbar_wait_bounded(bar, lph, 100000000ull);  // (its copies land before the CTA ends)
                        return false;
                    }
                    uint8_t *tile = smem + L::ring + st * BYTES;
                    const int l0 = nl & ~(CT - 1), v1 = (nv + CT - 1) & ~(CT - 1);
#pragma unroll 1
                    for (int b = 0; b < DPAD / 64; ++b) {
#pragma unroll 1
                        for (int i = l0 * 8 + lane; i < nl * 8; i += 32)
                            *reinterpret_cast<uint4 *>(tile + b * (BN * 128) + i * 16) = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                        for (int i = nv * 8 + lane; i < v1 * 8; i += 32)
                            *reinterpret_cast<uint4 *>(tile + b * (BN * 128) + i * 16) = make_uint4(0, 0, 0, 0);
                    }
                    tc::fence_async_shared();
                    __syncwarp();
                    if (lane == 0) arrive(full + 8 * st);
                }
                return next_stage();
            };
            // (a step of two loads as two turns of the loop: the code of one)
            const int n = sg.n;
#pragma unroll 1
            for (int i = 0; ok && i < 2 * (n + ahead - 1); ++i) {
                const bool is_v = i & 1;
                const int j = (i >> 1) - (is_v ? ahead - 1 : 0);
                if (j >= 0 && j < n) ok = load(is_v, j);
            }
        };
        // (warp 0 makes the tasks as it goes)
#pragma unroll 1
        while (ok) {
            const bool makes = warp == 0;
            if (makes) {
                Segment g;
                Task t = {};
                t.n = -1;
                if (next_segment(p.shape, p.num_seqs, spans, walk, g)) t = task_of(p, g, DPAD, walk.end, share);
                if (!(ok = wait_bar(bar_tfree + 8 * task, task_ph ^ 1, gave_up))) break;
                if (lane == 0) {
                    tasks[task] = t;
                    arrive(bar_task + 8 * task);
                }
                __syncwarp();
            }
            if (!makes && !wait_bar(bar_task + 8 * task, task_ph, gave_up)) break;
            if (tasks[task].n < 0) break;
            load_all(tasks[task]);
            if (!makes) arrive_warp(bar_tfree + 8 * task, lane);
            if (++task == kTasks) {
                task = 0;
                task_ph ^= 1;
            }
        }
        // every release of a stage has arrived before this CTA ends
#pragma unroll 1
        for (long long i = issued < DEPTH ? 0 : issued - DEPTH; ok && i < issued; ++i)
            ok = wait_bar(empty + 8 * static_cast<int>(i % DEPTH), static_cast<uint32_t>((i / DEPTH) & 1), gave_up);
        if (!ok && lane == 0) {
            // a wait ran out: let the copies in flight land before the CTA ends
            dev::flag_status(p.status, PD_DEV_WAIT_TIMEOUT);
            const long long last = issued < DEPTH ? issued : DEPTH;
#pragma unroll 1
            for (long long i = issued - last; i < issued; ++i)
                dev::mbar_wait_bounded(full + 8 * static_cast<int>(i % DEPTH), static_cast<uint32_t>((i / DEPTH) & 1),
                                       100000000ull);
        }
    } else if (warp == 1) {
        // ---- products: one thread issues them all, in the order S, P V, S, ... of
        // the streams in turn.  What it waits for is looked at as early as the order
        // allows: the queue of products is short, and whatever this thread spends
        // between two of them the tensor core may spend idle.
        if (tc::elect_one()) {
            int st = 0;
            uint32_t ph = 0, pph = 0, qph = 0, fph = 0;  // phases: of the ring; a bit for each stream
            bool ok = true;
            const uint32_t qa = base + L::q, ra = base + L::ring;
            const uint64_t q_desc = tc::smem_desc(qa, 16), k_desc = tc::smem_desc(ra, 16), v_desc = tc::smem_desc(ra, BN * 128);
            // (a negative scale: q as its negation, by the product itself)
            const uint32_t desc_s = kDescS | (!KV8 && p.negative ? 1u << 13 : 0u);
            // the next tile of the ring (K or V), once it has landed
            auto take = [&](int &stage) {
                stage = st;
                if (!wait_one(bar_full + 8 * st, ph, gave_up)) return false;
                if (++st == NST) {
                    st = 0;
                    ph ^= 1;
                }
                return true;
            };
            auto scores = [&](int buf, int qt, int stage) {
                const uint64_t qd = q_desc + qt * (kRowTile * 128 / 16), kd = k_desc + stage * (L::kStageBytes / 16);
                tc::fence_after();
#pragma unroll
                for (int k = 0; k < DPAD / 16; ++k)
                    tc::mma_ss(tmem + buf * 128, qd + ((k / 4) * (BR * 128) + (k % 4) * 32) / 16,
                               kd + ((k / 4) * (BN * 128) + (k % 4) * 32) / 16, desc_s, k > 0);
                tc::commit(bar_s + 8 * buf);
            };
            // O += P V as the parts of P come: the first while the softmax is at the second
            auto values = [&](int buf, int o, int stage, bool accumulate, bool done) {
                const uint64_t vd = v_desc + stage * (L::kStageBytes / 16);
                if (!accumulate) {  // (the last item's O has left)
                    if (!wait_one(bar_ofree + 8 * o, ((fph >> o) & 1) ^ 1, gave_up)) return false;
                    fph ^= 1u << o;
                }
#pragma unroll
                for (int h = 0; h < PARTS; ++h) {
                    if (!wait_one(bar_p + 8 * (PARTS * buf + h), (pph >> buf) & 1, gave_up)) return false;
                    tc::fence_after();
#pragma unroll
                    for (int k = h * (HB / 16); k < (h + 1) * (HB / 16); ++k)
                        tc::mma_ts(tmem + 256 + o * DPAD, tmem + buf * 128 + k * 8, vd + k * (2048 / 16), kDescO, accumulate || k > 0);
                    if (h + 1 < PARTS) tc::commit(bar_h + 8 * o);
                }
                pph ^= 1u << buf;
                if (ONE) tc::commit(bar_o);
                if (done) tc::commit(bar_done + 8 * o);
                return true;
            };
            auto release = [&](int stage) { tc::commit(bar_empty + 8 * stage); };
            auto queries_done = [&] { tc::commit(bar_qfree); };
            auto queries = [&](int t) {  // (from boxes of q all rows come at once)
                if (!KV8 && t > 0) return true;
                const bool got = wait_one(bar_q + 8 * t, (qph >> t) & 1, gave_up);
                qph ^= 1u << t;
                return got;
            };
            auto task_given = [&] {
                arrive(bar_tfree + 8 * task);
                if (++task == kTasks) {
                    task = 0;
                    task_ph ^= 1;
                }
            };
            for (;; task_given()) {
                if (!(ok = wait_one(bar_task + 8 * task, task_ph, gave_up))) break;
                const int n = tasks[task].n, two = tasks[task].two, end0 = tasks[task].end0, first1 = tasks[task].first1;
                if (n < 0) break;
                if (n == 0) continue;
                int ks = 0, vs = 0;
                if (!(ok = queries(0))) break;
                // (an item's first scores by the loop's own code: a copy of it is not in the
                // instruction cache when its turn comes, 1500 cycles an item)
                if (!ONE && two) {
#pragma unroll 1
                    for (int j = -1; ok && j < n; ++j) {
                        const bool more = j + 1 < n;
                        const int v = vs;
                        if (more && !(ok = take(ks))) break;
                        if (j >= 0 && j < end0 && !(ok = values(0, 0, v, j > 0, j + 1 == end0))) break;
                        if (more && j + 1 < end0) scores(0, 0, ks);
                        if (KV8 && j < 0 && !(ok = queries(1))) break;
                        if (j >= first1 && !(ok = values(1, 1, v, j > first1, !more))) break;
                        if (j >= 0) release(v);  // (before the scores: a commit waits for all that came before)
                        if (more) {
                            if (j + 1 >= first1) scores(1, 1, ks);
                            release(ks);
                            if (j + 2 == n) queries_done();
                            ok = take(vs);
                        }
                    }
                } else {
#pragma unroll 1
                    for (int j = -2; ok && j < n; ++j) {
                        const bool next = j + 2 < n;
                        const int t = j & 1;
                        if (j >= 0 && !(ok = take(vs))) break;
                        if (next && !(ok = take(ks))) break;
                        if (j >= 0) {
                            if (!(ok = values(t, ONE ? 0 : t, vs, j > (ONE ? 0 : 1), j + (ONE ? 1 : 2) >= n))) break;
                            release(vs);
                        }
                        if (next) {  // scores of tile j + 2, whose keys are the next of the ring
                            scores(t, 0, ks);
                            release(ks);
                            if (j + 3 == n) queries_done();
                        }
                    }
                }
                if (!ok) break;
            }
            if (!ok) {
                // let the products in flight end before TMEM is freed
                tc::commit(bar_tail);
                dev::mbar_wait_bounded(bar_tail, 0, 100000000ull);
            }
        }
        __syncwarp();
    } else if (!KV8) {
        // ---- queries: the rows of the next item, once the last one's scores are done ----
        uint32_t ph = 0;
        bool ok = true, any = false;
        for (; ok && next_task(); task_done()) {
            const Task &sg = tasks[task];
            if (sg.n == 0) continue;
            if (!(ok = wait_bar(bar_qfree, ph ^ 1, gave_up))) break;
            load_queries(sg, bar_q);
            ph ^= 1;
            any = true;
        }
        // the products have taken the last rows before this CTA ends
        if (ok && any) ok = wait_bar(bar_qfree, ph ^ 1, gave_up);
        if (!ok && any && lane == 0) dev::mbar_wait_bounded(bar_q, ph ^ 1, 100000000ull);
    } else {
        // ---- FP8: each landed tile of codes into an f16 tile of the ring (k_scale is in
        // the softmax scale, v_scale in the results) ----
        const Widen<DPAD, BN> widen(warp - 2, lane);
        int rs = 0, st = 0;
        uint32_t rph = 0, ph = 0;
        bool ok = true;
        long long handed = 0;
        auto convert = [&](bool is_v, int low, int end) {
            if (!wait_bar(bar_rfull + 8 * rs, rph, gave_up) || !wait_bar(bar_empty + 8 * st, ph ^ 1, gave_up)) return false;
            const uint8_t *src = smem + L::raw + rs * L::kRawBytes;
            uint8_t *dst = smem + L::ring + st * L::kStageBytes;
            widen(src, dst, is_v && (low > 0 || end < BN), low, end);
            tc::fence_async_shared();
            arrive_warp(bar_full + 8 * st, lane);
            arrive_warp(bar_rempty + 8 * rs, lane);  // (the reads come before the loads that refill it)
            if (++rs == L::kRawStages) {
                rs = 0;
                rph ^= 1;
            }
            ++handed;
            if (++st == NST) {
                st = 0;
                ph ^= 1;
            }
            return true;
        };
        for (; ok && next_task(); task_done()) {
            const Task &sg = tasks[task];
            const int ahead = sg.two ? 1 : 2, low = sg.low, len = sg.len;
            const int n = sg.n;
#pragma unroll 1
            for (int i = 0; ok && i < 2 * (n + ahead - 1); ++i) {
                const bool is_v = i & 1;
                const int j = (i >> 1) - (is_v ? ahead - 1 : 0), at = (sg.tile0 + j) * BN;
                if (j >= 0 && j < n) ok = convert(is_v, low - at, len - at);
            }
        }
        // every release of a stage has arrived before this CTA ends
#pragma unroll 1
        for (long long i = handed < NST ? 0 : handed - NST; ok && i < handed; ++i)
            ok = wait_bar(bar_empty + 8 * static_cast<int>(i % NST), static_cast<uint32_t>((i / NST) & 1), gave_up);
    }
    } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    if (warp < (ONE ? 8 : 12)) {
        // ---- softmax: a thread per row -----------------------------------------------
        const int t = (warp - 4) >> 2;            // the stream
        const int r = (warp & 3) * 32 + lane;     // the row of its tile
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t to = tmem + lanes + 256 + t * DPAD;
        const int D = p.head_dim;
        uint32_t sph = 0, oph = 0, hph = 0, qph = 0;  // phases, a bit for each buffer or stream
        bool ok = true, any = false;
        // FP8: the rows' scales, by the segments that have keys in turn in two places: the
        // other stream may still have to read the last one's when this one's are written (it
        // has by the time of a third: the queries of that come behind the second's last
        // scores, which were asked for behind all of the first's weights)
        float *row_scale = reinterpret_cast<float *>(smem + L::row_scale);
        int turn = 0, out_turn = 0;
        for (; ok && next_task(); task_done()) {
            const Task &sg = tasks[task];  // (read again wherever it is wanted, to hold no registers)
            const bool two = !ONE && sg.two;
            float scale = p.scale_log2;
            if constexpr (KV8) {
                row_scale = reinterpret_cast<float *>(smem + L::row_scale) + turn * BR;
                // -- this stream's query rows, a thread each, become f16 under a power of two that
                // brings the row's largest |q| into [2^14, 2^15), exactly but for values 2^-28
                // below it; its inverse joins the row's softmax scale.  With at most 128 rows
                // the streams share stream 0's.  (Rows from memory through registers, with the
                // largest by shuffles, took 12000 cycles an item.)
                if (sg.n > 0) {
                    if (warp == 4) {
                        if (!(ok = wait_bar(bar_qfree, qph ^ 1, gave_up))) break;
                        load_queries(sg, bar_qraw);
                    }
                    ok = wait_bar(bar_qraw, qph, gave_up);
                    if (!ok && tid == 128) dev::mbar_wait_bounded(bar_qraw, qph, 100000000ull);  // (its copies land before the CTA ends)
                    if (!ok) break;
                    qph ^= 1;
                }
                if ((two || t == 0) && sg.n > 0) {
                    const int row = t * kRowTile + r;
                    auto chunk = [&](int c) {
                        return reinterpret_cast<uint4 *>(smem + L::q + (c / 8) * (BR * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
                    };
                    __nv_bfloat162 big2 = __float2bfloat162_rn(0.f);
#pragma unroll 8
                    for (int c = 0; c < CHUNKS; ++c) {
                        const uint4 v = *chunk(c);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) big2 = __hmax2(big2, __habs2(reinterpret_cast<const __nv_bfloat162 &>(w[k])));
                    }
                    const float big = fmaxf(__low2float(big2), __high2float(big2));
                    const int ex = (__float_as_int(big) >> 23) & 0xff;                   // |q| < 2^(ex - 126)
                    const int up = min(max(141 - ex, -126), 127);                        // times 2^up: below 2^15
                    const float f = __int_as_float((127 + up) << 23 | (p.negative ? 1u << 31 : 0u));
                    const float down = up < 127 ? __int_as_float((127 - up) << 23) : 5.877471754111438e-39f;  // 2^-up
                    row_scale[row] = fmaxf(p.scale_log2 * down, FLT_MIN);
#pragma unroll 8
                    for (int c = 0; c < CHUNKS; ++c) {
                        uint4 v = *chunk(c);
                        v.x = dev::pack_f16x2(dev::bf16_lo_f32(v.x) * f, dev::bf16_hi_f32(v.x) * f);
                        v.y = dev::pack_f16x2(dev::bf16_lo_f32(v.y) * f, dev::bf16_hi_f32(v.y) * f);
                        v.z = dev::pack_f16x2(dev::bf16_lo_f32(v.z) * f, dev::bf16_hi_f32(v.z) * f);
                        v.w = dev::pack_f16x2(dev::bf16_lo_f32(v.w) * f, dev::bf16_hi_f32(v.w) * f);
                        *chunk(c) = v;
                    }
                    tc::fence_async_shared();
                    arrive_warp(bar_q + 8 * t, lane);
                }
            }
            // -- the row: its token and head, and the keys it sees.  (A row that is none,
            // past the item's tokens or heads, goes along with the last one's keys.)
            const int br = (two ? t * kRowTile : 0) + r;
            const int tk = fast_div(br, p.fd_heads);
            const bool live = tk < sg.tokens && br - tk * IH < sg.heads;
            const int at = sg.pos + min(tk, sg.tokens - 1);  // its position
            const int low = live ? first_key(p.shape, at) : sg.low;
            const int end = live ? at + 1 : sg.pos + sg.tokens;
            const int first_j = two ? (t ? sg.first1 : 0) : (ONE ? 0 : t), end_j = two && t == 0 ? sg.end0 : sg.n;
            const int end_all = __reduce_min_sync(0xffffffffu, end), low_all = __reduce_max_sync(0xffffffffu, low);  // of the warp's rows
            float m = kNegInf, l = 0.f;
            const float lift = live ? kLift : -kNegInf;
            bool begun = false, settled = false;  // a tile was seen; every row has its reference
            const int step = ONE || two ? 1 : 2;
#pragma unroll 1
            for (int j = first_j; j < end_j; j += step) {
                const int buf = ONE ? (j & 1) : t;
                const uint32_t ts = tmem + lanes + buf * 128;
                if (!(ok = wait_bar(bar_s + 8 * buf, (sph >> buf) & 1, gave_up))) break;
                sph ^= 1u << buf;
                tc::fence_after();
                if (KV8 && !begun) scale = row_scale[(two ? t * kRowTile : 0) + r];
                // -- A row's reference m is the largest score of its first 64 columns with a
                // key; after that no maximum is taken: weights may be as large as
                // kLift, and only when a row's weights of a part sum to more does its warp
                // look at the scores again and raise m (by a whole number, so that l and O
                // are scaled exactly).  FP32 and BF16 hold such weights as exactly as
                // weights below 1; kLift is what f16 holds.  Each part goes to the product
                // as it is done.
                const int tile_at = (sg.tile0 + j) * BN;
                auto hand = [&](const uint32_t (&pk)[HB / 2], int h) {
                    tc::st_columns<HB / 2>(ts + h * (HB / 2), pk);  // over scores that have been read
                    tc::wait_st();
                    tc::fence_before();
                    arrive_warp(bar_p + 8 * (PARTS * buf + h), lane);
                };
                bool waited = !ONE || !any;  // the last product onto O (that of the last item, too) is known to be done
                // What of a tile holds a border of some row's keys, 32 columns at a time: scores
                // outside become -infinity in tensor memory.
                if (tile_at + BN > end_all || tile_at < low_all) {
#pragma unroll 1
                    for (int c = 0; c < BN; c += 32) {
                        const bool over = tile_at + c + 32 > end_all, under = tile_at + c < low_all;
                        if (!over && !under) continue;
                        uint32_t x[32];
                        tc::ld_32x32(ts + c, x);
                        tc::wait_ld(x);
                        if (over) mask_columns<32>(x, end - tile_at - c);
                        if (under) mask_columns_below<32>(x, low - tile_at - c);
                        tc::st_32x32(ts + c, x);
                    }
                    tc::wait_st();
                }
                int part = 0;
                for (float most = lift;;) {
#pragma unroll 1
                    for (; part < PARTS; ++part) {
                        uint32_t x[HB], pk[HB / 2];
                        tc::ld_columns<HB>(ts + part * HB, x);
                        if (!settled) {  // rows without a reference take it, where they see any of the columns
                            const float mx = largest_of<HB>(x) * scale;
                            if (live && m == kNegInf) m = mx;
                            settled = __all_sync(0xffffffffu, !live || m > kNegInf);
                        }
                        const float sum = weigh<HB, KV8>(x, scale, m, pk);
                        if (__any_sync(0xffffffffu, sum > most)) break;
                        most = lift;
                        l += sum;
                        if (ONE && !waited) {
                            ok = wait_bar(bar_o, oph & 1, gave_up) && ok;  // (each phase of the barrier is waited for, in order)
                            oph ^= 1;
                        }
                        hand(pk, part);
                    }
                    if (part == PARTS) break;
                    // Rows raise their references: the products onto O have to be done, those of
                    // the last tile (with two streams they are where this one's scores are) and
                    // of the part before.  What their weights then sum to is taken as it is.
                    if (part > 0) {
                        ok = wait_bar(bar_h + 8 * t, (hph >> t) & 1, gave_up) && ok;
                    } else if (!waited) {
                        ok = wait_bar(bar_o, oph & 1, gave_up) && ok;
                        oph ^= 1;
                        waited = true;
                    }
                    tc::fence_after();
                    float mx = kNegInf, sum = 0.f;
#pragma unroll 1
                    for (int c = 0; c < HB; c += 32) {
                        uint32_t x[32], pk[16];
                        tc::ld_32x32(ts + part * HB + c, x);
                        tc::wait_ld(x);
                        mx = fmaxf(mx, largest_of<32>(x));
                        sum += weigh<32, KV8>(x, scale, m, pk);
                    }
                    // (a row's first 64 columns, with which there is no O yet, weigh 64 at most)
                    if (begun || part > 0) raise_reference<DPAD>(to, mx * scale, sum > lift, m, l);
                    most = -kNegInf;
                }
                begun = any = true;
                hph ^= 1u << t;
                if (!ok) break;
            }
            if (!ok) break;

            // -- the row's reference and sum for the way out, of the items that the stream had a
            // tile of, in turn in two places with a barrier each: by the time of a third the
            // first has been read, whose O had to leave before the second's products
            if (sg.n > 0) turn ^= 1;
            if (end_j > first_j) {
                reinterpret_cast<float2 *>(smem + L::stream_ml)[(out_turn * 2 + t) * kRowTile + r] = make_float2(m, l);
                arrive_warp(bar_ml + 8 * (2 * out_turn + t), lane);
                out_turn ^= 1;
            }
        }
    }
    } else {
    // ---- the way out: an item's O, as soon as its products are done, while the softmax
    // warps are at the next item ----------------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int r = (warp & 3) * 32 + lane, D = p.head_dim;
    const float2 *mls = reinterpret_cast<const float2 *>(smem + L::stream_ml);
    uint32_t mph = 0, dph = 0;  // phases of the streams' (m, l), a bit for each place, and O
    int turn = 0;               // the streams' places, a bit each
    bool ok = true, cut = false;
    while (ok && next_task()) {
        const Task &sg = tasks[task];
        const int n = sg.n, token = sg.token, tokens = sg.tokens, head = sg.head, heads = sg.heads;
        const bool two = !ONE && sg.two, whole = sg.whole;
        const int used = ONE ? (n > 0) : two ? (sg.end0 > 0 ? 1 : 0) | (n > sg.first1 ? 2 : 0) : (n > 0 ? 1 : 0) | (n > 1 ? 2 : 0);  // streams' O
        const long long slot = 2ll * blockIdx.x + (sg.begins ? 1 : 0);
        if (!whole && sg.begins && tid == 384) {
            p.cut[blockIdx.x] = {token, head, tokens, heads, sg.parts};
            cut = true;
        }
        task_done();
#pragma unroll 1
        for (int t = 0; ok && t < (two ? 2 : 1); ++t) {
            // (with at most 128 rows the streams' two partials of a row are folded)
            const int k1 = ONE || two ? t + 1 : 2;
            float2 ml[2] = {make_float2(kNegInf, 0.f), make_float2(kNegInf, 0.f)};
            for (int k = t; ok && k < k1; ++k) {
                if (!((used >> k) & 1)) continue;
                const int at = 2 * ((turn >> k) & 1) + k;
                ok = wait_bar(bar_ml + 8 * at, (mph >> at) & 1, gave_up);
                mph ^= 1u << at;
                turn ^= 1 << k;
                ml[k - t] = mls[at * kRowTile + r];
                ok = wait_bar(bar_done + 8 * k, (dph >> k) & 1, gave_up) && ok;
                dph ^= 1u << k;
            }
            if (!ok) break;
            tc::fence_after();
            const bool has0 = (used >> t) & 1 && ml[0].y != 0.f, has1 = k1 > t + 1 && (used >> 1) & 1 && ml[1].y != 0.f;
            const float M = fmaxf(has0 ? ml[0].x : kNegInf, has1 ? ml[1].x : kNegInf);
            const float f0 = !has0 ? 0.f : has1 ? dev::exp2_approx(ml[0].x - M) : 1.f, f1 = !has1 ? 0.f : has0 ? dev::exp2_approx(ml[1].x - M) : 1.f;
            const float l = (has0 ? ml[0].y * f0 : 0.f) + (has1 ? ml[1].y * f1 : 0.f);
            const float f = !whole ? 1.f : l == 0.f ? 0.f : __fdiv_rn(p.v_scale, l);
            // the row's sum: ln of it, or (m, l) of a partial
            const int br = t * kRowTile + r, tk = fast_div(br, p.fd_heads), part_rows = tokens * IH;
            if (whole) {
                if (p.lse && tk < tokens && br - tk * IH < heads)
                    p.lse[static_cast<long long>(token + tk) * p.num_q_heads + head + (br - tk * IH)] =
                        l == 0.f ? kNegInf : (M + log2f(l)) * 0.6931471805599453f;
            } else if (br < part_rows) {
                *reinterpret_cast<float2 *>(p.part_ml + (slot * p.slot_rows + br) * 2) = make_float2(M, l);
            }
            // 32 columns of this thread's row, scaled.  (A sum of 0 is one of no keys, whose O is 0.)
            const uint32_t from = tmem + lanes + 256 + t * DPAD;
            const bool any0 = (used >> t) & 1, any1 = k1 > t + 1 && (used >> 1) & 1;
            const uint64_t g0 = tc::pack_f32x2(f0 * f, f0 * f), g1 = tc::pack_f32x2(f1 * f, f1 * f);
            auto scaled = [](uint32_t &a, uint32_t &b, uint64_t f, uint64_t plus, bool add) {
                const uint64_t x = tc::pack_f32x2(__uint_as_float(a), __uint_as_float(b));
                float u, v;
                tc::unpack_f32x2(add ? tc::fma_f32x2(x, f, plus) : tc::mul_f32x2(x, f), u, v);
                a = __float_as_uint(u);
                b = __float_as_uint(v);
            };
            auto fetch = [&](int c, uint32_t (&x)[32]) {
                if (any0) {
                    tc::ld_32x32(from + c, x);
                    tc::wait_ld(x);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = 0;
                }
#pragma unroll
                for (int i = 0; i < 32; i += 2) scaled(x[i], x[i + 1], g0, 0, false);
                if (any1) {
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
                        uint32_t y[16];
                        tc::ld_32x16(from + DPAD + c + h, y);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            scaled(y[i], y[i + 1], g1, tc::pack_f32x2(__uint_as_float(x[h + i]), __uint_as_float(x[h + i + 1])), true);
                            x[h + i] = y[i];
                            x[h + i + 1] = y[i + 1];
                        }
                    }
                }
                if (c + 32 < DPAD) return;
                tc::fence_before();  // O has been read
                __syncwarp();
                if (lane == 0) {
                    if (any0) arrive(bar_ofree + 8 * t);
                    if (any1) arrive(bar_ofree + 8);
                }
            };
            if (whole) {
                const bool live = tk < tokens && br - tk * IH < heads;
                // Two threads their two rows, 32 bytes of one at a time (a whole sector).  (Each its
                // own row, 16 bytes at a time, takes eight prompts of 1024 tokens 82.3 us for 79.0;
                // four threads, 64 bytes, 79.7; through shared memory FP8 chunks and wide heads
                // take as long, the others longer.)
                const bool odd = lane & 1;
                const int own = live ? (tk * p.num_q_heads + br - tk * IH) * (D / 8) : -1, other = __shfl_xor_sync(0xffffffffu, own, 1);
                const int at0 = odd ? other : own, at1 = odd ? own : other;
                uint4 *o = reinterpret_cast<uint4 *>(p.out + (static_cast<long long>(token) * p.num_q_heads + head) * D);
#pragma unroll 1
                for (int c = 0; c < DPAD; c += 32) {
                    uint32_t x[32], y[16];
                    fetch(c, x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = dev::pack_bf16x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        uint32_t u[4], v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t r = __shfl_xor_sync(0xffffffffu, odd ? y[4 * k + i] : y[4 * k + 4 + i], 1);
                            u[i] = odd ? r : y[4 * k + i];
                            v[i] = odd ? y[4 * k + 4 + i] : r;
                        }
                        const int col = c + (k + odd) * 8;
                        if (at0 >= 0 && col < D) o[at0 + col / 8] = make_uint4(u[0], u[1], u[2], u[3]);
                        if (at1 >= 0 && col < D) o[at1 + col / 8] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            } else {
                // (four columns of 32 rows side by side: whole lines of memory)
                float *o = p.part_o + slot * p.slot_rows * DPAD + br * 4;
                const int step = partial_rows(part_rows);
#pragma unroll 1
                for (int c = 0; c < DPAD; c += 32) {
                    uint32_t x[32];
                    fetch(c, x);
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        if (br < part_rows) *reinterpret_cast<uint4 *>(o + (c + k) * step) = make_uint4(x[k], x[k + 1], x[k + 2], x[k + 3]);
                }
            }
        }
    }
    if (tid == 384 && !cut) p.cut[blockIdx.x] = {0, 0, 0, 0, 0};
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 1) tc::tmem_free_512(*tmem_s);
}

}  // namespace chunk
}  // namespace pd
