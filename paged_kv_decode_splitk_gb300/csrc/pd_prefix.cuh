// pd_prefix.cuh -- the shared-prefix pass of pd_decode_attn_prefix: attention
// partials of every sequence of a group over the group's one prefix.
//
// What it computes.  A group's query rows of one KV head (its sequences times
// the query heads that share the head) all meet the same P keys and values, so
// their scores are one matrix product, S = Q K^T, and their outputs another,
// O = exp2(S - m) V.  Per segment (a row block of up to 256 rows, a KV head, a
// run of key tiles) the pass writes each row's partial in base 2,
//   m  a reference (the largest score of the row's first tile, raised by whole
//      numbers when weights pass 2^15),
//   l = sum_t 2^(x_t - m),  o = sum_t 2^(x_t - m) V[t],   x_t = q.K[t] scale log2(e),
// which the merge folds with the other segments' and with the partials of the
// sequence's own tokens.
//
// GB300 mapping.
//   * CTAs work in teams of two.  A team's item is up to 512 rows of a KV head (256
//     at head dims above 128): each CTA has half of them, and both load every tile,
//     the second time from L2.  Rows that one CTA can take both have, and they take
//     the tiles in turn.  The two share nothing but the plan: every copy and
//     barrier is of one CTA (halves of a tile copied by each for both took as
//     long: 126.9 us whole, 127.3 in halves, 256 sequences behind 32768 tokens).
//   * Work is counted in units (item, a tile for both CTAs) in one line over all
//     groups; team c of C takes units [W c / C, W (c + 1) / C): every SM gets the
//     same number of tiles whatever the shapes, and a team's partials of item i go
//     to slots 2 (i + c) and 2 (i + c) + 1 (item and team both only grow along the
//     line, so slots are distinct, and there are at most items + C of them).  Where
//     teams are enough, every item has whole teams instead, its units shared evenly.
//   * One warp (two where none has to convert) loads: K and V tiles by TMA boxes of
//     64 columns x as many tokens as lie together in a cache block (16 to a whole
//     tile), gathered through the group's block table into a ring of tiles
//     (128-byte swizzle).  One warp issues tcgen05.mma: S (128 rows x kTile tokens) from
//     shared memory into TMEM, O += P V with P read from TMEM.  Two groups of
//     four warps do the softmax, a thread per row, S read from and P (BF16)
//     written back to TMEM over it.  The reference need not be the maximum, so
//     after the first tile none is taken: an exponential, half a multiply-add,
//     half an add and half a conversion per score is all there is.
//   * Two streams keep the tensor core and the softmax both busy: with more than
//     128 rows each stream has 128 of them and both use every tile; with fewer,
//     the streams take the tiles in turn (each its own O), folded in the end.  At
//     head dims above 128 one O fills TMEM: one stream, its S double-buffered.
//   * P is rounded to BF16 (half a step: 2^-9 to 2^-8 of each weight), the form
//     the tensor core multiplies with a BF16 V; l sums the unrounded weights in
//     FP32, S, O, m and l are FP32.  An FP8 cache is converted to f16 tiles
//     (exactly), and P is f16 there (2^-12 to 2^-11; a weight below 2^-14 is off by
//     up to 2^-25, and as a raised reference may lie up to 1 above the largest score,
//     the largest weight may be little more than a half: 2^-13 and 2^-24 of it).
//
// What bounds it, measured (8 KV heads, head dim 128, us of a step per 1024 more
// prefix tokens, from 8192 to 65536): 1024 rows 2.43 and 512 rows 1.22, the tensor core
// (2.24 and 1.12 at the library product's rate); 128 rows 0.60 and 256 rows 0.68, HBM
// (0.62); FP8 0.54 at 128 and 0.72 at 256 rows, the two warps that convert (HBM: 0.31).
// The rest is the chain of three launches, 10 us of the smallest step's 12.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <cfloat>

#include "pd.h"
#include "pd_device.cuh"
#include "pd_prefix_plan.h"
#include "pd_tcgen05.cuh"
#include "pd_tile.cuh"

namespace pd {
namespace prefix {

using namespace tile;

constexpr int kRegionBars = 32;

// Shared-memory plan (bytes from the 1024-aligned base).
template <int DPAD, bool KV8>
struct Plan {
    static constexpr bool kOne = DPAD > 128;  // one stream, S double-buffered
    static constexpr int kTile = tile_tokens(DPAD);
    static constexpr int kBlock = block_rows(DPAD);
    static constexpr int kStageBytes = kTile * DPAD * 2;
    static constexpr int kStages = KV8 ? 3 : (DPAD == 64 ? 6 : 4);
    static constexpr int kRawBytes = KV8 ? kTile * DPAD : 0;
    static constexpr int kRawStages = KV8 ? 3 : 0;
    static constexpr int kQBytes = (kOne ? 1 : 2) * kRowTile * DPAD * 2;
    static constexpr int q = 0;
    static constexpr int ring = q + kQBytes;
    static constexpr int raw = ring + kStages * kStageBytes;
    static constexpr int groups = raw + kRawStages * kRawBytes;
    static constexpr int bars = groups + kMaxGroups * static_cast<int>(sizeof(GroupPlan));
    static constexpr int misc = bars + kRegionBars * 8;
    static constexpr int row_scale = misc + 64;  // FP8: each query row's softmax scale
    static constexpr int stream_ml = row_scale + (KV8 ? 2 * 2 * kRowTile * 4 : 0);  // (m, l) of the streams' rows
    static constexpr int total = 1024 + stream_ml + (kOne ? 0 : 2 * kRowTile * 8);
    static constexpr int kThreads = 384;
};


// The most units of a team with whole teams for every item, by one warp (0: one line
// is better), and the teams then.
__device__ __forceinline__ int whole_teams(const GroupPlan *grp, int num_groups, int kv_heads, int of_item, long long units, int &c,
                                           int most, int items, float unit_us, float item_us, int lane) {
    WholeTry t;
    if (!try_whole(num_groups, units, c, most, items, t)) return 0;
    const int run = t.run(lane), teams = teams_in_all(grp, num_groups, kv_heads, of_item, run);
    const unsigned fits = __ballot_sync(0xffffffffu, teams <= t.limit);
    if (!fits) return 0;
    const int best = __ffs(fits) - 1, least = __shfl_sync(0xffffffffu, run, best), n = __shfl_sync(0xffffffffu, teams, best);
    if (!whole_pays(t, least, unit_us, item_us)) return 0;
    c = n;
    return least;
}

// The groups' units and items, by one warp: running sums over chunks of 32
// groups.  No units where group_starts is not non-decreasing within the batch or
// asks for more items than the workspace holds.
template <int DPAD, bool KV8>
__device__ __forceinline__ void plan_groups(const PrefixParams &p, GroupPlan *grp, long long *units_all, float *time_us, int *items_all, int lane,
                                            bool flag) {
    long long units = 0;
    float time = 0.f;  // of the units, this lane's share
    int items = 0;
    bool bad = false;
    for (int base = 0; base < p.num_groups; base += 32) {
        const int g = base + lane;
        GroupPlan r = {};
        long long mine = 0;
        int it = 0;
        if (g < p.num_groups) {
            const int a = p.group_starts ? p.group_starts[g] : 0;
            const int b = p.group_starts ? p.group_starts[g + 1] : p.num_seqs;
            int len = p.prefix_lens[g];
            const int most = p.max_prefix_blocks * static_cast<int>(p.block_size.d);
            if (len < 0 || len > most) {
                if (flag) dev::flag_status(p.status, PD_DEV_BAD_CONTEXT_LEN);
                len = len < 0 ? 0 : most;
            }
            bad |= a < 0 || b < a || b > p.num_seqs;
            r = plan_of<DPAD>(a, bad ? 0 : (b - a) * p.group, len);
            if (r.tiles > 0 && r.items > 0) {
                it = r.items * p.num_kv_heads;
                mine = r.head_units(item_rows(DPAD)) * p.num_kv_heads;
                time += mine * unit_time<DPAD, KV8>(min(r.rows, item_rows(DPAD)));
            }
        }
        long long su = mine;
        int si = it;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long ou = __shfl_up_sync(0xffffffffu, su, off);
            const int oi = __shfl_up_sync(0xffffffffu, si, off);
            if (lane >= off) {
                su += ou;
                si += oi;
            }
        }
        r.first_unit = units + su - mine;
        r.first_item = items + si - it;
        if (g < p.num_groups) grp[g] = r;
        units += __shfl_sync(0xffffffffu, su, 31);
        items += __shfl_sync(0xffffffffu, si, 31);
        if (items > p.max_items) break;
    }
    bad = __any_sync(0xffffffffu, bad) || items > p.max_items;
    if (bad && flag) dev::flag_status(p.status, PD_DEV_BAD_GROUPS);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) time += __shfl_xor_sync(0xffffffffu, time, off);
    *units_all = bad ? 0 : units;
    *time_us = time;
    *items_all = items;
}

// MULTI: more than one group.  (The rule that gives every item whole teams lies in
// the way of a call with one group, which has no use for it: 0.4 us of 15.)
template <int DPAD, bool KV8, bool MULTI>
__global__ void __launch_bounds__(Plan<DPAD, KV8>::kThreads, 1)
    prefix_kernel(const __grid_constant__ KvMaps<1> maps, const __grid_constant__ PrefixParams p) {
    using L = Plan<DPAD, KV8>;
    constexpr int BN = L::kTile;
    constexpr int BR = L::kBlock;
    constexpr int NST = L::kStages;
    constexpr bool ONE = L::kOne;
    constexpr int CHUNKS = DPAD / 8;  // 16-byte chunks of a 16-bit row
    constexpr uint32_t kDescS = tc::instr_desc(KV8 ? 0 : 1, kRowTile, BN, false);
    constexpr uint32_t kDescO = tc::instr_desc(KV8 ? 0 : 1, kRowTile, DPAD, true);
    const float kNegInf = -__int_as_float(0x7f800000);

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t base = dev::smem_addr(smem);
    GroupPlan *grp = reinterpret_cast<GroupPlan *>(smem + L::groups);
    // barriers: full[NST], empty[NST], raw_full[3], raw_empty[3], s_full[2],
    // p_full[2], o_done[2], q_full[2], tail, streams
    const uint32_t bars = base + L::bars;
    const uint32_t bar_full = bars, bar_empty = bar_full + 8 * NST, bar_rfull = bar_empty + 8 * NST,
                   bar_rempty = bar_rfull + 24, bar_s = bar_rempty + 24, bar_p = bar_s + 16, bar_o = bar_p + 16,
                   bar_q = bar_o + 16, bar_tail = bar_q + 16, bar_x = bar_tail + 8;
    const uint32_t bar_land = bar_rfull;  // (no raw stages: a last tile's landing, a barrier a stage)
    static_assert(2 * NST + 16 <= kRegionBars && (KV8 || NST <= 6), "barrier region");
    long long *units_s = reinterpret_cast<long long *>(smem + L::misc);
    unsigned *own_s = reinterpret_cast<unsigned *>(smem + L::misc + 8);  // sixteens of the sequences' own tokens
    int *items_s = reinterpret_cast<int *>(smem + L::misc + 12);
    float *time_s = reinterpret_cast<float *>(smem + L::misc + 16);
    volatile int *gave_up = reinterpret_cast<int *>(smem + L::misc + 20);
    uint32_t *tmem_s = reinterpret_cast<uint32_t *>(smem + L::misc + 24);
    long long *range_s = reinterpret_cast<long long *>(smem + L::misc + 32);
    int *share_s = reinterpret_cast<int *>(smem + L::misc + 48);  // teams, and the most units of one

    // (the warp's number from one lane, so that the compiler knows it to be the
    // same on all: the product warp's operands then live in uniform registers)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = blockIdx.x & 1, team = blockIdx.x >> 1;

    // ---- set-up that reads no global memory -----------------------------------
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            dev::mbar_init(bar_full + 8 * i, KV8 ? kConverters / 32 : 1);
            dev::mbar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; KV8 && i < 3; ++i) {
            dev::mbar_init(bar_rfull + 8 * i, 1);
            dev::mbar_init(bar_rempty + 8 * i, kConverters / 32);
        }
        for (int i = 0; !KV8 && i < NST; ++i) dev::mbar_init(bar_land + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            dev::mbar_init(bar_s + 8 * i, 1);
            dev::mbar_init(bar_p + 8 * i, 4);
            dev::mbar_init(bar_o + 8 * i, 1);
            dev::mbar_init(bar_q + 8 * i, 4);
        }
        dev::mbar_init(bar_tail, 1);
        dev::mbar_init(bar_x, 8);
        dev::fence_mbar_init();
        *gave_up = 0;
        *own_s = 0;
        dev::prefetch_tensormap(&maps.k[0]);
        dev::prefetch_tensormap(&maps.v[0]);
    }
    if (warp == 1) tc::tmem_alloc_512(dev::smem_addr(tmem_s));
    __syncthreads();      // (the sum of the own tokens starts at zero)
    dev::griddep_wait();  // q, the caches, tables and lengths are final
    if (warp == 0) {
        long long units;
        float time;
        int items;
        plan_groups<DPAD, KV8>(p, grp, &units, &time, &items, lane, blockIdx.x == 0);
        if (lane == 0) {
            *units_s = units;
            *time_s = time;
            *items_s = items;
        }
    } else if (warp > 1) {  // the sequences' own tokens (a sum of integers: the same in every CTA)
        long long own = 0;
#pragma unroll 4
        for (int s = tid - 64; s < p.num_seqs; s += L::kThreads - 64) own += min(max(p.context_lens[s], 0), p.max_own_tokens);
        // in sixteens, and no more of them than 32 bits hold from 320 threads
        const unsigned sum = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(min(own >> 4, 1ll << 23)));
        if (lane == 0 && sum) atomicAdd(own_s, sum);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    // Everything before this grid is done: the own-token pass, which needs nothing
    // of this one, may start wherever there is room.
    dev::griddep_launch_dependents();
    constexpr uint32_t tmem = 0;  // all 512 columns: the allocation starts at the first
    // (the own pass draws 5.4 MB of a BF16 cache a us from all SMs, 2.8 of FP8 codes)
    const long long W = *units_s;
    const float own_us = fmaxf(0.5f * static_cast<float>(*own_s) * (p.num_kv_heads * p.head_dim * (KV8 ? 32.f / 2.8e6f : 64.f / 5.4e6f)) * gridDim.x,
                               0.35f * static_cast<float>(p.num_seqs) * p.num_kv_heads);
    int C = 0;
    long long u = 0, u1 = 0;
    if constexpr (!MULTI) {
        if (W > 0) C = share_units(W, *items_s, grp[0].last_units(item_rows(DPAD)) == quotient(W, *items_s), *time_s, own_us, gridDim.x / 2);
        if (blockIdx.x == 0 && tid == 0) {  // the merge finds each row's partials from this
            *p.plan_total = {W, C, 0};
            p.plan_groups[0] = grp[0];
        }
        if (team < C) line_range(W, C, team, u, u1);
    } else {
        if (warp == 0) {  // (by one warp: twelve would share the issue slots)
            int run = 0;
            if (W > 0) {
                C = share_units(W, *items_s, false, *time_s, own_us, gridDim.x / 2);
                run = whole_teams(grp, p.num_groups, p.num_kv_heads, item_rows(DPAD), W, C, gridDim.x / 2, *items_s,
                                  __fdividef(*time_s, static_cast<float>(W)), KV8 ? 6.f : 3.f, lane);
                if (team < C && run > 0)
                    whole_range(grp, p.num_kv_heads, item_rows(DPAD), run, team, u, u1);
                else if (team < C)
                    line_range(W, C, team, u, u1);
            }
            if (lane == 0) {
                range_s[0] = u;
                range_s[1] = u1;
                share_s[0] = C;
                share_s[1] = run;
            }
        }
        __syncthreads();
        u = range_s[0];
        u1 = range_s[1];
        C = share_s[0];
        if (blockIdx.x == 0 && warp == 1) {
            const int run = share_s[1];
            if (lane == 0) *p.plan_total = {W, C, run > 0};
            for (int g = lane; g < p.num_groups; g += 32) {
                GroupPlan r = grp[g];
                plan_whole(grp, g, p.num_kv_heads, item_rows(DPAD), run, r);
                p.plan_groups[g] = r;
            }
            __syncwarp();
        }
    }
    const int bs = static_cast<int>(p.block_size.d);
    const int D = p.head_dim;
    Segment sg;
    // Registers: a softmax thread holds a whole tile row.  384 threads were
    // launched with 168 each: 128 x 88 + 256 x 208 is what all of them have.
    static_assert(L::kThreads == 384 && 88 + 2 * 208 <= 3 * 168, "the shares add up to the launch's registers");

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");

    if (warp == 0 || (!KV8 && warp == 2)) {
        // ---- loads: K and V tiles in the order the products take them ------------
        // (a warp for each where two are free)
        constexpr int COLS = KV8 ? (DPAD < 128 ? DPAD : 128) : kBoxCols;  // columns of a box
        const int CT = p.box_tokens;                         // tokens of a box
        const int NCH = BN / CT, NBOX = NCH * (DPAD / COLS);
        constexpr int DEPTH = KV8 ? L::kRawStages : NST;
        constexpr int BYTES = KV8 ? L::kRawBytes : L::kStageBytes;
        const uint32_t full = KV8 ? bar_rfull : bar_full, empty = KV8 ? bar_rempty : bar_empty;
        const uint32_t stage0 = base + (KV8 ? L::raw : L::ring);
        const uint64_t policy = dev::l2_evict_first_policy();
        const int chunk = lane % NCH, col = lane / NCH;
        int st = 0;
        uint32_t ph = 0;  // phase of the stage about to be filled
        uint32_t land_ph = 0;  // of the landing barriers, a bit each
        bool ok = true;
        long long issued = 0;
        while (ok && next_segment<BR>(grp, p.num_groups, u, u1, team, rank, sg)) {
            const int32_t *ids = p.prefix_table + static_cast<long long>(sg.group) * p.max_prefix_blocks;
            const int ahead = ONE || !sg.two ? 2 : 1;
            const bool mine = lane < NBOX;  // a box a lane
            // Block ids, 32 boxes' rows (chunks of CT tokens) at a time: lane l of `now`
            // has chunk 32 w + l of the run, `then` the 32 after them, asked for a
            // window ahead.  Past the prefix, and for a bad id (-1), it is one
            // outside the cache, which reads zeros.
            const int lg = 31 - __clz(NCH);
            auto ids_of = [&](int w) -> int {
                const int c = 32 * w + lane, j = c >> lg;
                const int tok = (sg.tile0 + j * sg.stride) * BN + (c & (NCH - 1)) * CT;
                if (j >= sg.n || tok >= sg.plen) return p.num_blocks;
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
                const int first = (sg.tile0 + j * sg.stride) * BN, tok = first + chunk * CT;
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
                const int nv = sg.plen - first;  // live tokens of the tile
                // A tile's box of live and dead tokens holds whatever the cache's
                // slots past the prefix hold; a dead V row must not reach the
                // product (0 x NaN), so those rows are zeroed before it is handed on.  It
                // lands at a barrier of its stage.
                const bool tail = !KV8 && is_v && nv < BN && (nv & (CT - 1));
                const uint32_t bar = (tail ? bar_land : full) + 8 * st;
                if (lane == 0) dev::mbar_arrive_expect_tx(bar, BYTES);
                __syncwarp();
                if (mine) {
                    const int sub = tok - fast_div(tok, p.block_size) * bs;
                    const uint32_t to = dst + col * (BN * (KV8 ? COLS : 128)) + chunk * (CT * (KV8 ? COLS : 128));
                    const CUtensorMap *map = is_v ? &maps.v[0] : &maps.k[0];
                    const int c1 = p.tok_dim == 1 ? sub : sg.kvh, c2 = p.tok_dim == 1 ? sg.kvh : sub;
                    dev::tma_load_4d(to, map, bar, col * COLS, c1, c2, id, policy);
                }
                if (tail) {
                    const uint32_t lph = (land_ph >> st) & 1;
                    land_ph ^= 1u << st;
                    if (!wait_bar(bar, lph, gave_up)) {
                        if (lane == 0) dev::mbar_wait_bounded(bar, lph, 100000000ull);  // (its copies land before the CTA ends)
                        return false;
                    }
                    uint8_t *tile = smem + L::ring + st * BYTES;
                    const int end = (nv + CT - 1) & ~(CT - 1);
                    for (int b = 0; b < DPAD / 64; ++b)
                        for (int i = nv * 8 + lane; i < end * 8; i += 32)
                            *reinterpret_cast<uint4 *>(tile + b * (BN * 128) + i * 16) = make_uint4(0, 0, 0, 0);
                    tc::fence_async_shared();
                    __syncwarp();
                    if (lane == 0) arrive(full + 8 * st);
                }
                return next_stage();
            };
            for (int i = 0; ok && i < sg.n + ahead - 1; ++i) {
                if (i < sg.n) ok = load(false, i);
                const int v = i - ahead + 1;
                if (ok && v >= 0) ok = load(true, v);
            }
        }
        // every release of a stage has arrived before this CTA ends
        for (long long i = issued < DEPTH ? 0 : issued - DEPTH; ok && i < issued; ++i)
            ok = wait_bar(empty + 8 * static_cast<int>(i % DEPTH), static_cast<uint32_t>((i / DEPTH) & 1), gave_up);
        if (!ok && lane == 0) {
            // a wait ran out: let the copies in flight land before the CTA ends
            dev::flag_status(p.status, PD_DEV_WAIT_TIMEOUT);
            const long long last = issued < DEPTH ? issued : DEPTH;
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
            uint32_t ph = 0, pph = 0, qph = 0;  // phases: of the ring; a bit for each stream
            bool ok = true;
            const uint32_t qa = base + L::q, ra = base + L::ring;
            const uint64_t q_desc = tc::smem_desc(qa, 16), k_desc = tc::smem_desc(ra, 16), v_desc = tc::smem_desc(ra, BN * 128);
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
                const uint64_t qd = q_desc + qt * (kRowTile * DPAD * 2 / 16), kd = k_desc + stage * (L::kStageBytes / 16);
                tc::fence_after();
#pragma unroll
                for (int k = 0; k < DPAD / 16; ++k)
                    tc::mma_ss(tmem + buf * 128, qd + ((k / 4) * (kRowTile * 128) + (k % 4) * 32) / 16,
                               kd + ((k / 4) * (BN * 128) + (k % 4) * 32) / 16, kDescS, k > 0);
                tc::commit(bar_s + 8 * buf);
            };
            auto values = [&](int buf, int o, int stage, bool accumulate, bool done) {
                const uint64_t vd = v_desc + stage * (L::kStageBytes / 16);
                tc::fence_after();
#pragma unroll
                for (int k = 0; k < BN / 16; ++k)
                    tc::mma_ts(tmem + 256 + o * DPAD, tmem + buf * 128 + k * 8, vd + k * (2048 / 16), kDescO, accumulate || k > 0);
                if (done) tc::commit(bar_o + 8 * o);
            };
            auto release = [&](int stage) { tc::commit(bar_empty + 8 * stage); };
            auto weights = [&](int buf) {
                const bool got = wait_one(bar_p + 8 * buf, (pph >> buf) & 1, gave_up);
                pph ^= 1u << buf;
                return got;
            };
            auto queries = [&](int t) {
                const bool got = wait_one(bar_q + 8 * t, (qph >> t) & 1, gave_up);
                qph ^= 1u << t;
                return got;
            };
            while (ok && next_segment<BR>(grp, p.num_groups, u, u1, team, rank, sg)) {
                const int n = sg.n;
                if (n == 0) continue;
                int ks = 0, vs = 0;
                if (!(ok = queries(0))) break;
                if (!(ok = take(ks))) break;
                if (!ONE && sg.two) {
                    scores(0, 0, ks);
                    if (!(ok = queries(1))) break;
                    scores(1, 1, ks);
                    release(ks);
                    if (!(ok = take(vs))) break;
                    for (int j = 0; ok && j < n; ++j) {
                        const bool more = j + 1 < n;
                        const int v = vs;
                        if (more && !(ok = take(ks))) break;
                        if (!(ok = weights(0))) break;
                        values(0, 0, v, j > 0, !more);
                        if (more) scores(0, 0, ks);
                        if (!(ok = weights(1))) break;
                        values(1, 1, v, j > 0, !more);
                        release(v);  // (before the scores: a commit waits for all that came before)
                        if (more) {
                            scores(1, 1, ks);
                            release(ks);
                            ok = take(vs);
                        }
                    }
                } else {
                    // scores of tile j, whose keys are the next of the ring
                    auto next_scores = [&](int j) {
                        scores(j & 1, 0, ks);
                        release(ks);
                    };
                    next_scores(0);
                    if (n > 1) {
                        if (!(ok = take(ks))) break;
                        next_scores(1);
                    }
                    for (int j = 0; ok && j < n; ++j) {
                        if (!(ok = take(vs))) break;
                        const bool next = j + 2 < n;
                        if (next && !(ok = take(ks))) break;
                        const int t = j & 1;
                        if (!(ok = weights(t))) break;
                        values(t, ONE ? 0 : t, vs, j > (ONE ? 0 : 1), ONE || j + 2 >= n);
                        release(vs);
                        if (next) next_scores(j + 2);
                    }
                }
            }
            if (!ok) {
                // let the products in flight end before TMEM is freed
                tc::commit(bar_tail);
                dev::mbar_wait_bounded(bar_tail, 0, 100000000ull);
            }
        }
        __syncwarp();
    } else if (KV8) {
        // ---- FP8: each landed tile of codes into an f16 tile of the ring -------------
        // (k_scale is in the softmax scale, v_scale in the merge).  V rows past the
        // prefix are zeroed on the way.
        const Widen<DPAD, BN> widen(warp - 2, lane);
        int rs = 0, st = 0;
        uint32_t rph = 0, ph = 0;
        bool ok = true;
        long long handed = 0;
        auto convert = [&](bool is_v, int nv) {
            if (!wait_bar(bar_rfull + 8 * rs, rph, gave_up) || !wait_bar(bar_empty + 8 * st, ph ^ 1, gave_up)) return false;
            const uint8_t *src = smem + L::raw + rs * L::kRawBytes;
            uint8_t *dst = smem + L::ring + st * L::kStageBytes;
            widen(src, dst, is_v && nv < BN, 0, nv);
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
        while (ok && next_segment<BR>(grp, p.num_groups, u, u1, team, rank, sg)) {
            const int ahead = ONE || !sg.two ? 2 : 1;
            for (int i = 0; ok && i < sg.n + ahead - 1; ++i) {
                if (i < sg.n) ok = convert(false, BN);
                const int v = i - ahead + 1;
                if (ok && v >= 0) ok = convert(true, sg.plen - (sg.tile0 + v * sg.stride) * BN);
            }
        }
        // every release of a stage has arrived before this CTA ends
        for (long long i = handed < NST ? 0 : handed - NST; ok && i < handed; ++i)
            ok = wait_bar(bar_empty + 8 * static_cast<int>(i % NST), static_cast<uint32_t>((i / NST) & 1), gave_up);
    }
    } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    if (warp < (ONE ? 8 : 12)) {
        // ---- softmax: a thread per row -----------------------------------------------
        const int t = (warp - 4) >> 2;            // the stream
        const int r = (warp & 3) * 32 + lane;     // the row of its tile
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t to = tmem + lanes + 256 + t * DPAD;
        uint32_t sph = 0, oph = 0, xph = 0;  // phases, a bit for each buffer or stream
        bool ok = true;
        // FP8: the rows' scales, in turn in two places: the other stream may still
        // have to read the last segment's when this one's are written (it has by
        // the time a third segment begins: its weights of the first went before)
        float *row_scale = reinterpret_cast<float *>(smem + L::row_scale);
        int turn = 0;
        while (ok && next_segment<BR>(grp, p.num_groups, u, u1, team, rank, sg)) {
            const bool two = sg.two;
            float scale = p.scale_log2;
            if constexpr (KV8) {
                row_scale = reinterpret_cast<float *>(smem + L::row_scale) + turn * 2 * kRowTile;
                turn ^= 1;
            }
            // -- this stream's query rows into shared memory (128-byte swizzle); with
            // at most 128 rows the streams share stream 0's.  (The last segment's
            // partials have to have left from there.)
            if (lane == 0) tc::bulk_wait_read<0>();
            __syncwarp();
            if ((two || t == 0) && sg.n > 0) {
                uint8_t *qt = smem + L::q + t * (kRowTile * DPAD * 2);
                // 32 rows x CHUNKS chunks over 32 lanes, sixteen loads in flight at once
                constexpr int BATCH = CHUNKS < 16 ? CHUNKS : 16;
#pragma unroll 1
                for (int i0 = 0; i0 < CHUNKS; i0 += BATCH) {
                    uint4 v[BATCH];
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int e = (i0 + i) * 32 + lane;
                        const int gr = t * kRowTile + (warp & 3) * 32 + e / CHUNKS, c = e % CHUNKS;  // row of the block, chunk
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (gr < sg.rows && c * 8 < D) {
                            const int x = sg.row0 + gr;
                            const int sq = fast_div(x, p.fd_group);
                            v[i] = __ldg(reinterpret_cast<const uint4 *>(
                                p.q + (static_cast<long long>(sg.seq0 + sq) * p.num_q_heads + sg.kvh * p.group + (x - sq * p.group)) * D +
                                c * 8));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        const int e = (i0 + i) * 32 + lane;
                        const int row = (warp & 3) * 32 + e / CHUNKS, c = e % CHUNKS;
                        if (p.negative) {
                            v[i].x ^= 0x80008000u, v[i].y ^= 0x80008000u, v[i].z ^= 0x80008000u, v[i].w ^= 0x80008000u;
                        }
                        if constexpr (KV8) {
                            // f16 rows under a power of two that brings the row's largest
                            // |q| into [2^14, 2^15), exactly but for values 2^-28 below it;
                            // its inverse joins the row's softmax scale
                            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                            float big = 0.f;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                big = fmaxf(big, fmaxf(fabsf(dev::bf16_lo_f32(w[k])), fabsf(dev::bf16_hi_f32(w[k]))));
#pragma unroll
                            for (int off = 1; off < CHUNKS; off <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
                            const int ex = (__float_as_int(big) >> 23) & 0xff;  // big < 2^(ex - 126)
                            const int up = min(max(141 - ex, -126), 127);       // times 2^up: below 2^15
                            const float f = __int_as_float((127 + up) << 23);
                            const float down = up < 127 ? __int_as_float((127 - up) << 23) : 5.877471754111438e-39f;  // 2^-up
                            if (c == 0) row_scale[t * kRowTile + row] = fmaxf(p.scale_log2 * down, FLT_MIN);
                            v[i].x = dev::pack_f16x2(dev::bf16_lo_f32(w[0]) * f, dev::bf16_hi_f32(w[0]) * f);
                            v[i].y = dev::pack_f16x2(dev::bf16_lo_f32(w[1]) * f, dev::bf16_hi_f32(w[1]) * f);
                            v[i].z = dev::pack_f16x2(dev::bf16_lo_f32(w[2]) * f, dev::bf16_hi_f32(w[2]) * f);
                            v[i].w = dev::pack_f16x2(dev::bf16_lo_f32(w[3]) * f, dev::bf16_hi_f32(w[3]) * f);
                        }
                        *reinterpret_cast<uint4 *>(qt + (c / 8) * (kRowTile * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v[i];
                    }
                }
                tc::fence_async_shared();
                arrive_warp(bar_q + 8 * t, lane);
            }
            float m = kNegInf, l = 0.f;
            bool first = true;
            const int step = ONE || two ? 1 : 2;
            for (int j = step == 2 ? t : 0; j < sg.n; j += step) {
                const int buf = ONE ? (j & 1) : t;
                const uint32_t ts = tmem + lanes + buf * 128;
                if (!(ok = wait_bar(bar_s + 8 * buf, (sph >> buf) & 1, gave_up))) break;
                sph ^= 1u << buf;
                tc::fence_after();
                if (KV8 && first) scale = row_scale[(two ? t * kRowTile : 0) + r];
                const int nv = sg.plen - (sg.tile0 + j * sg.stride) * BN;
                // -- A row's reference m is the largest score of its first tile; after
                // that no maximum is taken: weights may be as large as kLift, and
                // only when a row's weights of a tile sum to more does its warp look
                // at the scores again and raise m (by a whole number, so that l and O
                // are scaled exactly).  FP32 and BF16 hold such weights as exactly as
                // weights below 1; kLift is what f16 holds.
                uint32_t x[BN], pk[BN / 2];
                float sum;
                bool fresh = m == kNegInf, over = false;  // rows that take, or raise, their reference now
                bool waited = !ONE || first;  // the last product onto O is known to be done
                for (bool again = false;; again = true) {
                    tc::ld_columns<BN>(ts, x);
                    if (nv < BN) mask_columns<BN>(x, nv);
                    if (__any_sync(0xffffffffu, fresh || over)) {
                        const float mx = largest_of<BN>(x) * scale;
                        if (fresh) m = mx;
                        if (again) raise_reference<DPAD>(to, mx, over, m, l);
                    }
                    sum = weigh<BN, KV8>(x, scale, m, pk);
                    over = !(sum <= kLift);
                    fresh = false;
                    if (again || !__any_sync(0xffffffffu, over)) break;
                    if (!waited) {
                        ok = wait_bar(bar_o, oph & 1, gave_up);
                        oph ^= 1;
                        waited = true;
                        tc::fence_after();
                    }
                }
                first = false;
                l += sum;
                tc::st_columns<BN / 2>(ts, pk);  // over S, which has been read
                if (ONE && !waited) {  // (each phase of the barrier is waited for, in order)
                    ok = wait_bar(bar_o, oph & 1, gave_up) && ok;
                    oph ^= 1;
                }
                if (!ok) break;
                tc::wait_st();
                tc::fence_before();
                arrive_warp(bar_p + 8 * buf, lane);
            }
            if (!ok) break;
            // -- the partial of this row: (m, l) [slot][BR], o [slot][DPAD / 32][BR][32].
            // 32 columns at a time go through the shared memory of this warp's own
            // query rows (their products are done) and out as one copy of 4 KB, the
            // 16-byte chunks of a row by their place xor the row's, here (no bank is
            // hit twice) and in the workspace.
            const long long at = static_cast<long long>(sg.slot) * BR;
            constexpr int kBufs = DPAD / 64;
            uint8_t *stage = smem + L::q + t * (kRowTile * DPAD * 2) + (warp & 3) * 4096;
            const int warp_row = (ONE || two ? t * kRowTile : 0) + (warp & 3) * 32;  // of the block
            int copies = 0;
            auto store = [&](int c, const uint32_t (&x)[32]) {
                uint8_t *buf = stage + copies % kBufs * (kRowTile * 128);
                if (copies >= kBufs) {
                    if (lane == 0) tc::bulk_wait_read<kBufs - 1>();
                    __syncwarp();
                }
                ++copies;
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<uint4 *>(buf + lane * 128 + (((i / 4) ^ (lane & 7)) << 4)) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                tc::fence_async_shared();
                __syncwarp();
                if (lane == 0 && warp_row < sg.rows)
                    tc::bulk_store(p.part_o + ((static_cast<long long>(sg.slot) * (DPAD / 32) + c / 32) * BR + warp_row) * 32,
                                   dev::smem_addr(buf), 4096);
            };
            if (ONE || two) {
                const int row = t * kRowTile + r;
                const bool in = row < sg.rows;
                if (in) *reinterpret_cast<float2 *>(p.part_ml + (at + row) * 2) = make_float2(m, l);
                if (sg.n > 0) {
                    if (!(ok = wait_bar(bar_o + 8 * t, (oph >> t) & 1, gave_up))) break;
                    oph ^= 3;
                    tc::fence_after();
#pragma unroll 1
                    for (int c = 0; c < DPAD; c += 32) {
                        uint32_t x[32];
                        tc::ld_32x32(to + c, x);
                        tc::wait_ld(x);
                        store(c, x);
                    }
                    tc::fence_before();
                }
            } else {
                // the streams' two partials of the row, folded: each stream then writes
                // half of the columns
                float2 *ml = reinterpret_cast<float2 *>(smem + L::stream_ml);
                ml[t * kRowTile + r] = make_float2(m, l);
                arrive_warp(bar_x, lane);
                if (!(ok = wait_bar(bar_x, xph, gave_up))) break;
                xph ^= 1;
                for (int k = 0; k < 2 && ok; ++k) {
                    if (k < sg.n) {
                        ok = wait_bar(bar_o + 8 * k, (oph >> k) & 1, gave_up);
                        oph ^= 1u << k;
                    }
                }
                if (!ok) break;
                tc::fence_after();
                const float2 a = ml[r], b = ml[kRowTile + r];
                const float M = fmaxf(a.y == 0.f ? kNegInf : a.x, b.y == 0.f ? kNegInf : b.x);
                const float fa = a.y == 0.f ? 0.f : dev::exp2_approx(a.x - M), fb = b.y == 0.f ? 0.f : dev::exp2_approx(b.x - M);
                const bool in = r < sg.rows;
                if (in && t == 0)
                    *reinterpret_cast<float2 *>(p.part_ml + (at + r) * 2) =
                        make_float2(M, (a.y == 0.f ? 0.f : a.y * fa) + (b.y == 0.f ? 0.f : b.y * fb));
                if (sg.n > 0) {
#pragma unroll 1
                    for (int c = t * (DPAD / 2); c < (t + 1) * (DPAD / 2); c += 32) {
                        uint32_t x[32], y[32];
                        tc::ld_32x32(tmem + lanes + 256 + c, x);
                        tc::wait_ld(x);
                        if (sg.n > 1) {
                            tc::ld_32x32(tmem + lanes + 256 + DPAD + c, y);
                            tc::wait_ld(y);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float xa = fa == 0.f ? 0.f : __uint_as_float(x[i]) * fa;
                            x[i] = __float_as_uint(sg.n > 1 && fb != 0.f ? fmaf(__uint_as_float(y[i]), fb, xa) : xa);
                        }
                        store(c, x);
                    }
                    tc::fence_before();
                }
                // both streams have read both O before either lets one be overwritten
                arrive_warp(bar_x, lane);
                if (!(ok = wait_bar(bar_x, xph, gave_up))) break;
                xph ^= 1;
            }
        }
    }
    }
    if (warp >= 4 && lane == 0) tc::bulk_wait_all();
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 1) tc::tmem_free_512(*tmem_s);
}

}  // namespace prefix
}  // namespace pd
