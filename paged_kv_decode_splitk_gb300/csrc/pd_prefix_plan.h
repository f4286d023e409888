// pd_prefix_plan.h -- how the shared-prefix pass divides its work, and where the
// merge finds it: plain arithmetic on whole numbers, which the kernels run on the
// device and pd_debug_prefix_walk on the host.
#pragma once

#include <math.h>

#include "pd_prefix.h"

namespace pd {
namespace prefix {

constexpr int kRowTile = 128;   // rows of one MMA

#ifndef __CUDA_ARCH__
inline int min(int a, int b) { return a < b ? a : b; }
inline int max(int a, int b) { return a > b ? a : b; }
inline long long min(long long a, long long b) { return a < b ? a : b; }
inline long long max(long long a, long long b) { return a > b ? a : b; }
#endif

// a / b, near enough where its ceiling or floor is a choice.
__host__ __device__ inline float quick_quotient(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fdividef(a, b);
#else
    return a / b;
#endif
}

// The block of rows and the run of tiles a CTA works on at a time.
struct Segment {
    int kvh, plen, slot;
    int tile0, stride;  // tile j of the run is tile0 + j stride
    int n;      // tiles of the run (0: the last place of an item taken in turn has but one, the other CTA's)
    int row0;   // first row of this CTA within the group
    int rows;   // rows of this CTA
    int seq0;   // the group's first sequence
    int group;
    bool two;   // more than kRowTile rows: both streams use every tile
    bool pair;  // both CTAs use the same tiles, half of the rows each
};

// a / b, in 32 bits where both fit (a fifth of the instructions).
__host__ __device__ inline long long quotient(long long a, long long b) {
    if ((a | b) >> 32 == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return a / b;
}

template <int BR>
__host__ __device__ inline bool next_segment(const GroupPlan *grp, int num_groups, long long &u, long long u1,
                                             int team, int rank, Segment &s) {
    if (u >= u1) return false;
    int lo = 0, n = num_groups;  // the last group that begins at or before unit u
    while (n > 1) {
        const int half = n >> 1;
        if (grp[lo + half].first_unit <= u) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    const GroupPlan g = grp[lo];
    const long long per_head = g.head_units(2 * BR);
    const long long local = u - g.first_unit;
    s.kvh = static_cast<int>(quotient(local, per_head));
    const long long rem = local - s.kvh * per_head;
    const int item = static_cast<int>(quotient(rem, g.tiles));  // (the last item may have fewer units, never more)
    const int at = static_cast<int>(rem - static_cast<long long>(item) * g.tiles);  // place within the item
    const int rows = min(2 * BR, g.rows - item * 2 * BR);
    s.pair = is_pair(rows, 2 * BR);
    const int places = s.pair ? g.tiles : (g.tiles + 1) >> 1;
    const long long left = u1 - u;
    const int taken = left < places - at ? static_cast<int>(left) : places - at;  // of them
    s.stride = s.pair ? 1 : 2;
    s.tile0 = s.pair ? at : 2 * at + rank;
    s.n = s.tile0 + (taken - 1) * s.stride < g.tiles ? taken : taken - 1;
    const int half = (rows + 1) >> 1;
    s.row0 = item * 2 * BR + (s.pair && rank ? half : 0);
    s.rows = !s.pair ? rows : rank ? rows - half : half;
    s.plen = g.tokens;
    s.seq0 = g.first_seq;
    s.group = lo;
    s.slot = 2 * (g.first_item + s.kvh * g.items + item + team) + rank;
    s.two = s.rows > kRowTile;
    if (taken < 1) return false;  // (never; the walk over the units ends all the same)
    u += taken;
    return true;
}

// How many teams share the prefixes' units.  The own-token pass runs on the SMs
// the prefix pass leaves, and the step is shortest where both end together: with
// n SMs, C teams, units (and the start and end of items) of B us in all and U the
// own pass's time on one SM,
//   B / C = U / (n - 2 C).
// Of U's loads half is taken, since teams too few cost more than teams too many,
// but at least what its units cost when they have next to no tokens: where all SMs
// went to the prefixes the own pass began 4 us before the end, at theirs.  Measured
// (us, all 76 teams -> about as many as this gives): 64 sequences behind 8192
// tokens 47.3 -> 41.2 (24 teams; 16: 52.1), 256 behind 32768 136 -> 124 (60), six
// groups of wide heads 32.3 -> 30.7 (48), 32 behind 16385 over FP8 51.3 -> 46.9
// (48).  A team has four units or more beyond the first eight teams, or an item: each is a
// partial more of all its rows to write and fold (256 units without own tokens:
// 19.7 us on 76 teams, 17.0 on 32).  Where the items have as many units each
// (`even`) and there are teams enough, a count that gives every item whole teams
// spares those that would end one item and begin the next (256 units of 8 items
// over FP8: 21.5 us on 64 teams, 26.7 on 60), if it is near or costs less than that.
__host__ __device__ inline int share_units(long long units, int items, bool even, float units_us, float own_us, int most) {
    constexpr float item_us = 3.f;  // to begin and end an item
    const float all_us = units_us + item_us * items;
    const long long enough = max((units + 3) / 4, min(units, max(8ll, static_cast<long long>(items))));
    int c = static_cast<int>(ceilf(quick_quotient(2.f * most * all_us, own_us + 2.f * all_us)));
    c = static_cast<int>(max(1ll, min(enough, static_cast<long long>(min(c, most)))));
    if (even && c >= items) {
        const int down = c - static_cast<int>(static_cast<unsigned>(c) % static_cast<unsigned>(items)), up = down + items;
        if (down != c && up <= most && 16 * up <= 17 * c)
            c = up;
        else if (units_us * (c - down) <= item_us * static_cast<float>(c) * down)
            c = down;
    }
    return c;
}

// Teams of an item with at most about `run` units each (no more than it has units).
__host__ __device__ inline int teams_of(int units, int run) {
    return max(1, static_cast<int>(ceilf(fmaf(static_cast<float>(units), quick_quotient(1.f, static_cast<float>(run)), -1e-3f))));
}
__host__ __device__ inline int head_teams(const GroupPlan &g, int of_item, int run) {
    return g.tiles && g.items ? (g.items - 1) * teams_of(g.tiles, run) + teams_of(g.last_units(of_item), run) : 0;
}
// a / b of whole numbers from 0 and 1 to 255
__host__ __device__ inline int small_quotient(int a, int b) {
    return static_cast<int>((static_cast<float>(a) + 0.5f) * quick_quotient(1.f, static_cast<float>(b)));
}

// Whole teams for every item, where there are teams enough: a team that ends one
// item and begins the next spends 3 us on that (6 over FP8, where the ring of
// converted tiles fills anew), often more than its share of units is worth (three
// groups of wide FP8 heads 30.3 us on 52 teams in one line, 22 on 44 or 56 that
// happen to end with the items; 256 units of 8 items 18.3 on 48 teams, 23 on 44).
// Tried, a lane each, are 32 numbers of units that a team has at most, from the
// line's share on; the least with no more than about c teams is taken if it costs no
// more than that.  Where teams have a unit each, the line has whole teams already.
struct WholeTry {
    int limit;   // teams at most
    float even;  // units of a team in one line
    int share;
    __host__ __device__ int run(int lane) const { return share + lane * ((share + 15) / 16); }
};
__host__ __device__ inline bool try_whole(int num_groups, long long units, int c, int most, int items, WholeTry &t) {
    t.limit = min(most, c + c / 16);
    t.even = quick_quotient(static_cast<float>(units), static_cast<float>(c));
    t.share = static_cast<int>(ceilf(t.even));
    return units > c && items <= t.limit && num_groups <= 32;
}
__host__ __device__ inline int teams_in_all(const GroupPlan *grp, int num_groups, int kv_heads, int of_item, int run) {
    int teams = 0;
    for (int g = 0; g < num_groups; ++g) teams += kv_heads * head_teams(grp[g], of_item, run);
    return teams;
}
__host__ __device__ inline bool whole_pays(const WholeTry &t, int run, float unit_us, float item_us) {
    return !((static_cast<float>(run) - t.even) * unit_us > item_us);
}

// The units of a team where items have whole teams.
__host__ __device__ inline void whole_range(const GroupPlan *grp, int kv_heads, int of_item, int run, int team, long long &u,
                                            long long &u1) {
    int g = 0, n;
    while (team >= (n = kv_heads * head_teams(grp[g], of_item, run))) {
        team -= n;
        ++g;
    }
    const GroupPlan r = grp[g];
    const int last = r.last_units(of_item), of_last = teams_of(last, run);
    const int of_one = r.items > 1 ? teams_of(r.tiles, run) : of_last, head = (r.items - 1) * of_one + of_last;
    const int kvh = small_quotient(team, head), at = team - kvh * head;
    const int item = min(small_quotient(at, of_one), r.items - 1);
    const bool ends = item == r.items - 1;
    // even shares, the first ones a unit longer
    const int part = at - item * of_one, places = ends ? last : r.tiles, teams = ends ? of_last : of_one;
    const int least = places / teams, longer = places - least * teams;
    u = r.first_unit + kvh * r.head_units(of_item) + static_cast<long long>(item) * r.tiles + least * part + min(part, longer);
    u1 = u + least + (part < longer);
}

// The time of a unit on a team, measured (us): the conversion bounds an FP8 tile;
// two full row tiles of products a pair's; one, and memory, the others'.
template <int DPAD, bool KV8>
__host__ __device__ inline float unit_time(int rows) {
    const bool pair = is_pair(rows, item_rows(DPAD));
    const float us = KV8 || (!pair && rows > kRowTile) ? 1.6f : pair ? (DPAD == 256 ? 0.9f : 1.4f) : DPAD == 256 ? 1.f : 1.3f;
    return DPAD == 64 ? (KV8 ? 0.8f : 0.6f) * us : us;
}

// A group's rows and tiles; its units and items where it has any.
template <int DPAD>
__host__ __device__ inline GroupPlan plan_of(int first_seq, int rows, int tokens) {
    GroupPlan r = {};
    r.first_seq = first_seq;
    r.rows = rows;
    r.items = (rows + item_rows(DPAD) - 1) / item_rows(DPAD);
    r.tokens = tokens;
    r.tiles = (tokens + tile_tokens(DPAD) - 1) / tile_tokens(DPAD);
    return r;
}

// The units of a team in one line of W.
__host__ __device__ inline void line_range(long long W, int C, int team, long long &u, long long &u1) {
    u = quotient(W * team, C);
    u1 = quotient(W * (team + 1), C);
}

// The teams of group g, where items have whole teams of at most `run` units.
__host__ __device__ inline void plan_whole(const GroupPlan *grp, int g, int kv_heads, int of_item, int run, GroupPlan &r) {
    r.first_team = r.teams = r.last_teams = 0;
    if (run > 0) {
        for (int k = 0; k < g; ++k) r.first_team += kv_heads * head_teams(grp[k], of_item, run);
        r.teams = teams_of(r.tiles, run);
        r.last_teams = teams_of(r.last_units(of_item), run);
    }
}

// ---- where the merge finds a row's partials -----------------------------------------
// The team whose range [W c / C, W (c + 1) / C) holds unit u.
__host__ __device__ inline int team_of_unit(long long u, int C, long long W) {
    const long long num = (u + 1) * C - 1;
    if (num < 0x7fffffffLL)
        return static_cast<int>(static_cast<unsigned>(num) / static_cast<unsigned>(W));
    return static_cast<int>(num / W);
}

// Row x of a group and KV head (sequence times shared query heads): its item, and
// the item's first and last unit.
struct RowPlace {
    int item, r;        // the item, and the row within it
    int half;           // rows of the first CTA, where each has half
    bool pair;
    long long u0, u1;
};
template <int DPAD>
__host__ __device__ inline RowPlace place_of(const GroupPlan &g, int kvh, int x) {
    constexpr int IR = item_rows(DPAD);
    RowPlace p;
    p.item = x / IR;
    p.r = x - p.item * IR;
    const int of_item = min(IR, g.rows - p.item * IR);
    p.half = (of_item + 1) >> 1;
    p.pair = is_pair(of_item, IR);
    p.u0 = g.first_unit + kvh * g.head_units(IR) + static_cast<long long>(p.item) * g.tiles;
    p.u1 = p.u0 + (p.pair ? g.tiles : (g.tiles + 1) >> 1) - 1;
    return p;
}
// Its teams, where items have whole ones.
__host__ __device__ inline void whole_teams_of(const GroupPlan &g, int kvh, int item, int &c0, int &c1) {
    c0 = g.first_team + kvh * ((g.items - 1) * g.teams + g.last_teams) + item * g.teams;
    c1 = c0 + (item == g.items - 1 ? g.last_teams : g.teams) - 1;
}
// The partials that teams c0 to c1 left of it: `parts` of them, `step` slots apart,
// the first at `first` = slot x rows of a block + row.
struct RowParts {
    int parts, step;
    long long first;
};
template <int DPAD>
__host__ __device__ inline RowParts parts_of(const GroupPlan &g, int kvh, const RowPlace &p, int c0, int c1) {
    const int second = p.pair && p.r >= p.half;
    RowParts v;
    v.step = p.pair ? 2 : 1;  // (both CTAs' slots where they took the tiles in turn)
    v.parts = (c1 - c0 + 1) * (p.pair ? 1 : 2);
    v.first = (2ll * (g.first_item + kvh * g.items + p.item + c0) + second) * block_rows(DPAD) + (second ? p.r - p.half : p.r);
    return v;
}

}  // namespace prefix
}  // namespace pd
