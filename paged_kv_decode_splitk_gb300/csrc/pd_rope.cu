// pd_rope.cu -- rotary positions (pd_rope_*) and the append of new tokens to
// the paged cache (pd_append_kv[_fp8]): host side and kernels.
//
// Mathematics.  Pair i of a row at position t is turned by the angle t f[i].
// The handle keeps each frequency as F[i] = frac(f[i] / 2 pi) 2^64, from doubles
// (good to 2^-52 of the frequency), and t F[i] mod 2^64, one wrapping integer
// product, is the fraction of a turn of that F exactly: no reduction loses bits at
// far positions, and negative positions wrap like the rest.  Its upper 32 bits as a
// signed number are the angle in [-1/2, 1/2) turns; sine and cosine are sincospif's.
//
// What bounds it: every element is read and written once and costs about three
// flops, so HBM does (a decode step: the launch).  A thread owns one group of
// pairs of a token (16-byte loads of both halves) and walks kRows heads with it.
// All its loads are in flight while the block works out the sines and cosines of
// its few tokens, one or two a thread, into shared memory; a thread working out
// its own, four to eight, was bound by their instructions where only a part of
// the head turns (64 single tokens of 40 heads: 2.25 -> 1.72 us).  Measured against a
// plain copy's rate: 671 MB rotated in 96 us (103%), 151 MB of rows turned in part
// in 23.4 (95%), 805 MB of new tokens in 119 (99%), 154 MB into an FP8 cache in 31.4
// (72%; four times as many tokens 87%: what is left is the start, the lookups and
// the last wave).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>
#include <cstdio>
#include <new>
#include <vector>

#include "pd.h"
#include "pd_device.cuh"
#include "pd_internal.h"
#include "pd_tcgen05.cuh"

struct pd_rope {
    int head_dim, rot_dim, layout, device;
    float factor;            // on cosine and sine
    unsigned long long *turns;  // device: [rot_dim/2] turns per position, fixed point
};

namespace pd {
namespace {

// Heads a thread takes one after another, with the same sines and cosines.
constexpr int kRows = 4;
constexpr int kRopeThreads = 256;

// How a row of head_dim columns is dealt to threads: `units` of them, the
// first pair_units with W pairs each (pairs halves apart: columns [W u, W u + W)
// and the same half a rotation on; interleaved: the 2 W neighbours), the rest
// with the copied columns.
struct RowPlan {
    FastDiv units;   // per row
    FastDiv slots;   // threads that share a token's rows
    int pair_units;
    int half;        // rot_dim / 2
    int pitch;       // of the table of sines and cosines
    FastDiv fd_half;
    const unsigned long long *turns;
    float factor;
    float sign;      // -1: the inverse
};

struct RopeParams {
    RowPlan plan;
    const __nv_bfloat16 *x;
    __nv_bfloat16 *out;
    long long x_tok, x_head, o_tok, o_head;
    const int32_t *positions;
    int heads;
    int threads;     // tokens * slots * units
};

struct AppendParams {
    RowPlan plan;
    const __nv_bfloat16 *q, *k, *v;
    long long q_tok, k_tok, v_tok;
    __nv_bfloat16 *q_out;
    void *k_cache, *v_cache;
    float k_scale, v_scale;   // of a code: 1 over the cache's scales
    const int32_t *block_table, *context_lens, *token_starts;
    int max_blocks, num_seqs, num_blocks;
    int q_heads, kv_heads, head_dim;
    FastDiv block_size;
    int threads;
    unsigned int *status;
};

// W BF16 values as one load or store of 2 W bytes.
template <int W>
struct Vec {
    uint32_t w[W >= 2 ? W / 2 : 1];
};
template <int W>
__device__ __forceinline__ Vec<W> load_vec(const __nv_bfloat16 *p) {
    Vec<W> r;
    if constexpr (W == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
    } else if constexpr (W == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x, r.w[1] = v.y;
    } else if constexpr (W == 2) {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        r.w[0] = *reinterpret_cast<const unsigned short *>(p);
    }
    return r;
}
template <int W>
__device__ __forceinline__ float elem(const Vec<W> &v, int i) {
    return (i & 1) ? dev::bf16_hi_f32(v.w[i >> 1]) : dev::bf16_lo_f32(v.w[i >> 1]);
}
template <int W>
__device__ __forceinline__ void store_bf16(__nv_bfloat16 *p, const float (&f)[W]) {
    if constexpr (W == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(dev::pack_bf16x2(f[0], f[1]), dev::pack_bf16x2(f[2], f[3]),
                                                   dev::pack_bf16x2(f[4], f[5]), dev::pack_bf16x2(f[6], f[7]));
    else if constexpr (W == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(dev::pack_bf16x2(f[0], f[1]), dev::pack_bf16x2(f[2], f[3]));
    else if constexpr (W == 2)
        *reinterpret_cast<uint32_t *>(p) = dev::pack_bf16x2(f[0], f[1]);
    else
        *p = __float2bfloat16_rn(f[0]);
}
template <int W>
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const Vec<W> &v) {
    if constexpr (W == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    else if constexpr (W == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(v.w[0], v.w[1]);
    else if constexpr (W == 2)
        *reinterpret_cast<uint32_t *>(p) = v.w[0];
    else
        *reinterpret_cast<unsigned short *>(p) = static_cast<unsigned short>(v.w[0]);
}
// Two values -> two E4M3 codes (lo in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(d) : "f"(lo), "f"(hi));
    return d;
}
template <int W>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&f)[W], float scale) {
    uint32_t c[W >= 2 ? W / 2 : 1];
    if constexpr (W >= 2) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            float x, y;
            tc::unpack_f32x2(tc::mul_f32x2(tc::pack_f32x2(f[2 * i], f[2 * i + 1]), tc::pack_f32x2(scale, scale)), x, y);
            c[i] = pack_e4m3x2(x, y);
        }
    } else {
        c[0] = pack_e4m3x2(f[0] * scale, 0.f);
    }
    if constexpr (W == 8)
        *reinterpret_cast<uint2 *>(p) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    else if constexpr (W == 4)
        *reinterpret_cast<uint32_t *>(p) = c[0] | (c[1] << 16);
    else if constexpr (W == 2)
        *reinterpret_cast<unsigned short *>(p) = static_cast<unsigned short>(c[0]);
    else
        *p = static_cast<uint8_t>(c[0]);
}

// Cosines and sines of the tokens of a block, times the factor, in dynamic
// shared memory: pair i of the block's token j at j * pitch + i, the sines `span`
// behind the cosines.  Rows are a multiple of 4 pairs, for 16-byte loads.
struct TurnTable {
    float *c;
    int span;
};
extern __shared__ __align__(16) float turn_smem[];

// Tokens that a block's threads touch at most, where a token has `per` threads.
int block_tokens(int per) { return (kRopeThreads - 2) / per + 2; }

__device__ __forceinline__ void fill_turn(const RowPlan &p, const TurnTable &tab, int at, int pair, int position) {
    const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(position)) * p.turns[pair];
    // x half-turns: the upper 32 bits, signed, over 2^31
    const float x = static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    tab.c[at] = c * p.factor;
    tab.c[tab.span + at] = s * (p.factor * p.sign);
}

// The pairs of one thread.
template <int N>
struct Turn {
    float c[N], s[N];
    int live;  // pairs that turn: an interleaved unit may end in copied columns
};
template <int N>
__device__ __forceinline__ void load_turn(const float *p, float (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + i);
            v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = p[i];
    }
}
template <int N>
__device__ __forceinline__ Turn<N> turn_of(const RowPlan &p, const TurnTable &tab, int token, int first) {
    Turn<N> t;
    t.live = p.half - first;
    load_turn<N>(tab.c + token * p.pitch + first, t.c);  // (past `live`: of the row's padding)
    load_turn<N>(tab.c + tab.span + token * p.pitch + first, t.s);
    return t;
}

// One unit of one row.  HALF: W pairs, columns a and b (or, PASS, W copied
// columns at a).  Interleaved: 2 N columns at a, N pairs.
template <bool HALF, int W>
struct Unit {
    static constexpr int kPairs = HALF ? W : W / 2;
    Vec<W> a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16 *row, int ca, int cb, bool pass) {
        a = load_vec<W>(row + ca);
        if (HALF && !pass) b = load_vec<W>(row + cb);
    }
    // rotated values of the columns at a (fa) and, HALF, at b (fb), two pairs' (or
    // both of a pair's) products an instruction
    __device__ __forceinline__ void rotate(const Turn<kPairs> &t, float (&fa)[W], float (&fb)[W]) const {
        if constexpr (HALF && W > 1) {
#pragma unroll
            for (int i = 0; i < W; i += 2) {
                const uint64_t x = tc::pack_f32x2(elem<W>(a, i), elem<W>(a, i + 1)), y = tc::pack_f32x2(elem<W>(b, i), elem<W>(b, i + 1));
                const uint64_t c = tc::pack_f32x2(t.c[i], t.c[i + 1]), s = tc::pack_f32x2(t.s[i], t.s[i + 1]);
                const uint64_t m = tc::pack_f32x2(-t.s[i], -t.s[i + 1]);
                tc::unpack_f32x2(tc::fma_f32x2(x, c, tc::mul_f32x2(y, m)), fa[i], fa[i + 1]);
                tc::unpack_f32x2(tc::fma_f32x2(y, c, tc::mul_f32x2(x, s)), fb[i], fb[i + 1]);
            }
        } else if constexpr (HALF) {
            const float x = elem<W>(a, 0), y = elem<W>(b, 0);
            fa[0] = fmaf(x, t.c[0], -(y * t.s[0]));
            fb[0] = fmaf(y, t.c[0], x * t.s[0]);
        } else {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                const float x = elem<W>(a, 2 * i), y = elem<W>(a, 2 * i + 1);
                const bool live = i < t.live;
                float u, v;
                tc::unpack_f32x2(tc::fma_f32x2(tc::pack_f32x2(x, y), tc::pack_f32x2(t.c[i], t.c[i]),
                                               tc::mul_f32x2(tc::pack_f32x2(y, x), tc::pack_f32x2(-t.s[i], t.s[i]))), u, v);
                fa[2 * i] = live ? u : x;
                fa[2 * i + 1] = live ? v : y;
            }
        }
    }
    __device__ __forceinline__ void plain(float (&fa)[W], float (&fb)[W]) const {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            fa[i] = elem<W>(a, i);
            if (HALF) fb[i] = elem<W>(b, i);
        }
    }
};

// Columns of a unit: HALF, a pair unit u has columns W u and half + W u; a
// copied unit W columns from rot on.  Interleaved: W columns at W u.
template <bool HALF, int W>
__device__ __forceinline__ void unit_columns(const RowPlan &p, int u, int &ca, int &cb, bool &pass) {
    pass = u >= p.pair_units;
    if (HALF) {
        ca = pass ? 2 * p.half + (u - p.pair_units) * W : u * W;
        cb = p.half + u * W;
    } else {
        ca = u * W;
        cb = 0;
    }
}

// Blocks an SM has room for.  More hide the wait for the loads and the table: with
// neighbouring pairs 5 (48 registers) instead of 4 take 8191 tokens of wide heads
// from 25.1 to 23.4 us.  Pairs halves apart hold twice the columns, and at 4 (64
// registers) they spill: prompts of 805 MB go from 119 to 135 us.
template <bool HALF>
constexpr int kBlocks = HALF ? 3 : 5;

template <bool HALF, int W, int ROWS>
__global__ void __launch_bounds__(kRopeThreads, kBlocks<HALF>) rope_kernel(const __grid_constant__ RopeParams p) {
    dev::griddep_launch_dependents();
    const int id = blockIdx.x * kRopeThreads + threadIdx.x;
    const int n = fast_div(id, p.plan.units);
    const int u = id - n * static_cast<int>(p.plan.units.d);
    const int tok = fast_div(n, p.plan.slots);
    const int slot = n - tok * static_cast<int>(p.plan.slots.d);
    const int first = fast_div(fast_div(blockIdx.x * kRopeThreads, p.plan.units), p.plan.slots);  // the block's tokens
    const int last = fast_div(fast_div(min(blockIdx.x * kRopeThreads + kRopeThreads, p.threads) - 1, p.plan.units), p.plan.slots);
    const TurnTable tab = {turn_smem, (last - first + 1) * p.plan.pitch};
    int ca, cb;
    bool pass;
    unit_columns<HALF, W>(p.plan, u, ca, cb, pass);
    dev::griddep_wait();
    const __nv_bfloat16 *x = p.x + tok * p.x_tok;
    const int step = static_cast<int>(p.plan.slots.d);
    const bool in = id < p.threads;
    Unit<HALF, W> un[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int h = slot + r * step;
        if (in && h < p.heads) un[r].load(x + h * p.x_head, ca, cb, pass);
    }
    for (int e = threadIdx.x; e < (last - first + 1) * p.plan.half; e += kRopeThreads) {
        const int j = fast_div(e, p.plan.fd_half);
        fill_turn(p.plan, tab, e + j * (p.plan.pitch - p.plan.half), e - j * p.plan.half, p.positions[first + j]);
    }
    __syncthreads();
    if (!in) return;
    __nv_bfloat16 *o = p.out + tok * p.o_tok;
    Turn<Unit<HALF, W>::kPairs> t;
    if (!pass) t = turn_of<Unit<HALF, W>::kPairs>(p.plan, tab, tok - first, HALF ? u * W : u * W / 2);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int h = slot + r * step;
        if (h < p.heads) {
            __nv_bfloat16 *at = o + h * p.o_head;
            if (pass) {
                store_vec<W>(at + ca, un[r].a);
            } else {
                float fa[W], fb[W];
                un[r].rotate(t, fa, fb);
                store_bf16<W>(at + ca, fa);
                if (HALF) store_bf16<W>(at + cb, fb);
            }
        }
    }
}

// The last sequence whose first row is at or before row t (starts is
// non-decreasing), searched by the whole warp: each round narrows the range
// 32 times.
__device__ __forceinline__ int warp_find_sequence(const int32_t *starts, int num_seqs, int t, int lane) {
    int lo = 0, n = num_seqs;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const bool at = i < n && starts[lo + i] <= t;
        const int below = __popc(__ballot_sync(0xffffffffu, at));
        const int pick = (below > 0 ? below - 1 : 0) * step;
        lo += pick;
        n = min(step, n - pick);
    }
    return lo;
}

template <bool HALF, int W, bool KV8, int ROWS>
__global__ void __launch_bounds__(kRopeThreads, kBlocks<HALF>) append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ int place[kRopeThreads + 2][2];  // of the block's tokens: position (-1: left out) and cache cell (-1: no block)
    dev::griddep_launch_dependents();
    const int id = blockIdx.x * kRopeThreads + threadIdx.x;
    const int lane = threadIdx.x & 31;
    const int n = fast_div(id, p.plan.units);
    const int u = id - n * static_cast<int>(p.plan.units.d);
    const int tok = fast_div(n, p.plan.slots);
    const int slot = n - tok * static_cast<int>(p.plan.slots.d);
    const int first = fast_div(fast_div(blockIdx.x * kRopeThreads, p.plan.units), p.plan.slots);  // the block's tokens
    const int count = fast_div(fast_div(min(blockIdx.x * kRopeThreads + kRopeThreads, p.threads) - 1, p.plan.units), p.plan.slots) -
                      first + 1;
    const TurnTable tab = {turn_smem, count * p.plan.pitch};
    int ca, cb;
    bool pass;
    unit_columns<HALF, W>(p.plan, u, ca, cb, pass);
    dev::griddep_wait();

    // ---- every row's loads, in flight while the token's place is looked up ----
    const int step = static_cast<int>(p.plan.slots.d);
    const int rows = p.q_heads + 2 * p.kv_heads;
    const int D = p.head_dim;
    const bool in = id < p.threads;
    Unit<HALF, W> un[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int h = slot + r * step;
        if (in && h < rows) {
            const int hk = h - p.q_heads, hv = hk - p.kv_heads;
            const __nv_bfloat16 *src = hk < 0   ? p.q + tok * p.q_tok + h * D
                                       : hv < 0 ? p.k + tok * p.k_tok + hk * D
                                                : p.v + tok * p.v_tok + hv * D;
            un[r].load(src, ca, cb, pass);
        }
    }

    // ---- where the block's tokens go: a lane for each ----
    const int bs = static_cast<int>(p.block_size.d);
    for (int j0 = threadIdx.x - lane; j0 < count; j0 += kRopeThreads) {
        const int j = j0 + lane, token = first + j;
        int s = token, pos = -1;
        bool has = j < count;
        if (p.token_starts) {
            // a warp's tokens are in order: find its first one's sequence together,
            // then step on to each lane's own
            s = warp_find_sequence(p.token_starts, p.num_seqs, first + j0, lane);
            if (has) {
                while (s + 1 < p.num_seqs && p.token_starts[s + 1] <= token) ++s;
                const int end = p.token_starts[s + 1];
                has = token >= p.token_starts[s] && token < end;  // else a row of no sequence
                if (has) pos = p.context_lens[s] - (end - token);
            }
        } else if (has) {
            pos = p.context_lens[s] - 1;
            has = pos != -1;  // an empty sequence has no new token
        }
        if (has && (pos < 0 || pos >= p.max_blocks * bs)) {
            dev::flag_status(p.status, PD_DEV_BAD_CONTEXT_LEN);
            has = false;
        }
        int bid = -1;
        if (has) {
            bid = p.block_table[static_cast<long long>(s) * p.max_blocks + fast_div(pos, p.block_size)];
            if (bid < 0 || bid >= p.num_blocks) {
                dev::flag_status(p.status, PD_DEV_BAD_BLOCK_ID);
                bid = -1;
            }
        }
        if (j < count) {
            place[j][0] = has ? pos : -1;
            place[j][1] = bid;
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < count * p.plan.half; e += kRopeThreads) {
        const int j = fast_div(e, p.plan.fd_half);
        fill_turn(p.plan, tab, e + j * (p.plan.pitch - p.plan.half), e - j * p.plan.half, place[j][0]);
    }
    __syncthreads();
    if (!in) return;
    const int pos = place[tok - first][0], bid = place[tok - first][1];
    if (pos < 0) return;
    const bool bad = bid < 0;
    const long long cell = (static_cast<long long>(bid) * bs + (pos - fast_div(pos, p.block_size) * bs)) * p.kv_heads;
    Turn<Unit<HALF, W>::kPairs> t;
    if (!pass && slot < p.q_heads + p.kv_heads)  // (a thread's first row: the others lie behind it)
        t = turn_of<Unit<HALF, W>::kPairs>(p.plan, tab, tok - first, HALF ? u * W : u * W / 2);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int h = slot + r * step;
        if (h < rows) {
            const int hk = h - p.q_heads, hv = hk - p.kv_heads;
            const bool copied = pass || hv >= 0;
            const long long at = (cell + (hv < 0 ? hk : hv)) * D;  // in a cache
            if (KV8 && hk >= 0) {
                if (!bad) {
                    float fa[W], fb[W];
                    if (copied)
                        un[r].plain(fa, fb);
                    else
                        un[r].rotate(t, fa, fb);
                    const float scale = hv < 0 ? p.k_scale : p.v_scale;
                    uint8_t *o = static_cast<uint8_t *>(hv < 0 ? p.k_cache : p.v_cache) + at;
                    store_e4m3<W>(o + ca, fa, scale);
                    if (HALF && !pass) store_e4m3<W>(o + cb, fb, scale);
                }
            } else if (hk < 0 || !bad) {
                __nv_bfloat16 *o = hk < 0 ? p.q_out + (static_cast<long long>(tok) * p.q_heads + h) * D
                                          : static_cast<__nv_bfloat16 *>(hv < 0 ? p.k_cache : p.v_cache) + at;
                if (copied) {
                    store_vec<W>(o + ca, un[r].a);
                    if (HALF && !pass) store_vec<W>(o + cb, un[r].b);
                } else {
                    float fa[W], fb[W];
                    un[r].rotate(t, fa, fb);
                    store_bf16<W>(o + ca, fa);
                    if (HALF) store_bf16<W>(o + cb, fb);
                }
            }
        }
    }
}

// ---- host side --------------------------------------------------------------------

// Pairs a thread's load holds: as many of 8, 4, 2, 1 as divide half a rotation
// (and so, head_dim being a multiple of 8, the copied columns); interleaved
// units are always 8 columns.  Bound by the number of loads and stores, of 2 W bytes,
// where W is small: 32768 tokens x 40 heads of 128 columns take 98 us at W = 8 (rot
// 128; HBM), 107 at 4 (rot 120), 158 at 2 (116) and 440 at 1 (126), an append of 16384
// tokens 63, 81, 133 and 225, 64 single tokens 2.7 to 3.3.  A wider load of the second
// half would begin off its alignment.
int unit_width(int layout, int rot_dim) {
    if (layout == PD_ROPE_INTERLEAVED) return 8;
    const int half = rot_dim / 2;
    int w = 8;
    while (half % w) w /= 2;
    return w;
}

// A copy (no rotation) is a rotation of no pairs: rot_dim 0.
RowPlan plan_rows(int head_dim, int rot_dim, int layout, int w, const unsigned long long *turns, float factor,
                  bool inverse) {
    RowPlan p = {};
    p.half = rot_dim / 2;
    p.fd_half = make_fastdiv(p.half);
    p.pitch = (p.half + 3) / 4 * 4;
    if (layout == PD_ROPE_HALF) {
        p.pair_units = p.half / w;
        p.units = make_fastdiv(p.pair_units + (head_dim - rot_dim) / w);
    } else {
        p.pair_units = (rot_dim + w - 1) / w;
        p.units = make_fastdiv(head_dim / w);
    }
    p.turns = turns;
    p.factor = factor;
    p.sign = inverse ? -1.f : 1.f;
    return p;
}

template <class Params, class Kernel>
cudaError_t launch_rows(Kernel kern, const Params &p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.threads + kRopeThreads - 1) / kRopeThreads));
    cfg.blockDim = dim3(kRopeThreads);
    const int per = static_cast<int>(p.plan.units.d * p.plan.slots.d);
    cfg.dynamicSmemBytes = static_cast<size_t>(block_tokens(per)) * p.plan.pitch * 2 * sizeof(float);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Threads of a launch, with kRows rows each where that still fills the GPU
// and one each where the batch is small (more threads, a shorter chain).
// Returns false where they pass 31 bits.
bool deal_rows(RowPlan *plan, int tokens, int rows, bool *many, int *threads) {
    const long long units = static_cast<long long>(tokens) * plan->units.d;
    *many = units * rows > 4ll * 152 * 2048;
    plan->slots = make_fastdiv(*many ? (rows + kRows - 1) / kRows : rows);
    const long long n = units * plan->slots.d;
    if (n > 0x7fffffffLL - kRopeThreads) return false;
    *threads = static_cast<int>(n);
    return true;
}

template <int ROWS>
cudaError_t rope_dispatch(int layout, int w, const RopeParams &p, cudaStream_t st) {
    if (layout == PD_ROPE_INTERLEAVED) return launch_rows(rope_kernel<false, 8, ROWS>, p, st);
    if (w == 8) return launch_rows(rope_kernel<true, 8, ROWS>, p, st);
    if (w == 4) return launch_rows(rope_kernel<true, 4, ROWS>, p, st);
    if (w == 2) return launch_rows(rope_kernel<true, 2, ROWS>, p, st);
    return launch_rows(rope_kernel<true, 1, ROWS>, p, st);
}

template <bool KV8, int ROWS>
cudaError_t append_dispatch(int layout, int w, const AppendParams &p, cudaStream_t st) {
    if (layout == PD_ROPE_INTERLEAVED) return launch_rows(append_kernel<false, 8, KV8, ROWS>, p, st);
    if (w == 8) return launch_rows(append_kernel<true, 8, KV8, ROWS>, p, st);
    if (w == 4) return launch_rows(append_kernel<true, 4, KV8, ROWS>, p, st);
    if (w == 2) return launch_rows(append_kernel<true, 2, KV8, ROWS>, p, st);
    return launch_rows(append_kernel<true, 1, KV8, ROWS>, p, st);
}

int check_handle(const char *what, const pd_rope *rope) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return report_cuda(e, what);
    if (dev != rope->device)
        return report(PD_ERR_INVALID, "%s: the rotation was created on device %d, the current device is %d", what,
                      rope->device, dev);
    return PD_OK;
}

int append_impl(const char *what, const pd_rope *rope, const void *q, int64_t q_tok, const void *k, int64_t k_tok,
                const void *v, int64_t v_tok, void *q_out, void *k_cache, void *v_cache, float k_scale, float v_scale,
                const int32_t *block_table, int max_blocks, const int32_t *context_lens, const int32_t *token_starts,
                int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                int num_blocks, void *stream, bool kv8) {
    int rc = check_shape(q ? num_q_heads : num_kv_heads, num_kv_heads, head_dim, block_size);
    if (rc != PD_OK) return rc;
    if (kv8) {
        if (head_dim % 16 != 0)
            return report(PD_ERR_UNSUPPORTED, "FP8 cache: head_dim %d must be a multiple of 16", head_dim);
        if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || !(k_scale >= FLT_MIN) ||
            !(v_scale >= FLT_MIN) || !(1.f / k_scale >= FLT_MIN) || !(1.f / v_scale >= FLT_MIN))
            return report(PD_ERR_INVALID, "FP8 cache: k_scale and v_scale must be finite, positive and no subnormal numbers, nor their "
                                          "reciprocals");
    }
    if (num_tokens < 0 || num_seqs < 0)
        return report(PD_ERR_INVALID, "%s: num_tokens %d, num_seqs %d", what, num_tokens, num_seqs);
    if (!token_starts && num_tokens != num_seqs)
        return report(PD_ERR_INVALID, "%s: without token_starts every sequence has one token (num_tokens %d, num_seqs %d)",
                      what, num_tokens, num_seqs);
    if (rope) {
        if (rope->head_dim != head_dim)
            return report(PD_ERR_INVALID, "%s: head_dim %d, the rotation's is %d", what, head_dim, rope->head_dim);
        rc = check_handle(what, rope);
        if (rc != PD_OK) return rc;
    }
    if (num_tokens == 0 || num_seqs == 0) return report_ok();
    if (!k || !v || !k_cache || !v_cache || !block_table || !context_lens || (q && !q_out))
        return report(PD_ERR_INVALID, "%s: null tensor pointer", what);
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) ||
        !aligned16(v_cache))
        return report(PD_ERR_INVALID, "%s: q, k, v, q_out and the caches must be 16-byte aligned", what);
    const long long kv_row = static_cast<long long>(num_kv_heads) * head_dim;
    const long long q_row = q ? static_cast<long long>(num_q_heads) * head_dim : 0;
    if ((q && (q_tok < q_row || q_tok % 8)) || k_tok < kv_row || k_tok % 8 || v_tok < kv_row || v_tok % 8)
        return report(PD_ERR_INVALID,
                      "%s: token strides (q %lld, k %lld, v %lld) must be multiples of 8 elements and hold a token's rows",
                      what, static_cast<long long>(q_tok), static_cast<long long>(k_tok), static_cast<long long>(v_tok));
    if (q == q_out && q && q_tok != q_row)
        return report(PD_ERR_INVALID, "%s: in place (q_out == q) needs contiguous q", what);
    if (max_blocks <= 0 || num_blocks <= 0)
        return report(PD_ERR_INVALID, "max_blocks_per_seq (%d) and num_blocks (%d) must be positive", max_blocks,
                      num_blocks);
    if (static_cast<long long>(max_blocks) * block_size > 0x7fffffffLL)
        return report(PD_ERR_INVALID, "max_blocks_per_seq * block_size overflows int32");

    int err = PD_OK;
    AppendParams p = {};
    p.status = device_status_word(&err);
    if (!p.status) return err;
    const int layout = rope ? rope->layout : PD_ROPE_INTERLEAVED;
    const int rot = rope ? rope->rot_dim : 0;
    const int w = unit_width(layout, rot);
    p.plan = plan_rows(head_dim, rot, layout, w, rope ? rope->turns : nullptr, rope ? rope->factor : 1.f, false);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_tok = q_tok;
    p.k_tok = k_tok;
    p.v_tok = v_tok;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_scale = 1.f / k_scale;
    p.v_scale = 1.f / v_scale;
    p.block_table = block_table;
    p.context_lens = context_lens;
    p.token_starts = token_starts;
    p.max_blocks = max_blocks;
    p.num_seqs = num_seqs;
    p.num_blocks = num_blocks;
    p.q_heads = q ? num_q_heads : 0;
    p.kv_heads = num_kv_heads;
    p.head_dim = head_dim;
    p.block_size = make_fastdiv(block_size);
    bool many = false;
    if (!deal_rows(&p.plan, num_tokens, p.q_heads + 2 * num_kv_heads, &many, &p.threads))
        return report(PD_ERR_INVALID, "%s: launch too large (%d tokens)", what, num_tokens);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = kv8 ? (many ? append_dispatch<true, kRows>(layout, w, p, st) : append_dispatch<true, 1>(layout, w, p, st))
                              : (many ? append_dispatch<false, kRows>(layout, w, p, st) : append_dispatch<false, 1>(layout, w, p, st));
    if (e != cudaSuccess) return report_cuda(e, what);
    return report_ok();
}

int check_desc(const pd_rope_desc *d) {
    if (!d) return report(PD_ERR_INVALID, "null rope description");
    if (d->head_dim < 8 || d->head_dim > PD_MAX_HEAD_DIM || d->head_dim % 8)
        return report(PD_ERR_UNSUPPORTED, "rope: head_dim %d must be a multiple of 8 in [8, %d]", d->head_dim,
                      PD_MAX_HEAD_DIM);
    if (d->rot_dim < 2 || d->rot_dim > d->head_dim || d->rot_dim % 2)
        return report(PD_ERR_INVALID, "rope: rot_dim %d must be even and in [2, %d]", d->rot_dim, d->head_dim);
    if (d->layout != PD_ROPE_HALF && d->layout != PD_ROPE_INTERLEAVED)
        return report(PD_ERR_INVALID, "rope: unknown layout %d", d->layout);
    if (d->scaling < PD_ROPE_NONE || d->scaling > PD_ROPE_TABLE)
        return report(PD_ERR_INVALID, "rope: unknown scaling rule %d", d->scaling);
    if (!std::isfinite(d->attention_factor) || d->attention_factor < 0)
        return report(PD_ERR_INVALID, "rope: attention_factor must be finite and not negative");
    if (d->scaling == PD_ROPE_TABLE) {
        if (!d->frequencies) return report(PD_ERR_INVALID, "rope: the table rule needs frequencies");
        for (int i = 0; i < d->rot_dim / 2; ++i)
            if (!std::isfinite(d->frequencies[i])) return report(PD_ERR_INVALID, "rope: frequency %d is not finite", i);
        return PD_OK;
    }
    if (!std::isfinite(d->base) || d->base <= 1) return report(PD_ERR_INVALID, "rope: base must be finite and above 1");
    if (d->scaling == PD_ROPE_NONE) return PD_OK;
    if (!std::isfinite(d->factor) || d->factor <= 0) return report(PD_ERR_INVALID, "rope: factor must be finite and positive");
    if (d->scaling == PD_ROPE_NTK && d->rot_dim < 4) return report(PD_ERR_INVALID, "rope: the NTK rule needs rot_dim >= 4");
    if (d->scaling == PD_ROPE_BANDED || d->scaling == PD_ROPE_YARN) {
        if (!std::isfinite(d->original_context) || d->original_context <= 0)
            return report(PD_ERR_INVALID, "rope: original_context must be finite and positive");
        const bool unset = d->low_turns == 0 && d->high_turns == 0;
        if (!unset && !(std::isfinite(d->low_turns) && std::isfinite(d->high_turns) && d->low_turns > 0 &&
                        d->high_turns > d->low_turns))
            return report(PD_ERR_INVALID, "rope: low_turns and high_turns must be finite with 0 < low < high (or both 0)");
    }
    return PD_OK;
}

constexpr double kPi = 3.14159265358979323846;

// The rule's frequencies; returns c.
double rule_frequencies(const pd_rope_desc *d, double *f) {
    const int rot = d->rot_dim, half = rot / 2;
    const double s = d->factor;
    double base = d->base, low = d->low_turns, high = d->high_turns, c = 1.0;
    if (low == 0 && high == 0) {
        low = 1;
        high = d->scaling == PD_ROPE_YARN ? 32 : 4;
    }
    if (d->scaling == PD_ROPE_NTK) base *= std::pow(s, static_cast<double>(rot) / (rot - 2));
    double i0 = 0, i1 = 0;
    if (d->scaling == PD_ROPE_YARN) {
        auto pair_of = [&](double n) { return rot * std::log(d->original_context / (2 * kPi * n)) / (2 * std::log(base)); };
        i0 = std::fmax(std::floor(pair_of(high)), 0.0);
        i1 = std::fmin(std::ceil(pair_of(low)), rot - 1.0);
        c = s > 1 ? 0.1 * std::log(s) + 1 : 1.0;
    }
    for (int i = 0; i < half; ++i) {
        if (d->scaling == PD_ROPE_TABLE) {
            f[i] = d->frequencies[i];
            continue;
        }
        const double f0 = std::pow(base, -2.0 * i / rot);
        f[i] = f0;
        if (d->scaling == PD_ROPE_LINEAR) f[i] = f0 / s;
        if (d->scaling == PD_ROPE_BANDED) {
            const double n = d->original_context * f0 / (2 * kPi);
            const double w = std::fmin(std::fmax((n - low) / (high - low), 0.0), 1.0);
            f[i] = f0 * (w + (1 - w) / s);
        }
        if (d->scaling == PD_ROPE_YARN) {
            const double r = std::fmin(std::fmax((i - i0) / std::fmax(i1 - i0, 0.001), 0.0), 1.0);
            f[i] = f0 * (1 - r + r / s);
        }
    }
    return d->attention_factor > 0 ? d->attention_factor : c;
}

// Turns per position as a 64-bit binary fraction (whole turns drop out).
unsigned long long fixed_turns(double f) {
    double t = f / (2 * kPi);
    t -= std::floor(t);  // [0, 1]: a tiny negative rounds up to 1, which is no turn
    return t >= 1.0 ? 0ull : static_cast<unsigned long long>(t * 18446744073709551616.0);
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" {

int pd_rope_frequencies(const pd_rope_desc *desc, double *frequencies, double *attention_factor) {
    const int rc = check_desc(desc);
    if (rc != PD_OK) return rc;
    double f[PD_MAX_HEAD_DIM / 2];
    const double c = rule_frequencies(desc, f);
    for (int i = 0; frequencies && i < desc->rot_dim / 2; ++i) frequencies[i] = f[i];
    if (attention_factor) *attention_factor = c;
    return report_ok();
}

int pd_rope_create(const pd_rope_desc *desc, pd_rope **out) {
    if (!out) return report(PD_ERR_INVALID, "null out");
    *out = nullptr;
    const int rc = check_desc(desc);
    if (rc != PD_OK) return rc;
    double f[PD_MAX_HEAD_DIM / 2];
    unsigned long long turns[PD_MAX_HEAD_DIM / 2];
    const double c = rule_frequencies(desc, f);
    const int half = desc->rot_dim / 2;
    for (int i = 0; i < half; ++i) turns[i] = fixed_turns(f[i]);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return report_cuda(e, "cudaGetDevice");
    pd_rope *r = new (std::nothrow) pd_rope();
    if (!r) return report(PD_ERR_ALLOC, "rope handle: out of host memory");
    r->head_dim = desc->head_dim;
    r->rot_dim = desc->rot_dim;
    r->layout = desc->layout;
    r->device = dev;
    r->factor = static_cast<float>(c);
    void *p = nullptr;
    e = inject_alloc_failure() ? cudaErrorMemoryAllocation : cudaMalloc(&p, half * sizeof turns[0]);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        delete r;
        return report(PD_ERR_ALLOC, "rope table allocation failed: %s", cudaGetErrorString(e));
    }
    r->turns = static_cast<unsigned long long *>(p);
    e = cudaMemcpy(p, turns, half * sizeof turns[0], cudaMemcpyHostToDevice);
    // a copy from pageable host memory may return before its last part has landed
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        cudaFree(p);
        delete r;
        return report_cuda(e, "rope table copy");
    }
    *out = r;
    return report_ok();
}

void pd_rope_destroy(pd_rope *rope) {
    if (!rope) return;
    int cur = 0;
    cudaGetDevice(&cur);
    cudaSetDevice(rope->device);
    cudaDeviceSynchronize();
    cudaFree(rope->turns);
    cudaSetDevice(cur);
    delete rope;
}

int pd_rope_apply(const pd_rope *rope, const void *x, int64_t x_token_stride, int64_t x_head_stride,
                  const int32_t *positions, void *out, int64_t out_token_stride, int64_t out_head_stride,
                  int num_tokens, int num_heads, int inverse, void *stream) {
    if (!rope) return report(PD_ERR_INVALID, "pd_rope_apply: null handle");
    if (num_tokens < 0 || num_heads < 0)
        return report(PD_ERR_INVALID, "pd_rope_apply: num_tokens %d, num_heads %d", num_tokens, num_heads);
    if (inverse != 0 && inverse != 1) return report(PD_ERR_INVALID, "pd_rope_apply: inverse must be 0 or 1");
    const int rc = check_handle("pd_rope_apply", rope);
    if (rc != PD_OK) return rc;
    if (num_tokens == 0 || num_heads == 0) return report_ok();
    if (!x || !positions || !out) return report(PD_ERR_INVALID, "pd_rope_apply: null tensor pointer");
    if (!aligned16(x) || !aligned16(out))
        return report(PD_ERR_INVALID, "pd_rope_apply: x and out must be 16-byte aligned");
    const int64_t strides[4] = {x_token_stride, x_head_stride, out_token_stride, out_head_stride};
    for (int64_t s : strides)
        if (s <= 0 || s % 8)
            return report(PD_ERR_INVALID, "pd_rope_apply: strides must be positive multiples of 8 elements (got %lld)",
                          static_cast<long long>(s));
    if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride))
        return report(PD_ERR_INVALID, "pd_rope_apply: in place (out == x) needs equal strides");
    // rows of out that share elements would be written by several threads: a token's
    // heads lie within its stride, or a head's tokens within the head's
    const int64_t T = num_tokens, H = num_heads, D = rope->head_dim, ot = out_token_stride, oh = out_head_stride;
    const bool by_token = (H == 1 || oh >= D) && (T == 1 || (ot >= D && (ot - D) / oh >= H - 1));
    const bool by_head = (T == 1 || ot >= D) && (H == 1 || (oh >= D && (oh - D) / ot >= T - 1));
    if (!by_token && !by_head)
        return report(PD_ERR_INVALID, "pd_rope_apply: rows of out overlap (strides %lld and %lld, %d tokens of %d heads)",
                      static_cast<long long>(ot), static_cast<long long>(oh), num_tokens, num_heads);
    RopeParams p = {};
    const int w = unit_width(rope->layout, rope->rot_dim);
    p.plan = plan_rows(rope->head_dim, rope->rot_dim, rope->layout, w, rope->turns, rope->factor, inverse != 0);
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.x_tok = x_token_stride;
    p.x_head = x_head_stride;
    p.o_tok = out_token_stride;
    p.o_head = out_head_stride;
    p.positions = positions;
    p.heads = num_heads;
    bool many = false;
    if (!deal_rows(&p.plan, num_tokens, num_heads, &many, &p.threads))
        return report(PD_ERR_INVALID, "pd_rope_apply: launch too large (%d tokens of %d heads)", num_tokens, num_heads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = many ? rope_dispatch<kRows>(rope->layout, w, p, st) : rope_dispatch<1>(rope->layout, w, p, st);
    if (e != cudaSuccess) return report_cuda(e, "rope launch");
    return report_ok();
}

int pd_append_kv(const pd_rope *rope, const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride,
                 const void *v, int64_t v_token_stride, void *q_out, void *k_cache, void *v_cache,
                 const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens,
                 const int32_t *token_starts, int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads,
                 int head_dim, int block_size, int num_blocks, void *stream) {
    return append_impl("pd_append_kv", rope, q, q_token_stride, k, k_token_stride, v, v_token_stride, q_out, k_cache,
                       v_cache, 1.f, 1.f, block_table, max_blocks_per_seq, context_lens, token_starts, num_tokens,
                       num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, stream, false);
}

int pd_append_kv_fp8(const pd_rope *rope, const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride,
                     const void *v, int64_t v_token_stride, void *q_out, void *k_cache, void *v_cache, float k_scale,
                     float v_scale, const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens,
                     const int32_t *token_starts, int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads,
                     int head_dim, int block_size, int num_blocks, void *stream) {
    return append_impl("pd_append_kv_fp8", rope, q, q_token_stride, k, k_token_stride, v, v_token_stride, q_out,
                       k_cache, v_cache, k_scale, v_scale, block_table, max_blocks_per_seq, context_lens, token_starts,
                       num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, stream, true);
}

}  // extern "C"
