// pd_norm.cu -- the RMS norm of each query or key head with the position rotation in
// the same pass (pd_norm_rope_*), and both on the way into the paged cache
// (pd_append_kv_normed[_fp8]): host side and kernels.
//
// Mathematics.  A row x of D columns becomes
//   y = R (x r w'),  r = 1 / sqrt(sum x^2 / D + eps),  w' = offset + w,
// with R the rotation by the row's position (its factor among it).  With
// u = R^T dy (the transposed rotation of the gradient) and the sums over the row,
//   dx = r (u w' - x r^2 sum(x u w') / D),   dw = sum over rows of u x r.
//
// A row is held by D / 16 lanes (rounded up to 4, 8 or 16), two chunks of 8 columns
// each, in 16-byte loads: chunks that pair up where pairs are whole chunks apart, so that
// a rotation stays in the lane and needs a sine and a cosine for two columns; chunks half
// a row apart where pairs are neighbours (32 bytes side by side for a lane took an append
// of wide heads 131 us for 117); neighbouring chunks otherwise.  The row's sums go across
// its lanes by shuffles.  Sines and cosines are those of the block's tokens from a table in
// shared memory, as in pd_rope.cu, and
// a lane walks several heads of its token with them.  All arithmetic is FP32; a result
// is rounded once.  dw is summed in a fixed order: a lane's rows, the rows of a block, the
// blocks.
//
// What bounds it is memory: 4 bytes an element forward, 6 backward.  Where rows are many, the
// blocks that fit the GPU share the tokens out evenly, and a line of lanes walks the rows of
// its block with the loads of the next few rows in flight all the time.  16384 x 32 heads of
// 128 columns forward 46.6 us (5760 GB/s, 85% of a copy's rate), backward 73 (82%), an append
// of 32784 tokens with wide heads 117 (85%); a row a line with a block for each few of them
// measured 46.6, 79.8 and 148 (for 131 then), turns that are made for the rows in flight
// alone 50, 82 and 148, three blocks a multiprocessor with half the loads 46.4, 87.7 and 146.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "pd.h"
#include "pd_device.cuh"
#include "pd_internal.h"
#include "pd_rope.cuh"

namespace pd {
namespace {

using namespace rope;

constexpr int kNormThreads = kRopeThreads;
constexpr int kStreams = 152;        // blocks of a kernel that walks rows: a few for each multiprocessor
constexpr int kAhead = 4;            // rows whose loads are in flight
constexpr int kGradAhead = 2;        // of x and the gradient
constexpr int kTableBytes = 28672;   // of sines and cosines that a walk holds at most

// How a row's pairs lie in its lanes' chunks: kNeighbours, two columns side by side
// (also where nothing turns), kHalves, a lane's one chunk with its other, kScattered,
// anywhere.
enum Pairs { kNeighbours, kHalves, kScattered };

struct Norm {
    const __nv_bfloat16 *weight;  // null: 1 (with offset 0)
    float offset, eps, inv_dim;
    int head_dim;
};

struct NormParams {
    RowPlan plan;   // units: lanes of a row
    Norm norm;
    const __nv_bfloat16 *x;
    __nv_bfloat16 *out;
    long long x_tok, x_head, o_tok, o_head;
    const int32_t *positions;
    int heads;
    int threads;    // tokens * slots * units
    FastDiv fd_heads;     // of a walk: the heads, the tokens, and those whose turns are held at a time
    int tokens, held;
};

struct GradParams {
    RowPlan plan;   // (its sign makes the rotation the transposed one)
    Norm norm;
    const __nv_bfloat16 *x, *g;
    __nv_bfloat16 *dx;
    long long x_tok, x_head, g_tok, g_head, d_tok, d_head;
    const int32_t *positions;
    int heads;
    FastDiv fd_heads;
    int tokens, held;
    float *part;    // [blocks][lanes * 16]: sums of dw, a lane's chunks side by side; null: not wanted
};

struct NormAppendParams {
    RowPlan plan;
    Norm norm;      // (of q)
    const __nv_bfloat16 *k_weight;
    const __nv_bfloat16 *q, *k, *v;
    long long q_tok, k_tok, v_tok;
    __nv_bfloat16 *q_out;
    void *k_cache, *v_cache;
    float k_scale, v_scale;   // of a code: 1 over the cache's scales
    const int32_t *block_table, *context_lens, *token_starts;
    int max_blocks, num_seqs, num_blocks;
    int q_heads, kv_heads;
    FastDiv block_size;
    int threads;
    FastDiv fd_rows;      // of a walk: rows of a token
    int tokens, held;
    unsigned int *status;
};

// A lane's two chunks of a row.
struct Chunks {
    uint4 a, b;
};
__device__ __forceinline__ void widen(const uint4 &v, float *f) {
    f[0] = dev::bf16_lo_f32(v.x), f[1] = dev::bf16_hi_f32(v.x), f[2] = dev::bf16_lo_f32(v.y), f[3] = dev::bf16_hi_f32(v.y);
    f[4] = dev::bf16_lo_f32(v.z), f[5] = dev::bf16_hi_f32(v.z), f[6] = dev::bf16_lo_f32(v.w), f[7] = dev::bf16_hi_f32(v.w);
}
__device__ __forceinline__ uint4 narrow(const float *f) {
    return make_uint4(dev::pack_bf16x2(f[0], f[1]), dev::pack_bf16x2(f[2], f[3]), dev::pack_bf16x2(f[4], f[5]),
                      dev::pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void widen(const Chunks &v, float (&f)[16]) {
    widen(v.a, f);
    widen(v.b, f + 8);
}
// The sum over a row's lanes.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// A lane's columns: chunks at ca and cb, of which it has those within the row.
template <int LANES, Pairs PAIRS>
struct Columns {
    int u, ca, cb;
    bool a, b;
    __device__ __forceinline__ Columns(const RowPlan &p, int head_dim) {
        u = threadIdx.x % LANES;
        ca = 16 * u;
        cb = ca + 8;
        if (PAIRS == kNeighbours) {  // (16 bytes of neighbouring lanes side by side)
            const int first = (head_dim + 8) / 16 * 8;
            ca = 8 * u < first ? 8 * u : head_dim;
            cb = ca + first;
        } else if (PAIRS == kHalves) {
            const int paired = p.half / 8;  // lanes with chunks that pair up; the others have copied ones
            ca = u < paired ? 8 * u : 2 * p.half + 16 * (u - paired);
            cb = u < paired ? p.half + 8 * u : ca + 8;
        }
        a = ca < head_dim;
        b = cb < head_dim;
    }
    __device__ __forceinline__ Chunks load(const __nv_bfloat16 *row) const {
        Chunks v = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (a) v.a = *reinterpret_cast<const uint4 *>(row + ca);
        if (b) v.b = *reinterpret_cast<const uint4 *>(row + cb);
        return v;
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *row, const float (&f)[16]) const {
        if (a) *reinterpret_cast<uint4 *>(row + ca) = narrow(f);
        if (b) *reinterpret_cast<uint4 *>(row + cb) = narrow(f + 8);
    }
    __device__ __forceinline__ void weight(const __nv_bfloat16 *w, float offset, float (&f)[16]) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 1.f;
        if (!w) return;
        widen(load(w), f);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] += offset;
    }
};

// y over its row's root mean square, times the weight.
template <int LANES>
__device__ __forceinline__ void scale_row(float (&y)[16], const float (&w)[16], const Norm &norm) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(y[i], y[i], sum);
    const float scale = rsqrtf(fmaf(row_sum<LANES>(sum), norm.inv_dim, norm.eps));
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] *= scale * w[i];
}

// The turns of a lane's columns for one token.
template <int LANES, Pairs PAIRS>
struct Turns {
    float c[PAIRS == kScattered ? 1 : 8], s[PAIRS == kScattered ? 1 : 8];
    int live;           // pairs of the lane that turn (kNeighbours: of its chunks, 4 bits each)
    const float *cos;   // kScattered: the token's table
    int span, half;

    __device__ __forceinline__ void load(const RowPlan &p, const TurnTable &tab, int token, const Columns<LANES, PAIRS> &at) {
        cos = tab.c + token * p.pitch;
        span = tab.span;
        half = p.half;
        live = 0;
        if constexpr (PAIRS == kScattered) return;
        live = PAIRS == kHalves ? (at.ca < half ? 8 : 0) : min(max(half - at.ca / 2, 0), 4) + (min(max(half - at.cb / 2, 0), 4) << 4);
        if (live > 0) {  // (rows of the table are multiples of 4 pairs, and begin at one)
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const int pair = PAIRS == kHalves ? at.ca + i : (i ? at.cb : at.ca) / 2;
                if (pair < half) {
                    const float4 x = *reinterpret_cast<const float4 *>(cos + pair), y = *reinterpret_cast<const float4 *>(cos + span + pair);
                    c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
                    s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
                }
            }
        }
    }
    // `row`: kScattered: the row's LANES * 16 floats of shared memory (all lanes of the
    // warp take part).
    __device__ __forceinline__ void apply(float (&y)[16], float *row, const Columns<LANES, PAIRS> &at) const {
        if constexpr (PAIRS == kHalves) {
            if (live == 0) return;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = y[i], b = y[8 + i];
                y[i] = fmaf(a, c[i], -(b * s[i]));
                y[8 + i] = fmaf(b, c[i], a * s[i]);
            }
        } else if constexpr (PAIRS == kNeighbours) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = y[2 * i], b = y[2 * i + 1];
                if (i < 4 ? i < (live & 15) : i - 4 < live >> 4) {
                    y[2 * i] = fmaf(a, c[i], -(b * s[i]));
                    y[2 * i + 1] = fmaf(b, c[i], a * s[i]);
                }
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(row + at.ca + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int col = at.ca + i, pair = col < half ? col : col - half;
                if (pair < half) {
                    const float cc = cos[pair], ss = cos[span + pair];
                    y[i] = col < half ? fmaf(y[i], cc, -(row[col + half] * ss)) : fmaf(y[i], cc, row[pair] * ss);
                }
            }
        }
    }
};

// A thread's place: its line of lanes, the line's token and first head.
template <int LANES>
struct Place {
    int line, tok, slot, first, last;  // (first, last: of the block's tokens)
    bool in;
    __device__ __forceinline__ Place(const RowPlan &p, int block, int threads) {
        const int id = block * kNormThreads + threadIdx.x, n = id / LANES;
        line = threadIdx.x / LANES;
        tok = fast_div(n, p.slots);
        slot = n - tok * static_cast<int>(p.slots.d);
        first = fast_div(block * kNormThreads / LANES, p.slots);
        last = fast_div((min(block * kNormThreads + kNormThreads, threads) - 1) / LANES, p.slots);
        in = id < threads;
    }
};

// Shared memory of the scattered pairs' rows.
template <int LANES, Pairs PAIRS>
struct Exchange {
    float v[PAIRS == kScattered ? kNormThreads * 16 : 4];
    __device__ __forceinline__ float *row(int line) { return PAIRS == kScattered ? v + line * (LANES * 16) : nullptr; }
};

// One row a line: where rows are few.
template <int LANES, Pairs PAIRS>
__global__ void __launch_bounds__(kNormThreads, 4) norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ __align__(16) Exchange<LANES, PAIRS> rows;
    dev::griddep_launch_dependents();
    const Place<LANES> at(p.plan, blockIdx.x, p.threads);
    const Columns<LANES, PAIRS> cols(p.plan, p.norm.head_dim);
    const TurnTable tab = {turn_smem, (at.last - at.first + 1) * p.plan.pitch};
    dev::griddep_wait();
    Chunks v = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (at.in) v = cols.load(p.x + at.tok * p.x_tok + at.slot * p.x_head);
    for (int e = threadIdx.x; e < (at.last - at.first + 1) * p.plan.half; e += kNormThreads) {
        const int j = fast_div(e, p.plan.fd_half);
        fill_turn(p.plan, tab, e + j * (p.plan.pitch - p.plan.half), e - j * p.plan.half, p.positions[at.first + j]);
    }
    float w[16], y[16];
    cols.weight(p.norm.weight, p.norm.offset, w);
    __syncthreads();
    Turns<LANES, PAIRS> turns;
    turns.load(p.plan, tab, min(at.tok, at.last) - at.first, cols);
    widen(v, y);
    scale_row<LANES>(y, w, p.norm);
    turns.apply(y, rows.row(at.line), cols);
    if (at.in) cols.store(p.out + at.tok * p.o_tok + at.slot * p.o_head, y);
}

// The tokens that a block of a walk has, one after another.  (Every gridDim.x-th instead, so
// that all blocks are near each other in memory, is 6% slower forward and 8% backward.)
struct Share {
    int first, count;
    __device__ __forceinline__ explicit Share(int tokens)
        : first(static_cast<int>(static_cast<long long>(tokens) * blockIdx.x / gridDim.x)),
          count(static_cast<int>(static_cast<long long>(tokens) * (blockIdx.x + 1) / gridDim.x) - first) {}
    __device__ __forceinline__ int token(int i) const { return first + i; }
};

// The rows of the block's tokens, one after another in its lines, kAhead rows' loads in
// flight.
template <int LANES, Pairs PAIRS>
__global__ void __launch_bounds__(kNormThreads, 2) norm_walk_kernel(const __grid_constant__ NormParams p) {
    constexpr int LINES = kNormThreads / LANES;
    __shared__ __align__(16) Exchange<LANES, PAIRS> rows;
    dev::griddep_launch_dependents();
    const Columns<LANES, PAIRS> cols(p.plan, p.norm.head_dim);
    const Share mine(p.tokens);
    const int line = threadIdx.x / LANES;
    dev::griddep_wait();
    float w[16];
    cols.weight(p.norm.weight, p.norm.offset, w);
    for (int t0 = 0; t0 < mine.count; t0 += p.held) {
        const int count = min(p.held, mine.count - t0), all = count * p.heads;
        const TurnTable tab = {turn_smem, count * p.plan.pitch};
        Chunks v[kAhead];
        auto load = [&](int row) {
            const int j = fast_div(row, p.fd_heads);
            return cols.load(p.x + mine.token(t0 + j) * p.x_tok + (row - j * p.heads) * p.x_head);
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            v[k] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (line + k * LINES < all) v[k] = load(line + k * LINES);
        }
        if (t0 > 0) __syncthreads();  // (the last turns have been read)
        for (int e = threadIdx.x; e < count * p.plan.half; e += kNormThreads) {
            const int j = fast_div(e, p.plan.fd_half);
            fill_turn(p.plan, tab, e + j * (p.plan.pitch - p.plan.half), e - j * p.plan.half, p.positions[mine.token(t0 + j)]);
        }
        __syncthreads();
#pragma unroll 1
        for (int row0 = 0; row0 < all; row0 += kAhead * LINES) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int row = row0 + k * LINES + line, next = row + kAhead * LINES;
                float y[16];
                widen(v[k], y);
                if (next < all) v[k] = load(next);
                const int j = min(fast_div(row, p.fd_heads), count - 1);
                scale_row<LANES>(y, w, p.norm);
                Turns<LANES, PAIRS> turns;
                turns.load(p.plan, tab, j, cols);
                turns.apply(y, rows.row(line), cols);
                if (row < all) cols.store(p.out + mine.token(t0 + j) * p.o_tok + (row - j * p.heads) * p.o_head, y);
            }
        }
    }
}

template <int LANES, Pairs PAIRS>
__global__ void __launch_bounds__(kNormThreads, 2) norm_grad_kernel(const __grid_constant__ GradParams p) {
    constexpr int LINES = kNormThreads / LANES;
    __shared__ __align__(16) float rows[kNormThreads * 16];
    dev::griddep_launch_dependents();
    const Columns<LANES, PAIRS> cols(p.plan, p.norm.head_dim);
    const Share mine(p.tokens);
    const int line = threadIdx.x / LANES;
    dev::griddep_wait();
    float w[16], dw[16] = {};
    cols.weight(p.norm.weight, p.norm.offset, w);
    for (int t0 = 0; t0 < mine.count; t0 += p.held) {
        const int count = min(p.held, mine.count - t0), all = count * p.heads;
        const TurnTable tab = {turn_smem, count * p.plan.pitch};
        Chunks vx[kGradAhead], vg[kGradAhead];
        auto load = [&](int row, Chunks &x, Chunks &g) {
            const int j = fast_div(row, p.fd_heads), h = row - j * p.heads;
            x = cols.load(p.x + mine.token(t0 + j) * p.x_tok + h * p.x_head);
            g = cols.load(p.g + mine.token(t0 + j) * p.g_tok + h * p.g_head);
        };
#pragma unroll
        for (int k = 0; k < kGradAhead; ++k) {
            vx[k] = vg[k] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (line + k * LINES < all) load(line + k * LINES, vx[k], vg[k]);
        }
        if (t0 > 0) __syncthreads();  // (the last turns have been read)
        for (int e = threadIdx.x; e < count * p.plan.half; e += kNormThreads) {
            const int j = fast_div(e, p.plan.fd_half);
            fill_turn(p.plan, tab, e + j * (p.plan.pitch - p.plan.half), e - j * p.plan.half, p.positions[mine.token(t0 + j)]);
        }
        __syncthreads();
#pragma unroll 1
        for (int row0 = 0; row0 < all; row0 += kGradAhead * LINES) {
#pragma unroll
            for (int k = 0; k < kGradAhead; ++k) {
                const int row = row0 + k * LINES + line, next = row + kGradAhead * LINES;
                float x[16], u[16], xx = 0.f, xu = 0.f;
                widen(vx[k], x);
                widen(vg[k], u);
                if (next < all) load(next, vx[k], vg[k]);
                const int j = min(fast_div(row, p.fd_heads), count - 1);
                Turns<LANES, PAIRS> turns;
                turns.load(p.plan, tab, j, cols);
                turns.apply(u, rows + line * (LANES * 16), cols);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    xx = fmaf(x[i], x[i], xx);
                    xu = fmaf(x[i] * u[i], w[i], xu);
                }
                const float scale = rsqrtf(fmaf(row_sum<LANES>(xx), p.norm.inv_dim, p.norm.eps));
                const float back = row_sum<LANES>(xu) * p.norm.inv_dim * scale * scale;
                if (row < all) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        dw[i] = fmaf(u[i], x[i] * scale, dw[i]);
                        x[i] = scale * fmaf(-back, x[i], u[i] * w[i]);
                    }
                    cols.store(p.dx + mine.token(t0 + j) * p.d_tok + (row - j * p.heads) * p.d_head, x);
                }
            }
        }
    }
    if (!p.part) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(rows + threadIdx.x * 16 + i) = make_float4(dw[i], dw[i + 1], dw[i + 2], dw[i + 3]);
    __syncthreads();
    if (threadIdx.x < LANES * 16) {
        float sum = 0.f;
#pragma unroll 8
        for (int l = 0; l < LINES; ++l) sum += rows[l * (LANES * 16) + threadIdx.x];
        p.part[static_cast<long long>(blockIdx.x) * (LANES * 16) + threadIdx.x] = sum;
    }
}

// dw of 32 of the lanes' columns: 32 lines of threads sum the blocks' parts, every 32nd
// each, and the lines are summed in order.  halves: the first so many columns lie in the
// first chunks of as many lanes, as many more in their second ones (0: a lane's chunks are
// neighbours).
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float *part, int blocks, int pitch, int head_dim, int halves,
                                                                __nv_bfloat16 *dw) {
    __shared__ float sums[32][33];
    dev::griddep_launch_dependents();
    dev::griddep_wait();
    const int at = blockIdx.x * 32 + threadIdx.x;
    float sum = 0.f;
#pragma unroll 4
    for (int b = threadIdx.y; b < blocks; b += 32) sum += part[static_cast<long long>(b) * pitch + at];
    sums[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y > 0) return;
    for (int i = 1; i < 32; ++i) sum += sums[i][threadIdx.x];
    int col = at;
    if (at < 2 * halves) col = at / 16 * 8 + at % 8 + (at & 8 ? halves : 0);
    if (col < head_dim) dw[col] = __float2bfloat16_rn(sum);
}

// A row of an append on its way: queries to q_out, keys and values to the caches' cell.
template <int LANES, Pairs PAIRS, bool KV8>
__device__ __forceinline__ void append_row(const NormAppendParams &p, const Columns<LANES, PAIRS> &cols, const Turns<LANES, PAIRS> &turns,
                                           float *exchange, const float (&w)[16], const Chunks &v, int token, int h, int pos, int bid,
                                           bool in) {
    const int D = p.norm.head_dim, hk = h - p.q_heads, hv = hk - p.kv_heads, bs = static_cast<int>(p.block_size.d);
    float y[16];
    widen(v, y);
    scale_row<LANES>(y, w, p.norm);
    turns.apply(y, exchange, cols);
    if (!in || pos < 0) return;
    if (hk < 0) {
        cols.store(p.q_out + (static_cast<long long>(token) * p.q_heads + h) * D, y);
    } else if (bid >= 0) {
        const long long cell = (static_cast<long long>(bid) * bs + (pos - fast_div(pos, p.block_size) * bs)) * p.kv_heads;
        const long long to = (cell + (hv < 0 ? hk : hv)) * D;
        if (hv >= 0) widen(v, y);  // (values as they are)
        if constexpr (KV8) {
            uint8_t *o = static_cast<uint8_t *>(hv < 0 ? p.k_cache : p.v_cache) + to;
            const float f = hv < 0 ? p.k_scale : p.v_scale;
            if (cols.a) store_e4m3<8>(o + cols.ca, reinterpret_cast<const float(&)[8]>(y[0]), f);
            if (cols.b) store_e4m3<8>(o + cols.cb, reinterpret_cast<const float(&)[8]>(y[8]), f);
        } else {
            cols.store(static_cast<__nv_bfloat16 *>(hv < 0 ? p.k_cache : p.v_cache) + to, y);
        }
    }
}
template <int LANES, Pairs PAIRS>
__device__ __forceinline__ Chunks append_load(const NormAppendParams &p, const Columns<LANES, PAIRS> &cols, int token, int h) {
    const int D = p.norm.head_dim, hk = h - p.q_heads, hv = hk - p.kv_heads;
    return cols.load(hk < 0   ? p.q + token * p.q_tok + h * D
                     : hv < 0 ? p.k + token * p.k_tok + hk * D
                              : p.v + token * p.v_tok + hv * D);
}
// Both norms' weights in shared memory, a lane's columns side by side: by the first lines.
template <int LANES, Pairs PAIRS>
__device__ __forceinline__ void append_weights(const NormAppendParams &p, const Columns<LANES, PAIRS> &cols, float *weights) {
    const int line = threadIdx.x / LANES;
    if (line > 1) return;
    float w[16];
    cols.weight(line ? p.k_weight : p.norm.weight, p.norm.offset, w);
#pragma unroll
    for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4 *>(weights + line * (LANES * 16) + cols.u * 16 + i) = make_float4(w[i], w[i + 1], w[i + 2], w[i + 3]);
}

// One row a line: where rows are few.
template <int LANES, Pairs PAIRS, bool KV8>
__global__ void __launch_bounds__(kNormThreads, 4) norm_append_kernel(const __grid_constant__ NormAppendParams p) {
    __shared__ __align__(16) Exchange<LANES, PAIRS> exchange;
    __shared__ int place[kNormThreads / LANES + 2][2];  // of the block's tokens: position (-1: left out) and cache block (-1: none)
    dev::griddep_launch_dependents();
    const Place<LANES> at(p.plan, blockIdx.x, p.threads);
    const Columns<LANES, PAIRS> cols(p.plan, p.norm.head_dim);
    const int count = at.last - at.first + 1;
    const TurnTable tab = {turn_smem, count * p.plan.pitch};
    dev::griddep_wait();
    Chunks v = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (at.in) v = append_load(p, cols, at.tok, at.slot);
    float w[16];
    cols.weight(at.slot < p.q_heads ? p.norm.weight : p.k_weight, p.norm.offset, w);
    find_places(p, at.first, count, threadIdx.x & 31, place);
    __syncthreads();
    for (int e = threadIdx.x; e < count * p.plan.half; e += kNormThreads) {
        const int j = fast_div(e, p.plan.fd_half);
        fill_turn(p.plan, tab, e + j * (p.plan.pitch - p.plan.half), e - j * p.plan.half, place[j][0]);
    }
    __syncthreads();
    const int j = min(at.tok, at.last) - at.first;
    Turns<LANES, PAIRS> turns;
    turns.load(p.plan, tab, j, cols);
    append_row<LANES, PAIRS, KV8>(p, cols, turns, exchange.row(at.line), w, v, at.tok, at.slot, place[j][0], place[j][1], at.in);
}

// The rows of the block's tokens, one after another in its lines, as norm_walk_kernel.
constexpr int kPlaces = 256;  // tokens whose turns and places are held at most
static_assert(kNormThreads * 16 * 4 + 2 * 16 * 16 * 4 + kPlaces * 8 + kTableBytes <= 48 * 1024, "a walk's shared memory is what a block has unasked");
template <int LANES, Pairs PAIRS, bool KV8>
__global__ void __launch_bounds__(kNormThreads, 2) norm_append_walk_kernel(const __grid_constant__ NormAppendParams p) {
    constexpr int LINES = kNormThreads / LANES;
    __shared__ __align__(16) Exchange<LANES, PAIRS> exchange;
    __shared__ __align__(16) float weights[2 * LANES * 16];
    __shared__ int place[kPlaces][2];
    dev::griddep_launch_dependents();
    const Columns<LANES, PAIRS> cols(p.plan, p.norm.head_dim);
    const Share mine(p.tokens);
    const int line = threadIdx.x / LANES, rows = p.q_heads + 2 * p.kv_heads;
    dev::griddep_wait();
    append_weights(p, cols, weights);
    for (int t0 = 0; t0 < mine.count; t0 += p.held) {
        const int count = min(p.held, mine.count - t0), all = count * rows;
        const TurnTable tab = {turn_smem, count * p.plan.pitch};
        Chunks v[kAhead];
        auto load = [&](int row) {
            const int j = fast_div(row, p.fd_rows);
            return append_load(p, cols, mine.token(t0 + j), row - j * rows);
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            v[k] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (line + k * LINES < all) v[k] = load(line + k * LINES);
        }
        if (t0 > 0) __syncthreads();  // (the last turns and places have been read)
        find_places(p, mine.token(t0), count, threadIdx.x & 31, place);
        __syncthreads();
        for (int e = threadIdx.x; e < count * p.plan.half; e += kNormThreads) {
            const int j = fast_div(e, p.plan.fd_half);
            fill_turn(p.plan, tab, e + j * (p.plan.pitch - p.plan.half), e - j * p.plan.half, place[j][0]);
        }
        __syncthreads();
#pragma unroll 1
        for (int row0 = 0; row0 < all; row0 += kAhead * LINES) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int row = row0 + k * LINES + line, next = row + kAhead * LINES;
                const Chunks now = v[k];
                if (next < all) v[k] = load(next);
                const int j = min(fast_div(row, p.fd_rows), count - 1);
                Turns<LANES, PAIRS> turns;
                turns.load(p.plan, tab, j, cols);
                float w[16];
                const float *of = weights + (row - j * rows < p.q_heads ? 0 : LANES * 16) + cols.u * 16;
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(of + i);
                    w[i] = f.x, w[i + 1] = f.y, w[i + 2] = f.z, w[i + 3] = f.w;
                }
                append_row<LANES, PAIRS, KV8>(p, cols, turns, exchange.row(line), w, now, mine.token(t0 + j), row - j * rows, place[j][0], place[j][1],
                                              row < all);
            }
        }
    }
}

// ---- host side --------------------------------------------------------------------

int lanes_of(int head_dim) { return head_dim <= 64 ? 4 : (head_dim <= 128 ? 8 : 16); }

RowPlan plan_norm(const pd_rope *rope, int lanes, bool transposed) {
    RowPlan p = {};
    p.units = make_fastdiv(lanes);
    p.half = rope ? rope->rot_dim / 2 : 0;
    p.fd_half = make_fastdiv(p.half);
    p.pitch = (p.half + 3) / 4 * 4;
    p.turns = rope ? rope->turns : nullptr;
    p.factor = rope ? rope->factor : 1.f;
    p.sign = transposed ? -1.f : 1.f;
    return p;
}

Pairs pairs_of(const pd_rope *rope) {
    if (!rope || rope->layout == PD_ROPE_INTERLEAVED) return kNeighbours;
    return rope->rot_dim / 2 % 8 ? kScattered : kHalves;
}

// Whether `rows` rows of each of `tokens` tokens are many: more than eight times what the GPU's
// threads hold at a time; such are walked.
// (A launch has fewer than 2^31 rows, with those ahead of the last: too_many.)
bool too_many(int tokens, int rows) { return static_cast<long long>(tokens) * rows > 0x7fff0000LL; }
bool are_many(int tokens, int rows, int lanes) { return static_cast<long long>(tokens) * rows * lanes > 8ll * kStreams * 2048; }

// Else a line of lanes for each: the threads (false where they pass 31 bits, which rows
// that are not many do not).
void deal_rows(RowPlan *plan, int tokens, int rows, int *threads) {
    plan->slots = make_fastdiv(rows);
    *threads = tokens * rows * static_cast<int>(plan->units.d);
}

// Tokens whose turns a walk holds: the share of a block of `blocks`, or what there is room for.
int held_tokens(const RowPlan &plan, int tokens, int blocks, int most) {
    const int room = plan.pitch > 0 ? kTableBytes / (plan.pitch * 8) : most;
    return std::max(1, std::min({room, most, (tokens + blocks - 1) / blocks}));
}

template <class Params, class Kernel>
cudaError_t launch_walk(Kernel kern, const Params &p, int blocks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(kNormThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.held) * p.plan.pitch * 2 * sizeof(float);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// f(lanes, pairs) with both as compile-time constants.
template <class F>
cudaError_t by_shape(int lanes, Pairs pairs, F f) {
    auto with = [&](auto l) {
        if (pairs == kNeighbours) return f(l, std::integral_constant<Pairs, kNeighbours>());
        if (pairs == kHalves) return f(l, std::integral_constant<Pairs, kHalves>());
        return f(l, std::integral_constant<Pairs, kScattered>());
    };
    if (lanes == 4) return with(std::integral_constant<int, 4>());
    if (lanes == 8) return with(std::integral_constant<int, 8>());
    return with(std::integral_constant<int, 16>());
}

int check_norm(const char *what, const pd_rope *rope, int head_dim, const void *w0, const void *w1, float eps, float offset) {
    if (head_dim < 8 || head_dim > PD_MAX_HEAD_DIM || head_dim % 8)
        return report(PD_ERR_UNSUPPORTED, "%s: head_dim %d must be a multiple of 8 in [8, %d]", what, head_dim, PD_MAX_HEAD_DIM);
    if (!std::isfinite(eps) || eps < 0) return report(PD_ERR_INVALID, "%s: eps must be finite and not negative", what);
    if (!std::isfinite(offset)) return report(PD_ERR_INVALID, "%s: weight_offset is not finite", what);
    if (!aligned16(w0) || !aligned16(w1)) return report(PD_ERR_INVALID, "%s: weights must be 16-byte aligned", what);
    if (!rope) return PD_OK;
    if (rope->head_dim != head_dim)
        return report(PD_ERR_INVALID, "%s: head_dim %d, the rotation's is %d", what, head_dim, rope->head_dim);
    return check_handle(what, rope);
}

// Strides that hold 16-byte rows; rows: those of a tensor that is written do not overlap.
int check_strides(const char *what, const char *name, int64_t tok, int64_t head, int64_t T, int64_t H, int64_t D, bool written) {
    if (tok <= 0 || tok % 8 || head <= 0 || head % 8)
        return report(PD_ERR_INVALID, "%s: %s's strides must be positive multiples of 8 elements (got %lld and %lld)", what, name,
                      static_cast<long long>(tok), static_cast<long long>(head));
    if (!written) return PD_OK;
    const bool by_token = (H == 1 || head >= D) && (T == 1 || (tok >= D && (tok - D) / head >= H - 1));
    const bool by_head = (T == 1 || tok >= D) && (H == 1 || (head >= D && (head - D) / tok >= T - 1));
    if (by_token || by_head) return PD_OK;
    return report(PD_ERR_INVALID, "%s: rows of %s overlap (strides %lld and %lld, %lld tokens of %lld heads)", what, name,
                  static_cast<long long>(tok), static_cast<long long>(head), static_cast<long long>(T), static_cast<long long>(H));
}

Norm norm_of(const void *weight, float offset, float eps, int head_dim) {
    return {static_cast<const __nv_bfloat16 *>(weight), weight ? offset : 0.f, eps, 1.f / static_cast<float>(head_dim), head_dim};
}

int append_impl(const char *what, const pd_rope *rope, const void *q, int64_t q_tok, const void *k, int64_t k_tok, const void *v,
                int64_t v_tok, const void *q_weight, const void *k_weight, float eps, float offset, void *q_out, void *k_cache,
                void *v_cache, bool kv8, float k_scale, float v_scale, const int32_t *block_table, int max_blocks,
                const int32_t *context_lens, const int32_t *token_starts, int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads,
                int head_dim, int block_size, int num_blocks, void *stream) {
    int rc = check_norm(what, nullptr, head_dim, q_weight, k_weight, eps, offset);
    if (rc != PD_OK) return rc;
    rc = check_append(what, rope, q, q_tok, k, k_tok, v, v_tok, q_out, k_cache, v_cache, kv8, k_scale, v_scale, block_table, max_blocks,
                      context_lens, num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                      token_starts != nullptr);
    if (rc != PD_OK || num_tokens == 0 || num_seqs == 0) return rc;
    int err = PD_OK;
    NormAppendParams p = {};
    p.status = device_status_word(&err);
    if (!p.status) return err;
    const int lanes = lanes_of(head_dim);
    p.plan = plan_norm(rope, lanes, false);
    p.norm = norm_of(q_weight, offset, eps, head_dim);
    p.norm.offset = offset;  // (of k's weight, too)
    p.k_weight = static_cast<const __nv_bfloat16 *>(k_weight);
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
    p.block_size = make_fastdiv(block_size);
    const int rows = p.q_heads + 2 * num_kv_heads, blocks = std::min(2 * kStreams, num_tokens);
    if (too_many(num_tokens, rows)) return report(PD_ERR_INVALID, "%s: launch too large (%d tokens)", what, num_tokens);
    const bool many = are_many(num_tokens, rows, lanes);
    if (!many) deal_rows(&p.plan, num_tokens, rows, &p.threads);
    p.fd_rows = make_fastdiv(rows);
    p.tokens = num_tokens;
    p.held = held_tokens(p.plan, num_tokens, blocks, kPlaces);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = by_shape(lanes, pairs_of(rope), [&](auto l, auto pairs) {
        constexpr int L = decltype(l)::value;
        constexpr Pairs P = decltype(pairs)::value;
        if (kv8)
            return many ? launch_walk(norm_append_walk_kernel<L, P, true>, p, blocks, st) : launch_rows(norm_append_kernel<L, P, true>, p, st);
        return many ? launch_walk(norm_append_walk_kernel<L, P, false>, p, blocks, st) : launch_rows(norm_append_kernel<L, P, false>, p, st);
    });
    if (e != cudaSuccess) return report_cuda(e, what);
    return report_ok();
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" {

int pd_norm_rope_apply(const pd_rope *rope, const void *x, int64_t x_token_stride, int64_t x_head_stride, const void *weight, float eps,
                       float weight_offset, const int32_t *positions, void *out, int64_t out_token_stride, int64_t out_head_stride,
                       int num_tokens, int num_heads, int head_dim, void *stream) {
    const char *what = "pd_norm_rope_apply";
    if (num_tokens < 0 || num_heads < 0) return report(PD_ERR_INVALID, "%s: num_tokens %d, num_heads %d", what, num_tokens, num_heads);
    int rc = check_norm(what, rope, head_dim, weight, nullptr, eps, weight_offset);
    if (rc != PD_OK) return rc;
    if (num_tokens == 0 || num_heads == 0) return report_ok();
    if (!x || !out || (rope && !positions)) return report(PD_ERR_INVALID, "%s: null tensor pointer", what);
    if (!aligned16(x) || !aligned16(out)) return report(PD_ERR_INVALID, "%s: x and out must be 16-byte aligned", what);
    rc = check_strides(what, "x", x_token_stride, x_head_stride, num_tokens, num_heads, head_dim, false);
    if (rc == PD_OK) rc = check_strides(what, "out", out_token_stride, out_head_stride, num_tokens, num_heads, head_dim, true);
    if (rc != PD_OK) return rc;
    if (x == out && (x_token_stride != out_token_stride || x_head_stride != out_head_stride))
        return report(PD_ERR_INVALID, "%s: in place (out == x) needs equal strides", what);
    NormParams p = {};
    const int lanes = lanes_of(head_dim);
    p.plan = plan_norm(rope, lanes, false);
    p.norm = norm_of(weight, weight_offset, eps, head_dim);
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.x_tok = x_token_stride;
    p.x_head = x_head_stride;
    p.o_tok = out_token_stride;
    p.o_head = out_head_stride;
    p.positions = positions;
    p.heads = num_heads;
    const int blocks = std::min(2 * kStreams, num_tokens);
    if (too_many(num_tokens, num_heads))
        return report(PD_ERR_INVALID, "%s: launch too large (%d tokens of %d heads)", what, num_tokens, num_heads);
    const bool many = are_many(num_tokens, num_heads, lanes);
    if (!many) deal_rows(&p.plan, num_tokens, num_heads, &p.threads);
    p.fd_heads = make_fastdiv(num_heads);
    p.tokens = num_tokens;
    p.held = held_tokens(p.plan, num_tokens, blocks, 256);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = by_shape(lanes, pairs_of(rope), [&](auto l, auto pairs) {
        constexpr int L = decltype(l)::value;
        constexpr Pairs P = decltype(pairs)::value;
        return many ? launch_walk(norm_walk_kernel<L, P>, p, blocks, st) : launch_rows(norm_kernel<L, P>, p, st);
    });
    if (e != cudaSuccess) return report_cuda(e, what);
    return report_ok();
}

size_t pd_norm_rope_workspace_bytes(int head_dim) {
    if (head_dim <= 0 || head_dim > PD_MAX_HEAD_DIM) return 0;
    return static_cast<size_t>(2 * kStreams) * lanes_of(head_dim) * 16 * sizeof(float);
}

int pd_norm_rope_backward(const pd_rope *rope, const void *x, int64_t x_token_stride, int64_t x_head_stride, const void *weight, float eps,
                          float weight_offset, const int32_t *positions, const void *grad, int64_t grad_token_stride,
                          int64_t grad_head_stride, void *grad_x, int64_t grad_x_token_stride, int64_t grad_x_head_stride,
                          void *grad_weight, int num_tokens, int num_heads, int head_dim, void *workspace, size_t workspace_bytes,
                          void *stream) {
    const char *what = "pd_norm_rope_backward";
    if (num_tokens < 0 || num_heads < 0) return report(PD_ERR_INVALID, "%s: num_tokens %d, num_heads %d", what, num_tokens, num_heads);
    int rc = check_norm(what, rope, head_dim, weight, nullptr, eps, weight_offset);
    if (rc != PD_OK) return rc;
    if (grad_weight && !weight) return report(PD_ERR_INVALID, "%s: a weight's gradient without a weight", what);
    const bool none = num_tokens == 0 || num_heads == 0;
    if (none && !grad_weight) return report_ok();
    if (!none && (!x || !grad || !grad_x || (rope && !positions))) return report(PD_ERR_INVALID, "%s: null tensor pointer", what);
    if (!aligned16(x) || !aligned16(grad) || !aligned16(grad_x))
        return report(PD_ERR_INVALID, "%s: x, grad and grad_x must be 16-byte aligned", what);
    const int lanes = lanes_of(head_dim);
    if (grad_weight && (!workspace || workspace_bytes < pd_norm_rope_workspace_bytes(head_dim)))
        return report(PD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given%s", what, pd_norm_rope_workspace_bytes(head_dim),
                      workspace ? workspace_bytes : static_cast<size_t>(0), workspace ? "" : " (null)");
    if (!aligned16(workspace)) return report(PD_ERR_INVALID, "workspace must be 16-byte aligned");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int blocks = 0;
    if (!none) {
        rc = check_strides(what, "x", x_token_stride, x_head_stride, num_tokens, num_heads, head_dim, false);
        if (rc == PD_OK) rc = check_strides(what, "grad", grad_token_stride, grad_head_stride, num_tokens, num_heads, head_dim, false);
        if (rc == PD_OK) rc = check_strides(what, "grad_x", grad_x_token_stride, grad_x_head_stride, num_tokens, num_heads, head_dim, true);
        if (rc != PD_OK) return rc;
        if (too_many(num_tokens, num_heads))
            return report(PD_ERR_INVALID, "%s: launch too large (%d tokens of %d heads)", what, num_tokens, num_heads);
        GradParams p = {};
        p.plan = plan_norm(rope, lanes, true);
        p.norm = norm_of(weight, weight_offset, eps, head_dim);
        p.x = static_cast<const __nv_bfloat16 *>(x);
        p.g = static_cast<const __nv_bfloat16 *>(grad);
        p.dx = static_cast<__nv_bfloat16 *>(grad_x);
        p.x_tok = x_token_stride;
        p.x_head = x_head_stride;
        p.g_tok = grad_token_stride;
        p.g_head = grad_head_stride;
        p.d_tok = grad_x_token_stride;
        p.d_head = grad_x_head_stride;
        p.positions = positions;
        p.heads = num_heads;
        p.part = grad_weight ? static_cast<float *>(workspace) : nullptr;
        p.fd_heads = make_fastdiv(num_heads);
        p.tokens = num_tokens;
        blocks = std::min(2 * kStreams, num_tokens);
        p.held = held_tokens(p.plan, num_tokens, blocks, 256);
        const cudaError_t e = by_shape(lanes, pairs_of(rope), [&](auto l, auto pairs) {
            return launch_walk(norm_grad_kernel<decltype(l)::value, decltype(pairs)::value>, p, blocks, st);
        });
        if (e != cudaSuccess) return report_cuda(e, what);
    }
    if (grad_weight) {
        const Pairs pairs = pairs_of(rope);
        const int halves = pairs == kHalves ? rope->rot_dim / 2 : (pairs == kNeighbours ? (head_dim + 8) / 16 * 8 : 0);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(lanes * 16 / 32));
        cfg.blockDim = dim3(32, 32);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_weight_grad_kernel, static_cast<const float *>(workspace), blocks, lanes * 16,
                                                 head_dim, halves, static_cast<__nv_bfloat16 *>(grad_weight));
        if (e != cudaSuccess) return report_cuda(e, what);
    }
    return report_ok();
}

int pd_append_kv_normed(const pd_rope *rope, const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride, const void *v,
                        int64_t v_token_stride, const void *q_weight, const void *k_weight, float eps, float weight_offset, void *q_out,
                        void *k_cache, void *v_cache, const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens,
                        const int32_t *token_starts, int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                        int block_size, int num_blocks, void *stream) {
    return append_impl("pd_append_kv_normed", rope, q, q_token_stride, k, k_token_stride, v, v_token_stride, q_weight, k_weight, eps,
                       weight_offset, q_out, k_cache, v_cache, false, 1.f, 1.f, block_table, max_blocks_per_seq, context_lens, token_starts,
                       num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, stream);
}

int pd_append_kv_normed_fp8(const pd_rope *rope, const void *q, int64_t q_token_stride, const void *k, int64_t k_token_stride,
                            const void *v, int64_t v_token_stride, const void *q_weight, const void *k_weight, float eps,
                            float weight_offset, void *q_out, void *k_cache, void *v_cache, float k_scale, float v_scale,
                            const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens,
                            const int32_t *token_starts, int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                            int block_size, int num_blocks, void *stream) {
    return append_impl("pd_append_kv_normed_fp8", rope, q, q_token_stride, k, k_token_stride, v, v_token_stride, q_weight, k_weight, eps,
                       weight_offset, q_out, k_cache, v_cache, true, k_scale, v_scale, block_table, max_blocks_per_seq, context_lens,
                       token_starts, num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, stream);
}

}  // extern "C"
