// pd_rope.cuh -- what the rotary positions (pd_rope.cu) and the head norms with the
// rotation (pd_norm.cu) share: the handle, the table of a block's sines and cosines,
// the places of new tokens in the paged cache, and the launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>

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
namespace rope {

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
inline int block_tokens(int per) { return (kRopeThreads - 2) / per + 2; }

__device__ __forceinline__ void fill_turn(const RowPlan &p, const TurnTable &tab, int at, int pair, int position) {
    const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(position)) * p.turns[pair];
    // x half-turns: the upper 32 bits, signed, over 2^31
    const float x = static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(x, &s, &c);
    tab.c[at] = c * p.factor;
    tab.c[tab.span + at] = s * (p.factor * p.sign);
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

// Where the tokens first to first + count - 1 go, a lane for each: place[j] is the
// position (-1: left out) and the cache block (-1: none).
template <class Params>
__device__ __forceinline__ void find_places(const Params &p, int first, int count, int lane, int (*place)[2]) {
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

inline int check_handle(const char *what, const pd_rope *rope) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return report_cuda(e, what);
    if (dev != rope->device)
        return report(PD_ERR_INVALID, "%s: the rotation was created on device %d, the current device is %d", what,
                      rope->device, dev);
    return PD_OK;
}

// The checks of an append's arguments; PD_OK with no tokens or sequences: there is
// nothing to do.
inline int check_append(const char *what, const pd_rope *rope, const void *q, int64_t q_tok, const void *k, int64_t k_tok, const void *v,
                        int64_t v_tok, const void *q_out, const void *k_cache, const void *v_cache, bool kv8, float k_scale,
                        float v_scale, const int32_t *block_table, int max_blocks, const int32_t *context_lens, int num_tokens,
                        int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, bool starts) {
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
    if (!starts && num_tokens != num_seqs)
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
    return report_ok();
}

}  // namespace rope
}  // namespace pd
