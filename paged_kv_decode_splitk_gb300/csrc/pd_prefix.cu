// pd_prefix.cu -- pd_decode_attn_prefix[_fp8]: decode attention of a batch whose
// sequences share prefixes.  Host side and the merge; the prefix pass is
// pd_prefix.cuh, the pass over the sequences' own tokens the unit kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "pd.h"
#include "pd_device.cuh"
#include "pd_internal.h"
#include "pd_prefix.h"

namespace pd {
namespace prefix {
namespace {

static_assert(kMaxGroups == PD_MAX_PREFIX_GROUPS, "pd.h");

constexpr int kOwnUnits = 152 * 8;  // units of the own-token pass that are enough
constexpr int kMergeWarps = 8;
constexpr int kMergeCols = 128;  // columns of a row one warp merges (4 per lane)
constexpr int kMergeBatch = 8;   // partials whose o are loaded together

// The team whose range [W c / C, W (c + 1) / C) holds unit u.
__device__ __forceinline__ int team_of_unit(long long u, int C, long long W) {
    const long long num = (u + 1) * C - 1;
    if (num < 0x7fffffffLL)
        return static_cast<int>(static_cast<unsigned>(num) / static_cast<unsigned>(W));
    return static_cast<int>(num / W);
}

// One warp per (sequence, query head, 128 columns) folds the row's partials:
// first those of its prefix, in the order of the teams that made them (both
// CTAs' where they took the tiles in turn), then its own splits.
// With M the largest reference and w_i = 2^(m_i - M),
//   out = sum_i w_i o_i / sum_i w_i l_i,
// 0 where the row has no token at all.  Bound by latency on small batches (the
// chain: group, plan, (m, l), o) and by reading the partials from L2 on large.
__global__ void __launch_bounds__(kMergeWarps * 32) prefix_merge_kernel(const __grid_constant__ MergeParams p) {
    const float kNegInf = -__int_as_float(0x7f800000);
    dev::griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = p.head_dim, N = p.num_splits;
    const int BR = block_rows(p.dpad);
    const int chunks = D > kMergeCols ? 2 : 1;
    const long long item_id = static_cast<long long>(blockIdx.x) * kMergeWarps + warp;
    if (item_id >= static_cast<long long>(p.num_seqs) * p.num_q_heads * chunks) return;
    const long long row = item_id >> (chunks - 1);
    const int d0 = static_cast<int>(item_id - row * chunks) * kMergeCols + lane * 4;
    const bool cols = d0 < D;
    const int s = fast_div(static_cast<int>(row), p.fd_hq);
    const int h = static_cast<int>(row - static_cast<long long>(s) * p.num_q_heads);
    const int kvh = fast_div(h, p.fd_group);
    dev::griddep_wait();

    // ---- the row's group: the last one that begins at or before the sequence ----
    int L = p.context_lens[s];
    const long long W = *p.plan_total;
    GroupPlan g = {};
    for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
        GroupPlan mine = {};
        if (g0 + lane < p.num_groups) mine = p.plan_groups[g0 + lane];
        const int below = __popc(__ballot_sync(0xffffffffu, g0 + lane < p.num_groups && mine.first_seq <= s));
        if (below == 0) break;
        const int src = below - 1;
        g.first_unit = __shfl_sync(0xffffffffu, mine.first_unit, src);
        g.first_item = __shfl_sync(0xffffffffu, mine.first_item, src);
        g.tiles = __shfl_sync(0xffffffffu, mine.tiles, src);
        g.first_seq = __shfl_sync(0xffffffffu, mine.first_seq, src);
        g.rows = __shfl_sync(0xffffffffu, mine.rows, src);
        g.blocks = __shfl_sync(0xffffffffu, mine.blocks, src);
    }
    int nparts = 0, step = 2;      // prefix slots of the row, 2 apart, or (both CTAs') 1
    long long first = 0;           // (slot, row) of its first partial
    if (W > 0) {
        const int x = (s - g.first_seq) * p.group + (h - kvh * p.group);
        if (g.tiles > 0 && x < g.rows) {
            const int block = x / BR, r = x - block * BR;
            const int pairs = g.blocks >> 1, odd = g.blocks & 1, of_single = (g.tiles + 1) >> 1;
            const bool pair = block < 2 * pairs;
            const int item = block >> 1, places = pair ? g.tiles : of_single;
            const long long u = g.first_unit + kvh * (static_cast<long long>(pairs) * g.tiles + (odd ? of_single : 0)) +
                                static_cast<long long>(item) * g.tiles;
            const int C = teams_of(W, p.teams);
            const int c = team_of_unit(lane == 0 ? u : u + places - 1, C, W);
            const int c0 = __shfl_sync(0xffffffffu, c, 0), c1 = __shfl_sync(0xffffffffu, c, 1);
            step = pair ? 2 : 1;
            nparts = (c1 - c0 + 1) * (pair ? 1 : 2);
            const long long slot = 2ll * (g.first_item + kvh * (pairs + odd) + item + c0) + (pair ? block & 1 : 0);
            first = slot * BR + r;
        }
    }
    L = L < 0 ? 0 : (L > p.max_tokens ? p.max_tokens : L);
    const int chunk = split_chunk_tokens_fd(L, p.fd_split, p.fd_bs, p.min_kv_per_split);
    const int own = L > 0 ? (L + chunk - 1) / chunk : 0;
    const int total = nparts + own;

    // where partial i lies: (m, l) and, for this lane's columns, o
    auto ml_of = [&](int i) -> const float * {
        if (i >= nparts) return p.own_ml + (row * N + (i - nparts)) * 2;
        return p.part_ml + (first + static_cast<long long>(i * step) * BR) * 2;
    };
    auto o_of = [&](int i) -> const float * {
        if (i >= nparts) return p.own_o + (row * N + (i - nparts)) * D + d0;
        const long long at = first + static_cast<long long>(i * step) * BR;
        const long long sl = at / BR, r = at - sl * BR;
        return p.part_o + ((sl * (p.dpad / 8) + d0 / 8) * BR + r) * 8 + (d0 & 4);
    };

    // ---- the fold, 32 partials at a time: lane i has (m, l) of partial i ----
    float M = kNegInf, lsum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < total; i0 += 32) {
        const int n = min(32, total - i0);
        float2 v = make_float2(kNegInf, 0.f);
        if (lane < n) v = *reinterpret_cast<const float2 *>(ml_of(i0 + lane));
        float4 o[kMergeBatch];
#pragma unroll
        for (int j = 0; j < kMergeBatch; ++j)  // (asked for together with m and l)
            o[j] = cols && j < n ? *reinterpret_cast<const float4 *>(o_of(i0 + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
        // a partial without a token has l = 0, and its o was not written
        const bool dead = v.y == 0.f;
        float top = dead ? kNegInf : v.x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float Mn = fmaxf(M, top);
        const float keep = M == kNegInf ? 0.f : dev::exp2_approx(M - Mn);
        M = Mn;
        const float w = dead ? 0.f : dev::exp2_approx(v.x - M);
        float wl = dead ? 0.f : w * v.y;
        const float wo = i0 + lane < nparts ? w * p.v_scale : w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, off);
        lsum = lsum * keep + wl;
        acc.x *= keep;
        acc.y *= keep;
        acc.z *= keep;
        acc.w *= keep;
        for (int j0 = 0; j0 < n; j0 += kMergeBatch) {
            if (j0 > 0) {
#pragma unroll
                for (int j = 0; j < kMergeBatch; ++j)
                    o[j] = cols && j0 + j < n ? *reinterpret_cast<const float4 *>(o_of(i0 + j0 + j)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < kMergeBatch; ++j) {
                const float wj = __shfl_sync(0xffffffffu, wo, (j0 + j) & 31);
                const bool skip = __shfl_sync(0xffffffffu, dead, (j0 + j) & 31);
                if (j0 + j < n && !skip) {
                    acc.x = fmaf(o[j].x, wj, acc.x);
                    acc.y = fmaf(o[j].y, wj, acc.y);
                    acc.z = fmaf(o[j].z, wj, acc.z);
                    acc.w = fmaf(o[j].w, wj, acc.w);
                }
            }
        }
    }
    if (!cols) return;
    const bool none = lsum == 0.f;
    uint2 pk;
    pk.x = dev::pack_bf16x2(none ? 0.f : __fdiv_rn(acc.x, lsum), none ? 0.f : __fdiv_rn(acc.y, lsum));
    pk.y = dev::pack_bf16x2(none ? 0.f : __fdiv_rn(acc.z, lsum), none ? 0.f : __fdiv_rn(acc.w, lsum));
    *reinterpret_cast<uint2 *>(p.out + row * D + d0) = pk;
}

cudaError_t launch_prefix_merge(const MergeParams &p, cudaStream_t stream) {
    const long long items = static_cast<long long>(p.num_seqs) * p.num_q_heads * (p.head_dim > kMergeCols ? 2 : 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((items + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefix_merge_kernel, p);
}

int sm_count_of_device() {
    static std::mutex mu;
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (!cached[dev] && cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        cached[dev] = 0;
    }
    return cached[dev];
}

int dpad_of(int head_dim) { return head_dim <= 64 ? 64 : (head_dim <= 128 ? 128 : 256); }

// Where the parts of the workspace begin, in bytes (each a multiple of 256).
struct Layout {
    size_t own_o, own_ml, plan_total, plan_groups, part_ml, part_o, end;
    long long max_items;
};

Layout layout_of(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int head_dim, int num_splits) {
    Layout l = {};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const int BR = block_rows(dpad_of(head_dim));
    const size_t rows = static_cast<size_t>(num_seqs) * num_q_heads * num_splits;
    // every group's rows end in at most one item that is not full
    l.max_items = static_cast<long long>(num_kv_heads) *
                  (num_groups + static_cast<long long>(num_seqs) * (num_q_heads / num_kv_heads) / (2 * BR));
    const size_t slots = 2 * (static_cast<size_t>(l.max_items) + kMaxTeams);
    l.own_o = take(rows * head_dim * sizeof(float));
    l.own_ml = take(rows * 2 * sizeof(float));
    l.plan_total = take(sizeof(long long));
    l.plan_groups = take(sizeof(GroupPlan) * kMaxGroups);
    l.part_ml = take(slots * BR * 2 * sizeof(float));
    l.part_o = take(slots * BR * dpad_of(head_dim) * sizeof(float));
    l.end = at;
    return l;
}

template <bool KV8>
cudaError_t dispatch_prefix(int dpad, const CUtensorMap *tk, const CUtensorMap *tv, const PrefixParams &p, int teams,
                            cudaStream_t st) {
    if (dpad == 64) return launch_prefix<64, KV8>(tk, tv, p, teams, st);
    if (dpad == 128) return launch_prefix<128, KV8>(tk, tv, p, teams, st);
    return launch_prefix<256, KV8>(tk, tv, p, teams, st);
}

int decode_prefix_impl(const char *what, const void *q, const void *k_cache, const void *v_cache, bool kv8, float k_scale,
                       float v_scale, const int32_t *prefix_table, int max_prefix_blocks, const int32_t *prefix_lens,
                       const int32_t *group_starts, int num_groups, const int32_t *block_table, int max_blocks,
                       const int32_t *context_lens, void *out, int num_seqs, int num_q_heads, int num_kv_heads,
                       int head_dim, int block_size, int num_blocks, float inv_sqrt_d, int num_splits, void *workspace,
                       size_t workspace_bytes, void *stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size);
    if (rc != PD_OK) return rc;
    if (num_groups < 1 || num_groups > kMaxGroups)
        return report(PD_ERR_INVALID, "%s: num_groups %d outside 1..%d", what, num_groups, kMaxGroups);
    if (!group_starts && num_groups != 1)
        return report(PD_ERR_INVALID, "%s: without group_starts the batch is one group (num_groups %d)", what, num_groups);
    if (num_seqs < 0) return report(PD_ERR_INVALID, "num_seqs %d < 0", num_seqs);
    if (num_splits < 1 || num_splits > PD_MAX_DECODE_SPLITS)
        return report(PD_ERR_INVALID, "%s: num_splits %d outside 1..%d", what, num_splits, PD_MAX_DECODE_SPLITS);
    if (num_seqs == 0) return report_ok();
    if (!prefix_table || !prefix_lens) return report(PD_ERR_INVALID, "%s: null prefix table or lengths", what);
    if (max_prefix_blocks <= 0)
        return report(PD_ERR_INVALID, "%s: max_prefix_blocks %d must be positive", what, max_prefix_blocks);
    if (static_cast<long long>(max_prefix_blocks) * block_size > 0x7fffffffLL - 256)
        return report(PD_ERR_INVALID, "%s: max_prefix_blocks * block_size overflows int32", what);
    if (static_cast<long long>(num_seqs) * num_q_heads > 0x7fffffffLL - 256)
        return report(PD_ERR_INVALID, "%s: launch too large (%d sequences)", what, num_seqs);
    // num_splits is the most the own tokens are cut into.  A split has at least
    // PD_MIN_KV_PER_SPLIT tokens, so a table holds no more than `fit` of them; and
    // once units fill the GPU several times, more only add partials to fold.
    const int fit = (max_blocks * static_cast<long long>(block_size) + PD_MIN_KV_PER_SPLIT - 1) / PD_MIN_KV_PER_SPLIT;
    const long long units = static_cast<long long>(num_seqs) * num_kv_heads;
    const long long fill = (kOwnUnits + units - 1) / units;
    num_splits = static_cast<int>(std::max(1ll, std::min(static_cast<long long>(num_splits), std::min<long long>(fit, fill))));
    const Layout lay = layout_of(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, num_splits);
    if (lay.max_items > 0x3fffffffLL - kMaxTeams) return report(PD_ERR_INVALID, "%s: launch too large", what);
    if (!workspace || workspace_bytes < lay.end)
        return report(PD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given%s", what, lay.end,
                      workspace ? workspace_bytes : static_cast<size_t>(0), workspace ? "" : " (null)");
    if (!aligned16(workspace)) return report(PD_ERR_INVALID, "workspace must be 16-byte aligned");
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *own_o = reinterpret_cast<float *>(ws + lay.own_o);
    float *own_ml = reinterpret_cast<float *>(ws + lay.own_ml);

    KvView view;
    view.box_tokens = 16;  // as many as divide a block and a tile: fewer, larger boxes
    while (view.box_tokens < tile_tokens(dpad_of(head_dim)) && block_size % (2 * view.box_tokens) == 0) view.box_tokens *= 2;
    auto own_pass = [&](float *o, float *ml) {
        return launch_own_partials(q, k_cache, v_cache, block_table, max_blocks, context_lens, out, num_seqs, num_q_heads,
                                   num_kv_heads, head_dim, block_size, num_blocks, inv_sqrt_d, num_splits, o, ml, stream, kv8,
                                   k_scale, v_scale, &view);
    };
    rc = own_pass(nullptr, nullptr);  // every argument is checked before anything is launched
    if (rc != PD_OK) return rc;

    int err = PD_OK;
    PrefixParams p = {};
    p.status = device_status_word(&err);
    if (!p.status) return err;
    const int sms = sm_count_of_device();
    const int teams = sms < 2 ? 1 : std::min(sms / 2, kMaxTeams);
    const int group = num_q_heads / num_kv_heads;
    const double scale = static_cast<double>(inv_sqrt_d) * (kv8 ? static_cast<double>(k_scale) : 1.0) * 1.4426950408889634;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.prefix_table = prefix_table;
    p.prefix_lens = prefix_lens;
    p.group_starts = group_starts;
    p.num_groups = num_groups;
    p.max_prefix_blocks = max_prefix_blocks;
    p.num_blocks = num_blocks;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.head_dim = head_dim;
    p.block_size = make_fastdiv(block_size);
    p.fd_group = make_fastdiv(group);
    p.tok_dim = view.tok_dim;
    p.box_tokens = view.box_tokens;
    p.scale_log2 = static_cast<float>(std::fabs(scale));
    p.negative = scale < 0;
    p.max_items = static_cast<int>(lay.max_items);
    p.part_ml = reinterpret_cast<float *>(ws + lay.part_ml);
    p.part_o = reinterpret_cast<float *>(ws + lay.part_o);
    p.plan_groups = reinterpret_cast<GroupPlan *>(ws + lay.plan_groups);
    p.plan_total = reinterpret_cast<long long *>(ws + lay.plan_total);
    const int dpad = dpad_of(head_dim);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = kv8 ? dispatch_prefix<true>(dpad, &view.k, &view.v, p, teams, st)
                        : dispatch_prefix<false>(dpad, &view.k, &view.v, p, teams, st);
    if (e != cudaSuccess) return report_cuda(e, "prefix pass launch");
    // Beside it, the sequences' own tokens: the prefix pass is bound by its
    // products where rows are many, this one by memory.
    rc = own_pass(own_o, own_ml);
    if (rc != PD_OK) return rc;

    MergeParams m = {};
    m.plan_groups = p.plan_groups;
    m.plan_total = p.plan_total;
    m.part_ml = p.part_ml;
    m.part_o = p.part_o;
    m.own_o = own_o;
    m.own_ml = own_ml;
    m.context_lens = context_lens;
    m.out = static_cast<__nv_bfloat16 *>(out);
    m.num_groups = num_groups;
    m.num_seqs = num_seqs;
    m.num_q_heads = num_q_heads;
    m.num_kv_heads = num_kv_heads;
    m.group = group;
    m.head_dim = head_dim;
    m.dpad = dpad;
    m.num_splits = num_splits;
    m.min_kv_per_split = PD_MIN_KV_PER_SPLIT;
    m.max_tokens = max_blocks * block_size;
    m.teams = teams;
    m.v_scale = kv8 ? v_scale : 1.f;
    m.fd_hq = make_fastdiv(num_q_heads);
    m.fd_group = make_fastdiv(group);
    m.fd_split = make_fastdiv(num_splits);
    m.fd_bs = make_fastdiv(block_size);
    e = launch_prefix_merge(m, st);
    if (e != cudaSuccess) return report_cuda(e, "prefix merge launch");
    return report_ok();
}

}  // namespace
}  // namespace prefix
}  // namespace pd

extern "C" {

size_t pd_prefix_workspace_bytes(int num_seqs, int num_groups, int num_q_heads, int num_kv_heads, int head_dim,
                                 int num_splits) {
    if (num_seqs <= 0 || num_groups <= 0 || num_kv_heads <= 0 || num_q_heads < num_kv_heads ||
        num_q_heads % num_kv_heads || head_dim <= 0 || num_splits <= 0)
        return 0;
    return pd::prefix::layout_of(num_seqs, num_groups, num_q_heads, num_kv_heads, head_dim, num_splits).end;
}

int pd_decode_attn_prefix(const void *q, const void *k_cache, const void *v_cache, const int32_t *prefix_table,
                          int max_prefix_blocks, const int32_t *prefix_lens, const int32_t *group_starts, int num_groups,
                          const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens, void *out,
                          int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                          float inv_sqrt_d, int num_splits, void *workspace, size_t workspace_bytes, void *stream) {
    return pd::prefix::decode_prefix_impl("pd_decode_attn_prefix", q, k_cache, v_cache, false, 1.f, 1.f, prefix_table,
                                          max_prefix_blocks, prefix_lens, group_starts, num_groups, block_table,
                                          max_blocks_per_seq, context_lens, out, num_seqs, num_q_heads, num_kv_heads,
                                          head_dim, block_size, num_blocks, inv_sqrt_d, num_splits, workspace,
                                          workspace_bytes, stream);
}

int pd_decode_attn_prefix_fp8(const void *q, const void *k_cache, const void *v_cache, float k_scale, float v_scale,
                              const int32_t *prefix_table, int max_prefix_blocks, const int32_t *prefix_lens,
                              const int32_t *group_starts, int num_groups, const int32_t *block_table,
                              int max_blocks_per_seq, const int32_t *context_lens, void *out, int num_seqs, int num_q_heads,
                              int num_kv_heads, int head_dim, int block_size, int num_blocks, float inv_sqrt_d,
                              int num_splits, void *workspace, size_t workspace_bytes, void *stream) {
    return pd::prefix::decode_prefix_impl("pd_decode_attn_prefix_fp8", q, k_cache, v_cache, true, k_scale, v_scale,
                                          prefix_table, max_prefix_blocks, prefix_lens, group_starts, num_groups, block_table,
                                          max_blocks_per_seq, context_lens, out, num_seqs, num_q_heads, num_kv_heads,
                                          head_dim, block_size, num_blocks, inv_sqrt_d, num_splits, workspace,
                                          workspace_bytes, stream);
}

}  // extern "C"
