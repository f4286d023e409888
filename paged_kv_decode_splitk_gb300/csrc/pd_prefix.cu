// pd_prefix.cu -- pd_decode_attn_prefix[_fp8]: decode attention of a batch whose
// sequences share prefixes.  Host side and the merge; the prefix pass is
// pd_prefix.cuh, the pass over the sequences' own tokens the unit kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>
#include <vector>

#include "pd.h"
#include "pd_device.cuh"
#include "pd_internal.h"
#include "pd_prefix_plan.h"

namespace pd {
namespace prefix {
namespace {

static_assert(kMaxGroups == PD_MAX_PREFIX_GROUPS, "pd.h");

constexpr int kOwnUnits = 152 * 8;  // units of the own-token pass that are enough
constexpr int kMergeWarps = 8;
constexpr int kMergeBatch = 4;   // partials whose o are loaded together

// DPAD / 8 lanes per (sequence, query head), 8 columns each, fold the row's
// partials: first those of its prefix, in the order of the teams that made them
// (both CTAs' where they took the tiles in turn), then its own splits.  With M the
// largest reference and w_i = 2^(m_i - M),
//   out = sum_i w_i o_i / sum_i w_i l_i,
// 0 where the row has no token at all.  Bound by latency on small batches (the
// chain is the plan, then m, l and o together) and by reading the partials from
// L2 on large ones; three blocks fit an SM, so that a batch of 8192 rows is little
// more than a wave.  Fewer rows have several lines of lanes each, which
// share the partials.
template <int DPAD>
__global__ void __launch_bounds__(kMergeWarps * 32, 3) prefix_merge_kernel(const __grid_constant__ MergeParams p) {
    constexpr int LPR = DPAD / 8, RPW = 32 / LPR;  // lanes of a row, rows of a warp
    constexpr int BR = block_rows(DPAD);
    const float kNegInf = -__int_as_float(0x7f800000);
    dev::griddep_launch_dependents();
    __shared__ float fold[kMergeWarps * 32][9];   // ways > 1: each thread's columns
    __shared__ float2 fold_ml[kMergeWarps * RPW];
    const int lane = threadIdx.x & 31, sub = lane % LPR, mine = lane / LPR, head_lane = mine * LPR;
    const int line = threadIdx.x / LPR, ways = p.ways, way = line & (ways - 1);  // a row has `ways` lines of lanes
    const int D = p.head_dim, N = p.num_splits, rows = p.num_seqs * p.num_q_heads;
    const int row = blockIdx.x * (kMergeWarps * RPW / ways) + line / ways;
    const int d0 = sub * 8;
    const bool in = row < rows, cols = in && d0 < D;
    const int s = in ? fast_div(row, p.fd_hq) : 0;
    const int h = row - s * p.num_q_heads;
    const int kvh = in ? fast_div(h, p.fd_group) : 0;
    dev::griddep_wait();

    // ---- the row's group: the last one that begins at or before the sequence ----
    int L = in ? p.context_lens[s] : 0;
    const PlanTotal plan = *p.plan_total;
    const long long W = plan.units;
    GroupPlan g = {};
    for (int g0 = 0; g0 < p.num_groups; g0 += 32) {
        GroupPlan one = {};
        if (g0 + lane < p.num_groups) one = p.plan_groups[g0 + lane];
        int below = 0;
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
            const int sr = __shfl_sync(0xffffffffu, s, r * LPR);
            const unsigned b = __ballot_sync(0xffffffffu, g0 + lane < p.num_groups && one.first_seq <= sr);
            if (mine == r) below = __popc(b);
        }
        const int src = below > 0 ? below - 1 : 0;
        GroupPlan f;
        f.first_unit = __shfl_sync(0xffffffffu, one.first_unit, src);
        f.first_item = __shfl_sync(0xffffffffu, one.first_item, src);
        f.tiles = __shfl_sync(0xffffffffu, one.tiles, src);
        f.first_seq = __shfl_sync(0xffffffffu, one.first_seq, src);
        f.rows = __shfl_sync(0xffffffffu, one.rows, src);
        f.items = __shfl_sync(0xffffffffu, one.items, src);
        f.first_team = __shfl_sync(0xffffffffu, one.first_team, src);
        f.teams = __shfl_sync(0xffffffffu, one.teams, src);
        f.last_teams = __shfl_sync(0xffffffffu, one.last_teams, src);
        if (below > 0) g = f;
    }
    RowParts of = {0, 2, 0};
    const int x = (s - g.first_seq) * p.group + (h - kvh * p.group);
    if (const bool has = W > 0 && in && g.tiles > 0 && x < g.rows; __any_sync(0xffffffffu, has)) {
        const RowPlace at = place_of<DPAD>(g, kvh, has ? x : 0);
        int c0, c1;
        if (plan.whole) {
            whole_teams_of(g, kvh, at.item, c0, c1);
        } else {
            const int c = has ? team_of_unit(sub == 0 ? at.u0 : at.u1, plan.teams, W) : 0;
            c0 = __shfl_sync(0xffffffffu, c, head_lane), c1 = __shfl_sync(0xffffffffu, c, head_lane + 1);
        }
        if (has) of = parts_of<DPAD>(g, kvh, at, c0, c1);
    }
    const int nparts = of.parts, step = of.step;
    const long long first = of.first;  // (slot, row) of its first partial
    L = L < 0 ? 0 : (L > p.max_tokens ? p.max_tokens : L);
    const int chunk = split_chunk_tokens_fd(L, p.fd_split, p.fd_bs, p.min_kv_per_split);
    // (this line's share: partials way, way + ways, ...)
    const int all = nparts + (L > 0 ? (L + chunk - 1) / chunk : 0);
    const int total = all > way ? (all - way + ways - 1) / ways : 0;

    // where partial i of the share lies: (m, l) and, for this lane's columns, o
    auto ml_of = [&](int k) -> const float * {
        const int i = way + k * ways;
        if (i >= nparts) return p.own_ml + (static_cast<long long>(row) * N + (i - nparts)) * 2;
        return p.part_ml + (first + i * step * BR) * 2;
    };
    // (chunk k of a row of 32 columns lies at k xor the row's number mod 8: this
    // lane's two chunks are in one sector, in turned order for odd rows)
    const int prow = static_cast<int>(first % BR), flip = prow & 7;
    const float *part = p.part_o + ((first / BR * (DPAD / 32) + d0 / 32) * BR + prow) * 32;
    const int lo = ((d0 % 32 / 4) ^ flip) * 4, hi = ((d0 % 32 / 4 + 1) ^ flip) * 4;
    // ---- the fold, LPR partials at a time: lane i of the row has (m, l) of partial i ----
    int most = total;  // (all rows of a warp go through the loops together)
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
    float M = kNegInf, lsum = 0.f;
    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    for (int i0 = 0; i0 < most; i0 += LPR) {
        float2 v = make_float2(kNegInf, 0.f);
        if (i0 + sub < total) v = *reinterpret_cast<const float2 *>(ml_of(i0 + sub));
        float4 o[kMergeBatch][2];
        auto ask = [&](int j0) {
#pragma unroll
            for (int j = 0; j < kMergeBatch; ++j) {
                o[j][0] = o[j][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (cols && i0 + j0 + j < total) {
                    const int i = way + (i0 + j0 + j) * ways;
                    const bool of_prefix = i < nparts;
                    const float *at = of_prefix ? part + static_cast<long long>(i) * step * (DPAD * BR)
                                                : p.own_o + (static_cast<long long>(row) * N + (i - nparts)) * D + d0;
                    o[j][0] = *reinterpret_cast<const float4 *>(at + (of_prefix ? lo : 0));
                    o[j][1] = *reinterpret_cast<const float4 *>(at + (of_prefix ? hi : 4));
                }
            }
        };
        ask(0);  // (together with m and l)
        // a partial without a token has l = 0, and its o was not written
        const bool dead = v.y == 0.f;
        float top = dead ? kNegInf : v.x;
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float Mn = fmaxf(M, top);
        const float keep = M == kNegInf ? 0.f : dev::exp2_approx(M - Mn);
        M = Mn;
        const float w = dead ? 0.f : dev::exp2_approx(v.x - M);
        float wl = dead ? 0.f : w * v.y;
        const float wo = way + (i0 + sub) * ways < nparts ? w * p.v_scale : w;
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, off);
        lsum = lsum * keep + wl;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= keep;
        for (int j0 = 0; j0 < min(LPR, most - i0); j0 += kMergeBatch) {
            if (j0 > 0) ask(j0);
#pragma unroll
            for (int j = 0; j < kMergeBatch; ++j) {
                const int src = head_lane + ((j0 + j) & (LPR - 1));
                const float wj = __shfl_sync(0xffffffffu, wo, src);
                const bool skip = __shfl_sync(0xffffffffu, dead, src);
                if (i0 + j0 + j < total && !skip) {
                    acc[0] = fmaf(o[j][0].x, wj, acc[0]);
                    acc[1] = fmaf(o[j][0].y, wj, acc[1]);
                    acc[2] = fmaf(o[j][0].z, wj, acc[2]);
                    acc[3] = fmaf(o[j][0].w, wj, acc[3]);
                    acc[4] = fmaf(o[j][1].x, wj, acc[4]);
                    acc[5] = fmaf(o[j][1].y, wj, acc[5]);
                    acc[6] = fmaf(o[j][1].z, wj, acc[6]);
                    acc[7] = fmaf(o[j][1].w, wj, acc[7]);
                }
            }
        }
    }
    if (ways > 1) {
        // the lines of a row, folded in order by its first
        if (sub == 0) fold_ml[line] = make_float2(M, lsum);
#pragma unroll
        for (int k = 0; k < 8; ++k) fold[threadIdx.x][k] = acc[k];
        __syncthreads();
        if (way > 0) return;
        float Mall = M;
        for (int k = 1; k < ways; ++k) Mall = fmaxf(Mall, fold_ml[line + k].x);
        const float f0 = M == kNegInf ? 0.f : dev::exp2_approx(M - Mall);
        lsum *= f0;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] *= f0;
        for (int w = 1; w < ways; ++w) {
            const float2 ml = fold_ml[line + w];
            const float f = ml.x == kNegInf ? 0.f : dev::exp2_approx(ml.x - Mall);
            lsum = fmaf(ml.y, f, lsum);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = fmaf(fold[threadIdx.x + w * LPR][k], f, acc[k]);
        }
    }
    if (!cols) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = lsum == 0.f ? 0.f : __fdiv_rn(acc[k], lsum);
    *reinterpret_cast<uint4 *>(p.out + static_cast<long long>(row) * D + d0) =
        make_uint4(dev::pack_bf16x2(acc[0], acc[1]), dev::pack_bf16x2(acc[2], acc[3]), dev::pack_bf16x2(acc[4], acc[5]),
                   dev::pack_bf16x2(acc[6], acc[7]));
}

cudaError_t launch_prefix_merge(const MergeParams &p, cudaStream_t stream) {
    const int rows = p.num_seqs * p.num_q_heads, of_block = kMergeWarps * (256 / p.dpad) / p.ways;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows + of_block - 1) / of_block));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.dpad == 64) return cudaLaunchKernelEx(&cfg, prefix_merge_kernel<64>, p);
    if (p.dpad == 128) return cudaLaunchKernelEx(&cfg, prefix_merge_kernel<128>, p);
    return cudaLaunchKernelEx(&cfg, prefix_merge_kernel<256>, p);
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
                  (num_groups + static_cast<long long>(num_seqs) * (num_q_heads / num_kv_heads) / item_rows(dpad_of(head_dim)));
    const size_t slots = 2 * (static_cast<size_t>(l.max_items) + kMaxTeams);
    l.own_o = take(rows * head_dim * sizeof(float));
    l.own_ml = take(rows * 2 * sizeof(float));
    l.plan_total = take(sizeof(PlanTotal));
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
    p.context_lens = context_lens;
    p.max_own_tokens = max_blocks * block_size;
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
    // A scale of 0 becomes the smallest above it: a masked score, -infinity, then
    // still weighs 0, and every other still (all but) nothing against its reference.
    p.scale_log2 = std::max(static_cast<float>(std::fabs(scale)), FLT_MIN);
    p.negative = scale < 0;
    p.max_items = static_cast<int>(lay.max_items);
    p.part_ml = reinterpret_cast<float *>(ws + lay.part_ml);
    p.part_o = reinterpret_cast<float *>(ws + lay.part_o);
    p.plan_groups = reinterpret_cast<GroupPlan *>(ws + lay.plan_groups);
    p.plan_total = reinterpret_cast<PlanTotal *>(ws + lay.plan_total);
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
    // as many lines a row as one wave has room for, 8 at most (a third more, into a
    // second wave: 64 sequences behind 8192 tokens 41.2 -> 44.6 us)
    const long long lanes = static_cast<long long>(num_seqs) * num_q_heads * (dpad / 8);
    m.ways = 1;
    while (m.ways < 8 && 2 * m.ways * lanes <= 152 * 3 * kMergeWarps * 32) m.ways *= 2;
    m.num_splits = num_splits;
    m.min_kv_per_split = PD_MIN_KV_PER_SPLIT;
    m.max_tokens = max_blocks * block_size;
    m.v_scale = kv8 ? v_scale : 1.f;
    m.fd_hq = make_fastdiv(num_q_heads);
    m.fd_group = make_fastdiv(group);
    m.fd_split = make_fastdiv(num_splits);
    m.fd_bs = make_fastdiv(block_size);
    e = launch_prefix_merge(m, st);
    if (e != cudaSuccess) return report_cuda(e, "prefix merge launch");
    return report_ok();
}

// The division of a call's work as the prefix pass and the merge work it out.
template <int DPAD, bool KV8>
int walk(int num_seqs, int num_groups, const int32_t *group_starts, const int32_t *prefix_lens, int group, int num_kv_heads, float own_us,
         int most, int32_t *segments, int max_segments, int *num_segments, int64_t *parts, int32_t *totals) {
    constexpr int IR = item_rows(DPAD);
    std::vector<GroupPlan> grp(num_groups);
    long long W = 0;
    int items = 0;
    float time = 0.f;
    for (int g = 0; g < num_groups; ++g) {
        const int a = group_starts[g], b = group_starts[g + 1];
        if (a < 0 || b < a || b > num_seqs || prefix_lens[g] < 0 || prefix_lens[g] > 0x7fffffff - 256)
            return report(PD_ERR_INVALID, "pd_debug_prefix_walk: group %d", g);
        GroupPlan r = plan_of<DPAD>(a, (b - a) * group, prefix_lens[g]);
        r.first_unit = W;
        r.first_item = items;
        if (r.tiles > 0 && r.items > 0) {
            const long long units = r.head_units(IR) * num_kv_heads;
            W += units;
            items += r.items * num_kv_heads;
            time += units * unit_time<DPAD, KV8>(std::min(r.rows, IR));
        }
        grp[g] = r;
    }
    int C = 0, run = 0;
    if (W > 0 && num_groups == 1) {
        C = share_units(W, items, grp[0].last_units(IR) == quotient(W, items), time, own_us, most);
    } else if (W > 0) {
        C = share_units(W, items, false, time, own_us, most);
        WholeTry t;
        if (try_whole(num_groups, W, C, most, items, t)) {
            int lane = 0;
            while (lane < 32 && teams_in_all(grp.data(), num_groups, num_kv_heads, IR, t.run(lane)) > t.limit) ++lane;
            if (lane < 32 && whole_pays(t, t.run(lane), quick_quotient(time, static_cast<float>(W)), KV8 ? 6.f : 3.f)) {
                run = t.run(lane);
                C = teams_in_all(grp.data(), num_groups, num_kv_heads, IR, run);
            }
        }
    }
    int n = 0;
    for (int team = 0; team < C; ++team)
        for (int rank = 0; rank < 2; ++rank) {
            long long u = 0, u1 = 0;
            if (run > 0)
                whole_range(grp.data(), num_kv_heads, IR, run, team, u, u1);
            else
                line_range(W, C, team, u, u1);
            Segment s;
            while (next_segment<block_rows(DPAD)>(grp.data(), num_groups, u, u1, team, rank, s)) {
                if (n == max_segments) return report(PD_ERR_CAPACITY, "pd_debug_prefix_walk: more than %d segments", n);
                const int32_t v[10] = {team, rank, s.group, s.kvh, s.row0, s.rows, s.tile0, s.stride, s.n, s.slot};
                std::copy(v, v + 10, segments + 10ll * n++);
            }
        }
    *num_segments = n;
    // the merge's side: of each group, KV head and row
    for (int g = 0; g < num_groups; ++g) {
        GroupPlan r = grp[g];
        if (num_groups > 1) plan_whole(grp.data(), g, num_kv_heads, IR, run, r);
        for (int kvh = 0; kvh < num_kv_heads; ++kvh)
            for (int x = 0; x < r.rows; ++x, parts += 3) {
                RowParts v = {0, 2, 0};
                if (W > 0 && r.tiles > 0) {
                    const RowPlace at = place_of<DPAD>(r, kvh, x);
                    int c0, c1;
                    if (run > 0) {
                        whole_teams_of(r, kvh, at.item, c0, c1);
                    } else {
                        c0 = team_of_unit(at.u0, C, W);
                        c1 = team_of_unit(at.u1, C, W);
                    }
                    v = parts_of<DPAD>(r, kvh, at, c0, c1);
                }
                parts[0] = v.parts;
                parts[1] = v.step;
                parts[2] = v.first;
            }
    }
    totals[0] = C;
    totals[1] = run;
    totals[2] = block_rows(DPAD);
    totals[3] = tile_tokens(DPAD);
    return report_ok();
}

}  // namespace
}  // namespace prefix
}  // namespace pd

extern "C" {

int pd_debug_prefix_walk(int num_seqs, int num_groups, const int32_t *group_starts, const int32_t *prefix_lens, int num_q_heads,
                         int num_kv_heads, int head_dim, int fp8, float own_us, int max_teams, int32_t *segments,
                         int max_segments, int *num_segments, int64_t *parts, int32_t *totals) {
    using namespace pd::prefix;
    const int rc = pd::check_shape(num_q_heads, num_kv_heads, head_dim, 16);
    if (rc != PD_OK) return rc;
    if (num_seqs < 0 || num_groups < 1 || num_groups > kMaxGroups || max_teams < 1 || max_teams > kMaxTeams || max_segments < 0 ||
        static_cast<long long>(num_seqs) * num_q_heads > 0x7fffffffLL - 256 || !group_starts || !prefix_lens || !segments ||
        !num_segments || !parts || !totals)
        return pd::report(PD_ERR_INVALID, "pd_debug_prefix_walk: an argument is out of range or null");
    const int dpad = dpad_of(head_dim);
    try {
        const auto f = dpad == 64 ? (fp8 ? walk<64, true> : walk<64, false>) : dpad == 128 ? (fp8 ? walk<128, true> : walk<128, false>)
                                                                                           : (fp8 ? walk<256, true> : walk<256, false>);
        return f(num_seqs, num_groups, group_starts, prefix_lens, num_q_heads / num_kv_heads, num_kv_heads, own_us, max_teams, segments,
                 max_segments, num_segments, parts, totals);
    } catch (...) {  // (nothing but the host's memory can run out)
        return pd::report(PD_ERR_ALLOC, "pd_debug_prefix_walk: out of host memory");
    }
}

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
