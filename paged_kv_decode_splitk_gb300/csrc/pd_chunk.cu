// pd_chunk.cu -- pd_chunk_attn[_fp8]: attention of new tokens over the paged cache
// that holds them.  Host side, and the fold of the items that several CTAs had; the
// pass itself is pd_chunk.cuh.
//
// The fold is a launch of its own behind the pass, one block for every CTA and few rows: a
// cut item has as many partials as CTAs had a part, and most calls cut about one item a
// CTA.  It is bound by latency (what it reads is below 1 MB for 64 single tokens of 32 heads).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>

#include "pd.h"
#include "pd_chunk.h"
#include "pd_device.cuh"
#include "pd_internal.h"

namespace pd {
namespace chunk {
namespace {

constexpr int kFoldThreads = 256;
constexpr int kFoldBatch = 4;  // partials whose o are loaded together

// Block (c, y) folds rows of the item that CTA c began and did not end: its part in
// slot 2 c + 1, the others in slots 2 (c + i), i = 1, 2, ...  DPAD / 8 threads a row, 8
// columns each, a warp 8 rows x 4 of them (128 bytes of a partial, 64 of a result); with M the largest reference and w_i = 2^(m_i - M),
//   out = sum_i w_i o_i / sum_i w_i l_i,   lse = ln 2 (M + log2 sum_i w_i l_i).
// Where rows are few, several lines of lanes share a row's partials.  Bound by
// latency: the item, then m, l and o together.
template <int DPAD>
__global__ void __launch_bounds__(kFoldThreads) fold_kernel(const __grid_constant__ FoldParams p) {
    constexpr int LPR = DPAD / 8, LINES = kFoldThreads / LPR;
    const float kNegInf = -__int_as_float(0x7f800000);
    __shared__ float fold[kFoldThreads][9];  // ways > 1: each thread's columns
    __shared__ float2 fold_ml[LINES];
    dev::griddep_launch_dependents();
    dev::griddep_wait();
    const CutItem it = p.cut[blockIdx.x];
    const int rows = min(it.tokens * p.item_heads - static_cast<int>(blockIdx.y) * LINES, LINES);
    if (it.parts == 0 || rows <= 0) return;
    int of_row = 1;  // rows a block takes at once: a power of two
    while (of_row < rows) of_row *= 2;
    const int octet = threadIdx.x / 32 / (LPR / 4), quad = threadIdx.x / 32 % (LPR / 4);
    const int line = octet * 8 + threadIdx.x % 8, chunk = quad * 4 + threadIdx.x / 8 % 4, me = line * LPR + chunk;
    const int ways = LINES / of_row, way = line / of_row;
    const int row = blockIdx.y * LINES + line % of_row, d0 = chunk * 8;
    const int k = fast_div(row, p.fd_heads), h = row - k * p.item_heads, step = partial_rows(it.tokens * p.item_heads);
    const bool in = row < p.slot_rows && k < it.tokens && h < it.heads;
    float M = kNegInf, l = 0.f, acc[8] = {};
    for (int i0 = way; in && i0 < it.parts; i0 += ways * kFoldBatch) {
        float2 ml[kFoldBatch];
        float4 o[kFoldBatch][2];
#pragma unroll
        for (int j = 0; j < kFoldBatch; ++j) {
            const int i = i0 + j * ways;
            ml[j] = make_float2(kNegInf, 0.f);
            if (i < it.parts) {
                const long long slot = (2ll * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * p.slot_rows;
                const float *of = p.part_o + slot * DPAD + (d0 * step + row * 4);
                ml[j] = *reinterpret_cast<const float2 *>(p.part_ml + (slot + row) * 2);
                o[j][0] = *reinterpret_cast<const float4 *>(of);
                o[j][1] = *reinterpret_cast<const float4 *>(of + 4 * step);
            }
        }
        float top = M;  // (a partial without a key has l = 0)
#pragma unroll
        for (int j = 0; j < kFoldBatch; ++j)
            if (ml[j].y != 0.f) top = fmaxf(top, ml[j].x);
        const float keep = M == kNegInf ? 0.f : dev::exp2_approx(M - top);
        M = top;
        l *= keep;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] *= keep;
#pragma unroll
        for (int j = 0; j < kFoldBatch; ++j) {
            if (ml[j].y == 0.f) continue;
            const float w = dev::exp2_approx(ml[j].x - M);
            l = fmaf(w, ml[j].y, l);
            const float v[8] = {o[j][0].x, o[j][0].y, o[j][0].z, o[j][0].w, o[j][1].x, o[j][1].y, o[j][1].z, o[j][1].w};
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] = fmaf(w, v[c], acc[c]);
        }
    }
    if (ways > 1) {  // the lines of a row, folded in order by its first
        if (d0 == 0) fold_ml[line] = make_float2(M, l);
#pragma unroll
        for (int c = 0; c < 8; ++c) fold[me][c] = acc[c];
        __syncthreads();
        if (way > 0) return;
        float top = M;
        for (int w = 1; w < ways; ++w) top = fmaxf(top, fold_ml[line + w * of_row].x);
        const float keep = M == kNegInf ? 0.f : dev::exp2_approx(M - top);
        M = top;
        l *= keep;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] *= keep;
        for (int w = 1; w < ways; ++w) {
            const float2 ml = fold_ml[line + w * of_row];
            const float f = ml.x == kNegInf ? 0.f : dev::exp2_approx(ml.x - M);
            l = fmaf(ml.y, f, l);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] = fmaf(fold[me + w * of_row * LPR][c], f, acc[c]);
        }
    }
    if (!in) return;
    const long long at = static_cast<long long>(it.token + k) * p.num_q_heads + it.head + h;
    if (p.lse && d0 == 0) p.lse[at] = l == 0.f ? kNegInf : (M + log2f(l)) * 0.6931471805599453f;
    if (d0 >= p.head_dim) return;
    const float f = l == 0.f ? 0.f : __fdiv_rn(p.v_scale, l);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = f == 0.f ? 0.f : acc[c] * f;
    *reinterpret_cast<uint4 *>(p.out + at * p.head_dim + d0) =
        make_uint4(dev::pack_bf16x2(acc[0], acc[1]), dev::pack_bf16x2(acc[2], acc[3]), dev::pack_bf16x2(acc[4], acc[5]),
                   dev::pack_bf16x2(acc[6], acc[7]));
}

cudaError_t launch_fold(const FoldParams &p, int dpad, int ctas, cudaStream_t stream) {
    const int lines = kFoldThreads / (dpad / 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>((p.slot_rows + lines - 1) / lines));
    cfg.blockDim = dim3(kFoldThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (dpad == 64) return cudaLaunchKernelEx(&cfg, fold_kernel<64>, p);
    if (dpad == 128) return cudaLaunchKernelEx(&cfg, fold_kernel<128>, p);
    return cudaLaunchKernelEx(&cfg, fold_kernel<256>, p);
}

int dpad_of(int head_dim) { return head_dim <= 64 ? 64 : (head_dim <= 128 ? 128 : 256); }

// Where the parts of the workspace begin, in bytes (each a multiple of 256).
struct Layout {
    size_t cut, part_ml, part_o, end;
    int slot_rows;
};

Layout layout_of(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim) {
    const int dpad = dpad_of(head_dim);
    const Shape s = make_shape(num_q_heads, num_kv_heads, dpad, 0);
    Layout l = {};
    l.slot_rows = (std::min(s.block_tokens, num_tokens) * s.item_heads + 31) / 32 * 32;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const size_t rows = 2ull * kMaxCtas * l.slot_rows;
    l.cut = take(kMaxCtas * sizeof(CutItem));
    l.part_ml = take(rows * 2 * sizeof(float));
    l.part_o = take(rows * dpad * sizeof(float));
    l.end = at;
    return l;
}

// Single tokens alone, without a window or their sums' logarithms, are what
// pd_decode_attn computes, by units of a few heads and keys instead of a product's rows.
// It takes them over FP8 (16 behind 1024 tokens 27.3 us here, 15.3 there; 64 behind 4096
// 166 and 96; 200 behind 700 160 and 65), and over BF16 for at most four query heads a KV
// head, here and there (us):
//                        1 x 500    16 x 1024  16 x 8192  64 x 300   64 x 4096  200 x 700
//   16 over 16 of 64    12.2  7.6  22.8 25.1  131  141   37.1 20.2  247  191   138  101
//   16 over 8 of 128    13.0 10.1  18.8 14.4  91.5 82.6  27.8 14.5  172  154   102  92.9
//   32 over 8 of 128    12.8  9.8  18.6 15.0  92.1 83.2  28.8 14.6  172  156   103  94.0
//   16 over 4 of 256    14.1 12.0  19.1 15.0  92.4 95.4  23.3 25.0  172  198   101  93.7
// (it loses a little to the pass at some of the last and first head dims' sizes).  With 16
// heads a KV head products have rows enough for the pass to be the faster one in most places,
// with 8 in half of them at head dims of 64 and 256, but with 5 to 8 at 128 in none of these:
// such calls could be given away too.
//   40 over 8 of 128    12.8 10.1  18.7 15.3  91.8 83.9  28.8 14.7  173  155   103  94.6
//   64 over 8 of 128    12.9  9.9  18.7 15.9  92.0 84.6  28.7 15.0  173  157   105  98.4
//   32 over 4 of 128    12.8  9.7  15.4 15.0  51.4 46.1  19.1 16.5  93.7 85.5  58.3 58.3
//   32 over 4 of 64     10.8  8.0  12.8 10.0  32.8 40.5  16.2 17.7  69.8 78.5  43.9 34.0
//   16 over 2 of 256    13.3 12.9  15.2 18.1  52.3 54.2  16.5 20.9  93.7 110   57.4 48.8
//   32 over 2 of 128    11.6 10.8  14.4 16.1  31.8 37.6  14.0 20.4  53.6 79.2  36.8 31.1
bool tokens_alone(int group, bool kv8) { return kv8 ? group <= 16 : group <= 4; }

// Its splits: as many as give every multiprocessor four of a sequence's KV heads, no more
// than two for each multiprocessor and query head (as the Auto rule for one sequence: 1
// behind 8192 tokens takes 15.4 us with 10 and 17.5 with 16, over FP8 behind 32768 21.4 and
// 28.6), and no more than the workspace holds.
int token_splits(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, size_t workspace_bytes) {
    const long long units = static_cast<long long>(num_seqs) * num_kv_heads;
    const int most = std::max(1, std::min(PD_SPLITK_TARGET_WAVES * kMaxCtas / num_q_heads, PD_MAX_DECODE_SPLITS));
    int n = static_cast<int>(std::min<long long>(std::max<long long>(4 * kMaxCtas / units, 1), most));
    while (n > 1 && pd_workspace_bytes(num_seqs, num_q_heads, head_dim, n) > workspace_bytes) n /= 2;
    return n;
}

template <bool KV8>
cudaError_t dispatch(int dpad, const CUtensorMap *tk, const CUtensorMap *tv, const CUtensorMap *tq, const ChunkParams &p, int ctas,
                     cudaStream_t st) {
    if (dpad == 64) return launch_chunk<64, KV8>(tk, tv, tq, p, ctas, st);
    if (dpad == 128) return launch_chunk<128, KV8>(tk, tv, tq, p, ctas, st);
    return launch_chunk<256, KV8>(tk, tv, tq, p, ctas, st);
}

int chunk_impl(const char *what, const void *q, int64_t q_tok, const void *k_cache, const void *v_cache, bool kv8, float k_scale,
               float v_scale, const int32_t *block_table, int max_blocks, const int32_t *context_lens, const int32_t *token_starts,
               void *out, float *lse, int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
               int num_blocks, float inv_sqrt_d, int window, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_shape(num_q_heads, num_kv_heads, head_dim, block_size);
    if (rc != PD_OK) return rc;
    if (num_tokens < 0 || num_seqs < 0)
        return report(PD_ERR_INVALID, "%s: num_tokens %d, num_seqs %d", what, num_tokens, num_seqs);
    if (!token_starts && num_tokens != num_seqs)
        return report(PD_ERR_INVALID, "%s: without token_starts every sequence has one token (num_tokens %d, num_seqs %d)", what,
                      num_tokens, num_seqs);
    if (window < 0) return report(PD_ERR_INVALID, "%s: window %d < 0", what, window);
    if (num_tokens == 0 || num_seqs == 0) return report_ok();
    if (q && (q_tok % 8 || q_tok < static_cast<int64_t>(num_q_heads) * head_dim))
        return report(PD_ERR_INVALID, "%s: q's token stride %lld must be a multiple of 8 elements and hold a token's rows", what,
                      static_cast<long long>(q_tok));
    if (static_cast<long long>(max_blocks) * block_size > 0x7fffffffLL - 256)
        return report(PD_ERR_INVALID, "%s: max_blocks_per_seq * block_size overflows int32", what);
    if (num_tokens > 0x7fffffff - 256) return report(PD_ERR_INVALID, "%s: launch too large (%d tokens)", what, num_tokens);
    const Layout lay = layout_of(num_tokens, num_q_heads, num_kv_heads, head_dim);
    if (!workspace || workspace_bytes < lay.end)
        return report(PD_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given%s", what, lay.end,
                      workspace ? workspace_bytes : static_cast<size_t>(0), workspace ? "" : " (null)");
    if (!aligned16(workspace)) return report(PD_ERR_INVALID, "workspace must be 16-byte aligned");
    uint8_t *ws = static_cast<uint8_t *>(workspace);

    const double scale = static_cast<double>(inv_sqrt_d) * (kv8 ? static_cast<double>(k_scale) : 1.0) * 1.4426950408889634;
    if (!token_starts && !lse && (window == 0 || window >= static_cast<long long>(max_blocks) * block_size) && scale >= FLT_MIN &&
        q_tok == static_cast<int64_t>(num_q_heads) * head_dim && tokens_alone(num_q_heads / num_kv_heads, kv8)) {
        const int splits = token_splits(num_seqs, num_q_heads, num_kv_heads, head_dim, workspace_bytes);
        return kv8 ? pd_decode_attn_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, max_blocks, context_lens, out, num_seqs,
                                        num_q_heads, num_kv_heads, head_dim, block_size, num_blocks, inv_sqrt_d, splits, workspace,
                                        workspace_bytes, PD_GQA_PACK_OFF, stream)
                   : pd_decode_attn(q, k_cache, v_cache, block_table, max_blocks, context_lens, out, num_seqs, num_q_heads, num_kv_heads,
                                    head_dim, block_size, num_blocks, inv_sqrt_d, splits, workspace, workspace_bytes, PD_GQA_PACK_OFF,
                                    stream);
    }
    const int dpad = dpad_of(head_dim);
    KvView view;
    view.box_tokens = 16;  // as many as divide a block and a tile: fewer, larger boxes
    while (view.box_tokens < tile_tokens(dpad) && block_size % (2 * view.box_tokens) == 0) view.box_tokens *= 2;
    // (pd_decode_attn's checks, and the caches' maps)
    rc = launch_own_partials(q, k_cache, v_cache, block_table, max_blocks, context_lens, out, num_seqs, num_q_heads, num_kv_heads,
                             head_dim, block_size, num_blocks, inv_sqrt_d, 1, nullptr, nullptr, stream, kv8, k_scale, v_scale, &view);
    if (rc != PD_OK) return rc;

    int err = PD_OK;
    ChunkParams p = {};
    p.status = device_status_word(&err);
    if (!p.status) return err;
    p.max_tokens = max_blocks * block_size;
    // (a window no table can fill is none)
    p.shape = make_shape(num_q_heads, num_kv_heads, dpad, window < p.max_tokens ? window : 0);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_tok = q_tok;
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.lse = lse;
    p.block_table = block_table;
    p.context_lens = context_lens;
    p.token_starts = token_starts;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.head_dim = head_dim;
    p.block_size = make_fastdiv(block_size);
    p.fd_heads = make_fastdiv(p.shape.item_heads);
    p.tok_dim = view.tok_dim;
    p.box_tokens = view.box_tokens;
    p.query_box = query_box_tokens(p.shape);
    // A scale of 0 becomes the smallest above it: a masked score, -infinity, then
    // still weighs 0, and every other still (all but) nothing against its reference.
    p.scale_log2 = std::max(static_cast<float>(std::fabs(scale)), FLT_MIN);
    p.negative = scale < 0;
    p.v_scale = kv8 ? v_scale : 1.f;
    p.slot_rows = lay.slot_rows;
    p.cut = reinterpret_cast<CutItem *>(ws + lay.cut);
    p.part_ml = reinterpret_cast<float *>(ws + lay.part_ml);
    p.part_o = reinterpret_cast<float *>(ws + lay.part_o);
    CUtensorMap tq = {};
    rc = encode_query_map(&tq, q, head_dim, num_q_heads, num_tokens, q_tok, p.shape.item_heads, p.query_box);
    if (rc != PD_OK) return rc;
    // no more CTAs than the most units these sizes can make would be shared by
    const long long items = static_cast<long long>(num_seqs) + num_tokens / p.shape.block_tokens;
    const long long most = items * p.shape.heads * most_block_units(p.shape, p.max_tokens);
    if (most > kMaxUnits)
        return report(PD_ERR_INVALID, "%s: launch too large (%d tokens, tables of %d, a window of %d)", what, num_tokens, p.max_tokens, window);
    const int sms = sm_count_of_device();
    const int ctas = static_cast<int>(std::min<long long>(std::max(1, std::min(sms, kMaxCtas)), (most + kCtaUnits - 1) / kCtaUnits));
    p.ctas = make_fastdiv(ctas);
    p.most_units = static_cast<int>(most);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = kv8 ? dispatch<true>(dpad, &view.k, &view.v, &tq, p, ctas, st) : dispatch<false>(dpad, &view.k, &view.v, &tq, p, ctas, st);
    if (e != cudaSuccess) return report_cuda(e, "chunk attention launch");
    if (ctas > 1) {  // (one CTA cuts no item)
        FoldParams f = {};
        f.cut = p.cut;
        f.part_ml = p.part_ml;
        f.part_o = p.part_o;
        f.out = p.out;
        f.lse = lse;
        f.num_q_heads = num_q_heads;
        f.head_dim = head_dim;
        f.slot_rows = lay.slot_rows;
        f.fd_heads = p.fd_heads;
        f.item_heads = p.shape.item_heads;
        f.v_scale = p.v_scale;
        e = launch_fold(f, dpad, ctas, st);
        if (e != cudaSuccess) return report_cuda(e, "chunk attention fold launch");
    }
    return report_ok();
}

}  // namespace
}  // namespace chunk
}  // namespace pd

extern "C" {

size_t pd_chunk_workspace_bytes(int num_tokens, int num_q_heads, int num_kv_heads, int head_dim) {
    if (num_tokens <= 0 || num_kv_heads <= 0 || num_q_heads < num_kv_heads || num_q_heads % num_kv_heads || head_dim <= 0 ||
        head_dim > PD_MAX_HEAD_DIM)
        return 0;
    return pd::chunk::layout_of(num_tokens, num_q_heads, num_kv_heads, head_dim).end;
}

int pd_chunk_attn(const void *q, int64_t q_token_stride, const void *k_cache, const void *v_cache, const int32_t *block_table,
                  int max_blocks_per_seq, const int32_t *context_lens, const int32_t *token_starts, void *out, float *lse,
                  int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                  float inv_sqrt_d, int window, void *workspace, size_t workspace_bytes, void *stream) {
    return pd::chunk::chunk_impl("pd_chunk_attn", q, q_token_stride, k_cache, v_cache, false, 1.f, 1.f, block_table, max_blocks_per_seq,
                                 context_lens, token_starts, out, lse, num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim,
                                 block_size, num_blocks, inv_sqrt_d, window, workspace, workspace_bytes, stream);
}

int pd_chunk_attn_fp8(const void *q, int64_t q_token_stride, const void *k_cache, const void *v_cache, float k_scale, float v_scale,
                      const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens, const int32_t *token_starts,
                      void *out, float *lse, int num_tokens, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
                      int block_size, int num_blocks, float inv_sqrt_d, int window, void *workspace, size_t workspace_bytes,
                      void *stream) {
    return pd::chunk::chunk_impl("pd_chunk_attn_fp8", q, q_token_stride, k_cache, v_cache, true, k_scale, v_scale, block_table,
                                 max_blocks_per_seq, context_lens, token_starts, out, lse, num_tokens, num_seqs, num_q_heads,
                                 num_kv_heads, head_dim, block_size, num_blocks, inv_sqrt_d, window, workspace, workspace_bytes, stream);
}

int pd_debug_chunk_walk(int num_seqs, const int32_t *token_starts, const int32_t *context_lens, int num_q_heads, int num_kv_heads,
                        int head_dim, int window, int max_ctas, int32_t *segments, int max_segments, int *num_segments,
                        int64_t *totals) {
    using namespace pd::chunk;
    const int rc = pd::check_shape(num_q_heads, num_kv_heads, head_dim, 16);
    if (rc != PD_OK) return rc;
    if (num_seqs < 0 || window < 0 || max_ctas < 1 || max_ctas > kMaxCtas || max_segments < 0 || !context_lens || !segments ||
        !num_segments || !totals)
        return pd::report(PD_ERR_INVALID, "pd_debug_chunk_walk: an argument is out of range or null");
    const int dpad = dpad_of(head_dim);
    const Shape s = make_shape(num_q_heads, num_kv_heads, dpad, window);
    for (int i = 0; i < num_seqs; ++i)
        if (context_lens[i] < 0 || context_lens[i] > 0x7fffffff - 256 ||
            (token_starts && (token_starts[i] < 0 || token_starts[i + 1] < token_starts[i])))
            return pd::report(PD_ERR_INVALID, "pd_debug_chunk_walk: sequence %d", i);
    const auto spans = [&](int i) {
        Span q = {i, 1, 0, context_lens[i]};
        if (token_starts) q.first = token_starts[i], q.n = token_starts[i + 1] - token_starts[i];
        q.past = q.len - q.n;
        return q;
    };
    // (bounded as the launch is, by each sequence's length)
    long long most = 0;
    for (int i = 0; i < num_seqs; ++i)
        most += (1ll + spans(i).n / s.block_tokens) * s.heads * most_block_units(s, context_lens[i]);
    if (most > kMaxUnits) return pd::report(PD_ERR_INVALID, "pd_debug_chunk_walk: too large");
    int W = 0;
    for (int i = 0; i < num_seqs; ++i) W += s.heads * head_units(s, spans(i));
    const int share = cta_units(W, pd::make_fastdiv(max_ctas)), C = (W + share - 1) / share;
    int n = 0;
    for (int c = 0; c < C; ++c) {
        Walk w = {};
        w.u = c * share;
        w.end = std::min(W, (c + 1) * share);
        int rest = w.u;
        while (rest >= s.heads * head_units(s, spans(w.seq))) rest -= s.heads * head_units(s, spans(w.seq++));
        w.span = spans(w.seq);
        const int of_head = head_units(s, w.span);
        w.kvh = rest / of_head / s.head_parts;
        w.part = rest / of_head % s.head_parts;
        rest %= of_head;
        for (int of = blocks_of(s, w.span.n); of > 1;) {  // (by halves where a warp takes 32nds)
            const int step = (of + 1) / 2;
            const bool up = units_before(s, w.span, w.block + step) <= rest;
            w.block += up ? step : 0;
            of = up ? of - step : step;
        }
        w.skip = rest - units_before(s, w.span, w.block);
        Segment g;
        while (next_segment(s, num_seqs, spans, w, g)) {
            if (n == max_segments) return pd::report(PD_ERR_CAPACITY, "pd_debug_chunk_walk: more than %d segments", n);
            const int32_t v[11] = {c, g.seq, g.kvh, g.head, g.heads, g.token, g.tokens, g.tile0, g.n, g.begins ? (g.whole ? 2 : 1) : 0,
                                   g.item_last / share};
            std::copy(v, v + 11, segments + 11ll * n++);
        }
    }
    *num_segments = n;
    totals[0] = W;
    totals[1] = C;
    totals[2] = s.block_tokens;
    totals[3] = 1 << s.tile_log2;
    totals[4] = s.item_heads;
    totals[5] = query_box_tokens(s);
    return pd::report_ok();
}

}  // extern "C"
