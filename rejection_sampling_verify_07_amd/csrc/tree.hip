// C ABI of the calls around the scoring of trees of guesses: edits of logits and
// attention over paged caches.  Argument checks, workspace layout and kernel launches; the operations are documented in
// include/specverify.h.
#include "specverify.h"
#include "specverify_profile.h"

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "sv_common.hpp"
#include "sv_host.hpp"
#include "sv_adjust.hpp"
#include "sv_tree_attention.hpp"

static_assert(SV_MAX_DRAFT == sv::kAdjustMost && SV_MAX_DRAFT == sv::kTreeMostGuesses, "draft limit mismatch");

namespace {

constexpr int32_t kMaxTokens = (1 << 30) - 1;  // a text's count of one token stays below the table entry's flags

// ---- edits of logits

// Threads of a workgroup, of 8 tokens of the vocabulary each.  320 rows of 151936 bf16 logits with texts of up to 8000
// tokens: 46 us with 512, 45 with 1024, 51 with 256; one row of 50304 fp32 logits 4.9 us, 5.1 with 256, 7.5 with 1024.
// (With smaller tables in LDS more workgroups stay on a CU, with larger ones fewer of them read the texts.)
constexpr int kAdjustThreads = 512;
constexpr int kAdjustTokens = 8;
// Bias entries that a table of 16 bits can number.
constexpr int32_t kAdjustFewBiases = 65535;
// Workgroups that the rows of a sequence are divided for: each counts the text anew.  One sequence of 65 rows of 151936
// fp32 logits under masks: 30 us with 256, 29.5 with 1024, 48 with 4096; 4 of 9 bf16 rows 12.8, 11.5 and 16.2.
constexpr int64_t kAdjustGroups = 1024;

// Bytes of logits (of all rows; in place only masked vectors are stored whole) from which whole vectors are stored past the
// caches.  Past them and through them, bf16 rows of 151936, three of four sequences under masks: 320 rows in place 45 and 45
// us with one set of logits, which the 256 MB cache holds, 48 and 54 with three in turn, 59 and 63 with four; four sets in
// turn of 210 rows (64 MB) in place 36 and 37, apart 52 and 55; of 80 rows (24 MB) 23 and 23, apart 24 and 25.  Between
// these, calls apart would gain too: 130 rows 29 and 36.
constexpr double kAdjustPast = 64e6;

sv_status_t check_adjust(const sv_adjust_shape_t* sh, const sv_adjust_t* ad, const void* logits, const void* out)
{
    if (sh == nullptr || ad == nullptr) return SV_ERR_INVALID_ARGUMENT;
    const int32_t dt = dtype_of(sh);
    if (dt != SV_DTYPE_F32 && dt != SV_DTYPE_BF16 && dt != SV_DTYPE_F16) return SV_ERR_INVALID_ARGUMENT;
    if (sh->batch < 1 || sh->max_draft < 0 || sh->total_draft < 0 || sh->vocab < 1) return SV_ERR_INVALID_ARGUMENT;
    const int64_t all = (int64_t)sh->batch * sh->max_draft, rows = (int64_t)sh->total_draft + sh->batch;
    if (sh->total_draft > all || (sh->cu_draft == nullptr && sh->total_draft != all)) return SV_ERR_INVALID_ARGUMENT;
    if (sh->row_stride < sh->vocab || sh->out_row_stride < sh->vocab) return SV_ERR_INVALID_ARGUMENT;
    if (ad->tokens != nullptr && (ad->max_tokens < 0 || (sh->batch > 1 && ad->token_stride < ad->max_tokens)))
        return SV_ERR_INVALID_ARGUMENT;
    if (ad->total_bias < 0 || (ad->total_bias > 0 && (ad->bias_ids == nullptr || ad->bias_values == nullptr)))
        return SV_ERR_INVALID_ARGUMENT;
    if (ad->masks != nullptr) {
        if (ad->num_masks < 1 || ad->mask_stride < (sh->vocab + 31) / 32) return SV_ERR_INVALID_ARGUMENT;
        if (ad->mask_rows == nullptr && ad->num_masks < rows) return SV_ERR_INVALID_ARGUMENT;
    }
    for (const void* p : {(const void*)sh->cu_draft, (const void*)sh->draft_ids, (const void*)sh->parents,
                          (const void*)ad->tokens, (const void*)ad->lengths, (const void*)ad->prompt_lengths,
                          (const void*)ad->repetition, (const void*)ad->presence, (const void*)ad->frequency,
                          (const void*)ad->bias_ids, (const void*)ad->bias_values, (const void*)ad->cu_bias,
                          (const void*)ad->masks, (const void*)ad->mask_rows})
        if (!aligned(p, 4)) return SV_ERR_INVALID_ARGUMENT;
    const size_t es = esize_of(sh->dtype);
    if (logits == nullptr || out == nullptr || !aligned(logits, es) || !aligned(out, es)) return SV_ERR_INVALID_ARGUMENT;
    if (sh->vocab > SV_MAX_VOCAB || sh->max_draft > SV_MAX_DRAFT || rows > INT32_MAX / 2) return SV_ERR_UNSUPPORTED;
    if (ad->tokens != nullptr && ad->max_tokens > kMaxTokens) return SV_ERR_UNSUPPORTED;
    if (sh->row_stride > INT64_MAX / 16 / rows || sh->out_row_stride > INT64_MAX / 16 / rows ||
        ad->token_stride > INT64_MAX / 16 / sh->batch || ad->token_stride < INT64_MIN / 16 ||
        (ad->masks != nullptr && ad->mask_stride > INT64_MAX / 16 / ad->num_masks))
        return SV_ERR_UNSUPPORTED;
    // in place row by row, or apart
    if (logits == out) return sh->row_stride == sh->out_row_stride || rows == 1 ? SV_OK : SV_ERR_INVALID_ARGUMENT;
    const uintptr_t x = (uintptr_t)logits, y = (uintptr_t)out;
    const uintptr_t xn = (uintptr_t)((rows - 1) * sh->row_stride + sh->vocab) * es,
                    yn = (uintptr_t)((rows - 1) * sh->out_row_stride + sh->vocab) * es;
    return x < y + yn && y < x + xn ? SV_ERR_INVALID_ARGUMENT : SV_OK;
}

sv_status_t adjust_logits_common(const sv_adjust_shape_t* sh, const sv_adjust_t* ad, const void* logits, void* out,
                                 hipStream_t stream, const sv_profile_events_t* prof)
{
    const sv_status_t st = check_adjust(sh, ad, logits, out);
    if (st != SV_OK) return st;
    const int64_t es = (int64_t)esize_of(sh->dtype);
    sv::AdjustArgs a{};
    a.in = static_cast<const char*>(logits);
    a.out = static_cast<char*>(out);
    a.in_stride = sh->row_stride * es;
    a.out_stride = sh->out_row_stride * es;
    a.cu = sh->cu_draft;
    a.ids = sh->draft_ids;
    a.parents = sh->parents;
    a.batch = sh->batch;
    a.kmax = sh->max_draft;
    a.total_draft = sh->total_draft;
    a.vocab = sh->vocab;
    a.tokens = ad->max_tokens > 0 ? ad->tokens : nullptr;
    a.lengths = ad->lengths;
    a.prompt = ad->prompt_lengths;
    a.token_stride = ad->token_stride;
    a.max_tokens = ad->max_tokens;
    a.repetition = ad->repetition;
    a.presence = ad->presence;
    a.frequency = ad->frequency;
    a.bias_ids = ad->bias_ids;
    a.bias_values = ad->bias_values;
    a.cu_bias = ad->cu_bias;
    a.total_bias = ad->total_bias;
    a.masks = reinterpret_cast<const uint8_t*>(ad->masks);
    a.mask_stride = ad->masks != nullptr ? ad->mask_stride * 4 : 0;
    a.num_masks = ad->num_masks;
    a.mask_rows = ad->mask_rows;
    a.past = ((double)sh->total_draft + sh->batch) * sh->vocab * (double)es >= kAdjustPast;
    const int64_t rows = sh->max_draft + 1;
    const auto launch = [&](auto dt, auto inplace, auto bias) -> sv_status_t {
        constexpr int DT = decltype(dt)::value, NT = kAdjustThreads, CT = NT * kAdjustTokens;
        a.nchunk = (sh->vocab + CT - 1) / CT;
        const int64_t one = (int64_t)sh->batch * a.nchunk;
        const int64_t runs = std::min(std::max<int64_t>(kAdjustGroups / one, 1), rows);
        a.run_rows = (int32_t)((rows + runs - 1) / runs);
        a.runs = (int32_t)((rows + a.run_rows - 1) / a.run_rows);
        if (!launchable((double)one * a.runs, NT)) return SV_ERR_UNSUPPORTED;
        launch_stream_nt(prof, sv::adjust_kernel<DT, decltype(inplace)::value, decltype(bias)::value, CT, NT>,
                         (uint32_t)(one * a.runs), NT, stream, a);
        return launch_status();
    };
    return by_dtype(sh->dtype, [&](auto dt) {
        const auto by_bias = [&](auto inplace) {
            if (a.total_bias == 0) return launch(dt, inplace, std::integral_constant<int, sv::BIAS_NONE>{});
            if (a.total_bias <= kAdjustFewBiases) return launch(dt, inplace, std::integral_constant<int, sv::BIAS_16>{});
            return launch(dt, inplace, std::integral_constant<int, sv::BIAS_32>{});
        };
        return logits == out ? by_bias(std::true_type{}) : by_bias(std::false_type{});
    });
}

// ---- attention over paged caches

// Workgroups that the line of keys is dealt to: two per CU, one where LDS and registers hold no second one.  (48 ragged
// trees on 1000 to 8000 positions: 169 us with 512, 214 with 256, 178 with 1024.)
constexpr int32_t kTreeGroups = 512;
constexpr int32_t kTreeGroupsWide = 256;
// (Row, head)s from which each has D / 4 lanes of a join, not a wave: one row of 32 heads on 32001 positions 40 us with
// D / 4 lanes, 35 with the wave; 48 ragged trees of up to 9 rows 167 and 168, 64 of 8 rows and 64 columns 95 and 99.
constexpr int64_t kJoinSplit = 4096;

// Columns of a pair's cache up to which one workgroup takes the whole pair, without a deal and a join: so many for any
// call, twice as many from 64 workgroups on, four times from 256.  64 rows of 32/8 heads of 128 on up to 512 positions:
// 27 us dealt, 19.5 whole, on 256 22 and 12.6, on 1024 34 and 35; one row on 112 11.5 and 8.6, on 512 11.3 and 17.8.
constexpr int64_t kTreeWhole = 1 << 14;

struct TreePlan {
    bool whole;
    int32_t mt, wg_rows, row_tiles, groups, rows, capacity;
    int64_t grid, join;
    size_t off_plan, off_ml, off_acc, bytes;
};

TreePlan tree_plan(const sv_tree_shape_t* sh)
{
    TreePlan p{};
    p.rows = sh->total_draft + sh->batch;
    p.capacity = sh->max_pages * sh->page_size;
    const int32_t rep = sh->q_heads / sh->kv_heads;
    const int64_t rows = (int64_t)(sh->max_draft + 1) * rep;  // of one key head
    // 16-row tiles per wave: two where 64 rows do not do (and the registers hold them).  48 ragged trees of up to 36 rows a
    // key head: 169 us with one, 175 with two.
    const int32_t most = sh->head_dim == 256 ? 1 : 2;
    p.mt = rows <= sv::kAttnWaves * 16 ? 1 : most;
    p.wg_rows = p.mt * 16 * sv::kAttnWaves;
    p.row_tiles = (int32_t)((rows + p.wg_rows - 1) / p.wg_rows);
    const int64_t rounds = (int64_t)sh->batch * sh->kv_heads * (((int64_t)p.capacity + sv::kTreeRound - 1) / sv::kTreeRound);
    const int64_t target = std::max((sh->head_dim == 256 ? kTreeGroupsWide : kTreeGroups) / p.row_tiles, 1);
    const int64_t pairs = (int64_t)sh->batch * sh->kv_heads, workgroups = pairs * p.row_tiles;
    p.whole = (int64_t)p.capacity * sh->head_dim <= kTreeWhole * (workgroups >= 256 ? 4 : workgroups >= 64 ? 2 : 1);
    p.groups = p.whole ? (int32_t)pairs : (int32_t)std::min(target, rounds);
    p.grid = p.row_tiles == 1 ? p.groups : (int64_t)(p.groups + 7) / 8 * 8 * p.row_tiles;
    p.join = (int64_t)sh->batch * (sh->max_draft + 1) * sh->q_heads;
    const size_t slots = p.whole ? 0 : 2 * (size_t)p.groups * (size_t)p.row_tiles * (size_t)p.wg_rows;
    p.off_plan = 0;
    p.off_ml = align_up((size_t)(sh->batch + 3) * 4);
    p.off_acc = align_up(p.off_ml + slots * sizeof(float2));
    p.bytes = align_up(p.off_acc + slots * (size_t)sh->head_dim * sizeof(float));
    return p;
}

sv_status_t check_tree(const sv_tree_shape_t* sh, float scale)
{
    if (sh == nullptr) return SV_ERR_INVALID_ARGUMENT;
    const int32_t dt = dtype_of(sh);
    if (dt != SV_DTYPE_F32 && dt != SV_DTYPE_BF16 && dt != SV_DTYPE_F16) return SV_ERR_INVALID_ARGUMENT;
    if (sh->batch < 1 || sh->max_draft < 0 || sh->total_draft < 0 || sh->q_heads < 1 || sh->kv_heads < 1 ||
        sh->head_dim < 1 || sh->pages < 1 || sh->page_size < 1 || sh->max_pages < 1)
        return SV_ERR_INVALID_ARGUMENT;
    if (sh->q_heads % sh->kv_heads != 0) return SV_ERR_INVALID_ARGUMENT;
    const int64_t all = (int64_t)sh->batch * sh->max_draft;
    if (sh->total_draft > all || (sh->cu_draft == nullptr && sh->total_draft != all)) return SV_ERR_INVALID_ARGUMENT;
    if (sh->page_table == nullptr ? sh->max_pages != 1 || sh->pages < sh->batch
                                  : sh->batch > 1 && sh->table_stride < sh->max_pages)
        return SV_ERR_INVALID_ARGUMENT;
    for (const int32_t* p : {sh->cu_draft, sh->parents, sh->lengths, sh->page_table})
        if (!aligned(p, 4)) return SV_ERR_INVALID_ARGUMENT;
    if (!(scale > 0.0f) || !isfinite(scale) || !isfinite((float)((double)scale * 1.4426950408889634)))
        return SV_ERR_INVALID_ARGUMENT;
    if (dt == SV_DTYPE_F32) return SV_ERR_UNSUPPORTED;
    if (sh->head_dim != 64 && sh->head_dim != 128 && sh->head_dim != 256) return SV_ERR_UNSUPPORTED;
    if (sh->page_table != nullptr && sh->page_size % 16 != 0) return SV_ERR_UNSUPPORTED;
    if (sh->max_draft > SV_MAX_DRAFT || (int64_t)sh->max_pages * sh->page_size > kMaxPositions)
        return SV_ERR_UNSUPPORTED;
    if (((int64_t)sh->total_draft + sh->batch) * sh->q_heads > INT32_MAX / 2) return SV_ERR_UNSUPPORTED;
    if ((int64_t)(sh->q_heads / sh->kv_heads) * (sh->max_draft + 1) > INT32_MAX / 256) return SV_ERR_UNSUPPORTED;
    const double rounds = (double)sh->max_pages * sh->page_size / sv::kTreeRound + 1 + 2 * sv::kTreeExtra;
    if ((double)sh->batch * sh->kv_heads * rounds > (double)INT32_MAX) return SV_ERR_UNSUPPORTED;
    if (sh->table_stride > INT64_MAX / 8 / sh->batch) return SV_ERR_UNSUPPORTED;
    const TreePlan p = tree_plan(sh);
    if (!launchable((double)p.grid, sv::kAttnThreads) || !launchable((double)(p.join / sv::kWaves + 1), sv::kThreads))
        return SV_ERR_UNSUPPORTED;
    return SV_OK;
}

template <int DT, int D, int MT>
sv_status_t run_tree(const TreePlan& p, const sv::TreeArgs& a, hipStream_t stream, const sv_profile_events_t* prof)
{
    launch_stream_nt(prof, sv::tree_part_kernel<DT, D, MT>, (uint32_t)p.grid, sv::kAttnThreads, stream, a);
    if (launch_status() != SV_OK) return SV_ERR_HIP;
    if (p.whole) return SV_OK;
    constexpr int ROWS = MT * 16 * sv::kAttnWaves;
    const auto join = [&](auto split) {
        constexpr bool SPLIT = decltype(split)::value;
        const int64_t per = sv::kWaves * (SPLIT ? 1 : sv::kWave / (D / 4));  // (row, head)s of a workgroup
        hipLaunchKernelGGL((sv::tree_join_kernel<DT, D, ROWS, SPLIT>), dim3((uint32_t)((p.join + per - 1) / per)),
                           dim3(sv::kThreads), 0, stream, a);
    };
    if (D == 256 || p.join < kJoinSplit) join(std::true_type{});
    else if constexpr (D != 256) join(std::false_type{});
    return launch_status();
}

sv_status_t tree_attention_common(const sv_tree_shape_t* sh, const void* q, const sv_cache_t* k, const sv_cache_t* v,
                                  float scale, void* out, float* out_lse, void* workspace, size_t* workspace_bytes,
                                  hipStream_t stream, const sv_profile_events_t* prof)
{
    if (workspace_bytes == nullptr) return SV_ERR_INVALID_ARGUMENT;
    const sv_status_t st = check_tree(sh, scale);
    if (st != SV_OK) return st;
    const TreePlan p = tree_plan(sh);
    if (workspace == nullptr) {
        *workspace_bytes = p.bytes;
        return SV_OK;
    }
    if (q == nullptr || out == nullptr || !aligned(q, 16) || !aligned(out, 8) || !aligned(out_lse, 4) ||
        !aligned(workspace, kAlign))
        return SV_ERR_INVALID_ARGUMENT;
    if (sh->q_row_stride < 0 || sh->q_head_stride < 0 || sh->q_row_stride % 8 != 0 || sh->q_head_stride % 8 != 0 ||
        sh->out_row_stride < 0 || sh->out_head_stride < 0 || sh->out_row_stride % 4 != 0 ||
        sh->out_head_stride % 4 != 0)
        return SV_ERR_INVALID_ARGUMENT;
    if (!distinct_rows(sh->out_row_stride, p.rows, sh->out_head_stride, sh->q_heads, sh->head_dim))
        return SV_ERR_INVALID_ARGUMENT;
    if (!cache_ok(k) || !cache_ok(v)) return SV_ERR_INVALID_ARGUMENT;
    if (!cache_fits(k, sh->pages, sh->kv_heads) || !cache_fits(v, sh->pages, sh->kv_heads) ||
        !stride_ok(sh->q_row_stride, p.rows) || !stride_ok(sh->q_head_stride, sh->q_heads) ||
        !stride_ok(sh->out_row_stride, p.rows) || !stride_ok(sh->out_head_stride, sh->q_heads))
        return SV_ERR_UNSUPPORTED;
    if (*workspace_bytes < p.bytes) return SV_ERR_WORKSPACE_TOO_SMALL;
    sv::TreeArgs a{};
    a.q = static_cast<const char*>(q);
    a.k = static_cast<const char*>(k->data);
    a.v = static_cast<const char*>(v->data);
    a.out = static_cast<char*>(out);
    a.lse = out_lse;
    a.q_row = sh->q_row_stride * 2;
    a.q_head = sh->q_head_stride * 2;
    a.out_row = sh->out_row_stride * 2;
    a.out_head = sh->out_head_stride * 2;
    a.k_page = k->batch_stride * 2;
    a.k_head = k->head_stride * 2;
    a.v_page = v->batch_stride * 2;
    a.v_head = v->head_stride * 2;
    a.k_pos = (int32_t)(k->position_stride * 2);
    a.v_pos = (int32_t)(v->position_stride * 2);
    a.cu = sh->cu_draft;
    a.parents = sh->total_draft > 0 ? sh->parents : nullptr;
    a.lengths = sh->lengths;
    a.table = sh->page_table;
    a.table_stride = sh->table_stride;
    a.batch = sh->batch;
    a.rows = p.rows;
    a.kmax = sh->max_draft;
    a.pages = sh->pages;
    a.capacity = p.capacity;
    // g / grains as (g * mul) >> shift, exact for g < 2^31: mul = ceil(2^shift / grains) exceeds 2^shift / grains by less
    // than 1, and 2^shift >= 2^31 * grains
    a.grains = sh->page_table != nullptr ? sh->page_size / 16 : kMaxPositions / 16 + 64;
    a.grains_shift = 31;
    while ((1ull << (a.grains_shift - 31)) < (uint64_t)a.grains) ++a.grains_shift;
    a.grains_mul = (uint32_t)(((1ull << a.grains_shift) + (uint64_t)a.grains - 1) / (uint64_t)a.grains);
    a.q_heads = sh->q_heads;
    a.kv_heads = sh->kv_heads;
    a.rep = sh->q_heads / sh->kv_heads;
    a.c = (float)((double)scale * 1.4426950408889634);
    a.groups = p.groups;
    a.whole = p.whole;
    a.tiles = p.row_tiles;
    a.plan = ws_at<int32_t>(workspace, p.off_plan);
    a.ml = ws_at<float2>(workspace, p.off_ml);
    a.acc = ws_at<float>(workspace, p.off_acc);
    const auto by_rows = [&](auto dt, auto dim) -> sv_status_t {
        constexpr int DT = decltype(dt)::value, D = decltype(dim)::value;
        if constexpr (DT == sv::DT_F32) {
            return SV_ERR_UNSUPPORTED;
        } else {
            if constexpr (D != 256)
                if (p.mt == 2) return run_tree<DT, D, 2>(p, a, stream, prof);
            return run_tree<DT, D, 1>(p, a, stream, prof);
        }
    };
    return by_dtype(sh->dtype, [&](auto dt) -> sv_status_t {
        switch (sh->head_dim) {
            case 64: return by_rows(dt, std::integral_constant<int, 64>{});
            case 128: return by_rows(dt, std::integral_constant<int, 128>{});
            default: return by_rows(dt, std::integral_constant<int, 256>{});
        }
    });
}

}  // namespace

extern "C" {

sv_status_t spec_tree_attention(const sv_tree_shape_t* shape, const void* q, const sv_cache_t* k, const sv_cache_t* v,
                                float scale, void* out, float* out_lse, void* workspace, size_t* workspace_bytes,
                                hipStream_t stream)
{
    return tree_attention_common(shape, q, k, v, scale, out, out_lse, workspace, workspace_bytes, stream, nullptr);
}

sv_status_t spec_tree_attention_profiled(const sv_profile_events_t* events, const sv_tree_shape_t* shape, const void* q,
                                         const sv_cache_t* k, const sv_cache_t* v, float scale, void* out,
                                         float* out_lse, void* workspace, size_t* workspace_bytes, hipStream_t stream)
{
    return tree_attention_common(shape, q, k, v, scale, out, out_lse, workspace, workspace_bytes, stream, events);
}

sv_status_t spec_adjust_logits(const sv_adjust_shape_t* shape, const sv_adjust_t* adjust, const void* logits, void* out,
                               hipStream_t stream)
{
    return adjust_logits_common(shape, adjust, logits, out, stream, nullptr);
}

sv_status_t spec_adjust_logits_profiled(const sv_profile_events_t* events, const sv_adjust_shape_t* shape,
                                        const sv_adjust_t* adjust, const void* logits, void* out, hipStream_t stream)
{
    return adjust_logits_common(shape, adjust, logits, out, stream, events);
}

}  // extern "C"
