// C ABI of the calls around the scoring of trees of guesses: edits of logits.
// Argument checks and kernel launches; the operations are documented in
// include/specverify.h.
#include "specverify.h"
#include "specverify_profile.h"

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "sv_common.hpp"
#include "sv_host.hpp"
#include "sv_adjust.hpp"

static_assert(SV_MAX_DRAFT == sv::kAdjustMost, "draft limit mismatch");

namespace {

constexpr int32_t kMaxTokens = 1 << 30;

// ---- edits of logits

// Tokens of the vocabulary per workgroup.
constexpr int kAdjustChunk = 8192;
// Workgroups that the rows of a sequence are divided for.
constexpr int64_t kAdjustGroups = 1024;

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
    a.mask_stride = ad->mask_stride * 4;
    a.num_masks = ad->num_masks;
    a.mask_rows = ad->mask_rows;
    a.nchunk = (sh->vocab + kAdjustChunk - 1) / kAdjustChunk;
    const int64_t rows = sh->max_draft + 1, one = (int64_t)sh->batch * a.nchunk;
    const int64_t runs = std::min(std::max<int64_t>(kAdjustGroups / one, 1), rows);
    a.run_rows = (int32_t)((rows + runs - 1) / runs);
    a.runs = (int32_t)((rows + a.run_rows - 1) / a.run_rows);
    if (!launchable((double)one * a.runs, sv::kThreads)) return SV_ERR_UNSUPPORTED;
    const uint32_t grid = (uint32_t)(one * a.runs);
    return by_dtype(sh->dtype, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value, CT = kAdjustChunk;
        const bool bias = a.total_bias > 0;
        if (logits == out && bias) launch_stream(prof, sv::adjust_kernel<DT, true, true, CT>, grid, stream, a);
        else if (logits == out) launch_stream(prof, sv::adjust_kernel<DT, true, false, CT>, grid, stream, a);
        else if (bias) launch_stream(prof, sv::adjust_kernel<DT, false, true, CT>, grid, stream, a);
        else launch_stream(prof, sv::adjust_kernel<DT, false, false, CT>, grid, stream, a);
        return launch_status();
    });
}

}  // namespace

extern "C" {

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
