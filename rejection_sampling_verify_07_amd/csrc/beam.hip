// C ABI of the beam-decoding calls: argument checks, workspace layout and
// kernel launches.  The operations are documented in include/specverify.h.
#include "specverify.h"
#include "specverify_profile.h"

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "sv_common.hpp"
#include "sv_host.hpp"
#include "sv_beam.hpp"

static_assert(SV_MAX_BEAMS == sv::kBeamMaxBeams, "beam limit mismatch");
static_assert(SV_MAX_SELECT == sv::kBeamMaxSelect, "selection limit mismatch");

namespace {

// The caller's dtype field as an integer (any int may be stored there by a C caller).
template <class Shape>
int32_t dtype_of(const Shape* sh)
{
    static_assert(sizeof(sh->dtype) == sizeof(int32_t), "sv_dtype_t is an int-sized enum");
    int32_t v;
    memcpy(&v, &sh->dtype, sizeof v);
    return v;
}

// ---- beam selection

constexpr int kBeamLoads = 4;  // 16-byte loads per thread of the streaming pass

struct BeamPlan {
    int32_t rows, nchunk, nblk, nblkp;
    size_t off_blkmax, off_parts, bytes;
};

BeamPlan beam_plan(const sv_beam_shape_t* sh)
{
    BeamPlan p{};
    p.rows = sh->groups * sh->beams;
    p.nchunk = chunks_for(sh->vocab, vec_of(sh->dtype), kBeamLoads);
    p.nblk = p.nchunk * kBeamLoads * (sv::kThreads * 16 / sv::kBeamBlockBytes);
    p.nblkp = (p.nblk + sv::kWave - 1) / sv::kWave * sv::kWave;
    p.off_blkmax = 0;
    p.off_parts = align_up((size_t)p.rows * (size_t)p.nblkp * sizeof(float));
    p.bytes = align_up(p.off_parts + (size_t)p.rows * (size_t)p.nchunk * sv::kWaves * sizeof(sv::BeamPart));
    return p;
}

sv_status_t check_beam(const sv_beam_shape_t* sh, float temperature, int32_t pad_token)
{
    if (sh == nullptr) return SV_ERR_INVALID_ARGUMENT;
    const int32_t dt = dtype_of(sh);
    if (dt != SV_DTYPE_F32 && dt != SV_DTYPE_BF16 && dt != SV_DTYPE_F16) return SV_ERR_INVALID_ARGUMENT;
    if (sh->groups < 1 || sh->beams < 1 || sh->vocab < 1 || sh->num_select < 1 || sh->row_stride < sh->vocab)
        return SV_ERR_INVALID_ARGUMENT;
    if (!(temperature > 0.0f) || !isfinite(temperature) || !isfinite(scale_of(temperature)))
        return SV_ERR_INVALID_ARGUMENT;
    if (pad_token < 0 || pad_token >= sh->vocab) return SV_ERR_INVALID_ARGUMENT;
    if (sh->vocab > SV_MAX_VOCAB || sh->beams > SV_MAX_BEAMS || sh->num_select > SV_MAX_SELECT)
        return SV_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)sh->groups * sh->beams;
    if (rows * chunks_for(sh->vocab, vec_of(sh->dtype), 1) > INT32_MAX) return SV_ERR_UNSUPPORTED;
    if ((int64_t)sh->row_stride > INT64_MAX / 8 / rows) return SV_ERR_UNSUPPORTED;
    return SV_OK;
}

sv_status_t beam_select_common(const sv_beam_shape_t* sh, const void* logits, const float* scores,
                               const uint8_t* finished, float temperature, int32_t pad_token, float* out_scores,
                               int32_t* out_tokens, int32_t* out_parents, void* workspace, size_t* workspace_bytes,
                               hipStream_t stream, const sv_profile_events_t* prof)
{
    if (workspace_bytes == nullptr) return SV_ERR_INVALID_ARGUMENT;
    const sv_status_t st = check_beam(sh, temperature, pad_token);
    if (st != SV_OK) return st;
    const BeamPlan p = beam_plan(sh);
    if (workspace == nullptr) {
        *workspace_bytes = p.bytes;
        return SV_OK;
    }
    const size_t es = esize_of(sh->dtype);
    if (logits == nullptr || scores == nullptr || out_scores == nullptr || out_tokens == nullptr ||
        out_parents == nullptr)
        return SV_ERR_INVALID_ARGUMENT;
    if (!aligned(logits, es) || !aligned(scores, 4) || !aligned(out_scores, 4) || !aligned(out_tokens, 4) ||
        !aligned(out_parents, 4) || !aligned(workspace, kAlign))
        return SV_ERR_INVALID_ARGUMENT;
    if (*workspace_bytes < p.bytes) return SV_ERR_WORKSPACE_TOO_SMALL;
    return by_dtype(sh->dtype, [&](auto dtc) {
        constexpr int DT = decltype(dtc)::value;
        const sv::RowSet rs{static_cast<const char*>(logits), nullptr, (int64_t)(sh->row_stride * (int64_t)es), 0,
                            p.rows};
        float* blkmax = ws_at<float>(workspace, p.off_blkmax);
        sv::BeamPart* parts = ws_at<sv::BeamPart>(workspace, p.off_parts);
        launch_stream(prof, sv::beam_stream_kernel<DT, kBeamLoads>, (uint32_t)p.rows * (uint32_t)p.nchunk, stream, rs,
                      scores, finished, sh->vocab, p.nchunk, p.nblkp, scale_of(temperature), blkmax, parts);
        if (launch_status() != SV_OK) return SV_ERR_HIP;
        const sv::PickArgs pa{rs, scores, finished, sh->beams, sh->vocab, sh->num_select, p.nchunk * sv::kWaves,
                              p.nblk, p.nblkp, pad_token, temperature, blkmax, parts, out_scores, out_tokens,
                              out_parents};
        hipLaunchKernelGGL((sv::beam_pick_kernel<DT>), dim3(sh->groups), dim3(sv::kPickThreads), 0, stream, pa);
        return launch_status();
    });
}

}  // namespace

extern "C" {

sv_status_t spec_beam_select(const sv_beam_shape_t* shape, const void* logits, const float* scores,
                             const uint8_t* finished, float temperature, int32_t pad_token, float* out_scores,
                             int32_t* out_tokens, int32_t* out_parents, void* workspace, size_t* workspace_bytes,
                             hipStream_t stream)
{
    return beam_select_common(shape, logits, scores, finished, temperature, pad_token, out_scores, out_tokens,
                              out_parents, workspace, workspace_bytes, stream, nullptr);
}

sv_status_t spec_beam_select_profiled(const sv_profile_events_t* events, const sv_beam_shape_t* shape,
                                      const void* logits, const float* scores, const uint8_t* finished,
                                      float temperature, int32_t pad_token, float* out_scores, int32_t* out_tokens,
                                      int32_t* out_parents, void* workspace, size_t* workspace_bytes,
                                      hipStream_t stream)
{
    return beam_select_common(shape, logits, scores, finished, temperature, pad_token, out_scores, out_tokens,
                              out_parents, workspace, workspace_bytes, stream, events);
}

}  // extern "C"
