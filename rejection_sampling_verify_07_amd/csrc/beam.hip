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
#include "sv_reorder.hpp"

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

// ---- state reorder

// Whether the places of [slabs][beams][heads][positions][row_bytes] with these
// strides are all distinct: every stride clears the extent of the dimensions
// inside it.
bool distinct_places(const sv_state_shape_t* sh, int64_t beams)
{
    int64_t size[4] = {sh->slabs, beams, sh->heads, sh->positions};
    int64_t stride[4] = {sh->slab_stride, sh->beam_stride, sh->head_stride, sh->position_stride};
    int64_t extent = sh->row_bytes;
    bool done[4] = {};
    for (int k = 0; k < 4; ++k) {
        int at = -1;  // the smallest stride left, of the dimensions that have more than one place
        for (int i = 0; i < 4; ++i)
            if (!done[i] && size[i] > 1 && (at < 0 || stride[i] < stride[at])) at = i;
        if (at < 0) return true;
        done[at] = true;
        if (stride[at] < extent || stride[at] > (INT64_MAX - extent) / (size[at] - 1)) return false;
        extent += stride[at] * (size[at] - 1);
    }
    return true;
}

// Columns per thread of the reorder.  4-byte pieces: 2 (60 us against 71 us with 1 and 60 us with 4 on 325 MB moved
// between 6 places, 211 / 206 / 220 us on 868 MB between 16); 16-byte pieces: 1 (77 us against 84 us with 2 on 629 MB
// between 4 places, equal on 8 and more).
constexpr int kReorderCols4 = 2;
// States from which the sources are read past the caches, where rows are whole 16-byte pieces: 1354 us against
// 1526 us on 4.3 GB of states, 84 against 96 us on 201 MB, but 11.3 against 10.4 us on 39 MB.  (Rows of 180 bytes share
// cache lines between waves: 70 against 60 us on 163 MB, so pieces of 4 bytes are read through them.)
constexpr double kReorderPastCaches = 128e6;

int reorder_cols(const sv_state_shape_t* sh, int vecb)
{
    return vecb == 16 || sh->beams > 16 ? 1 : kReorderCols4;
}

void launch_reorder(const sv_state_shape_t* sh, int vecb, bool past, const sv::ReorderArgs& a, uint32_t grid,
                    hipStream_t s, const sv_profile_events_t* prof)
{
    constexpr int C = kReorderCols4, M = SV_MAX_BEAMS;
    const int32_t w = sh->beams;
    if (vecb == 16) {
        if (w <= 8 && past) launch_stream(prof, sv::state_reorder_kernel<16, 8, 1, true>, grid, s, a);
        else if (w <= 8) launch_stream(prof, sv::state_reorder_kernel<16, 8, 1, false>, grid, s, a);
        else if (past) launch_stream(prof, sv::state_reorder_kernel<16, 16, 1, true>, grid, s, a);
        else launch_stream(prof, sv::state_reorder_kernel<16, 16, 1, false>, grid, s, a);
    } else if (vecb == 4) {
        if (w <= 8) launch_stream(prof, sv::state_reorder_kernel<4, 8, C, false>, grid, s, a);
        else if (w <= 16) launch_stream(prof, sv::state_reorder_kernel<4, 16, C, false>, grid, s, a);
        else if (past) launch_stream(prof, sv::state_reorder_kernel<4, M, 1, true>, grid, s, a);
        else launch_stream(prof, sv::state_reorder_kernel<4, M, 1, false>, grid, s, a);
    } else if (vecb == 2) {
        if (w <= 16) launch_stream(prof, sv::state_reorder_kernel<2, 16, C, false>, grid, s, a);
        else launch_stream(prof, sv::state_reorder_kernel<2, M, 1, false>, grid, s, a);
    } else {
        if (w <= 16) launch_stream(prof, sv::state_reorder_kernel<1, 16, C, false>, grid, s, a);
        else launch_stream(prof, sv::state_reorder_kernel<1, M, 1, false>, grid, s, a);
    }
}

sv_status_t state_reorder_common(const sv_state_shape_t* sh, void* states, const int32_t* parents,
                                 const int32_t* lengths, hipStream_t stream, const sv_profile_events_t* prof)
{
    if (sh == nullptr) return SV_ERR_INVALID_ARGUMENT;
    if (sh->slabs < 1 || sh->groups < 1 || sh->beams < 1 || sh->heads < 1 || sh->positions < 0 || sh->row_bytes < 0)
        return SV_ERR_INVALID_ARGUMENT;
    if (sh->beams > SV_MAX_BEAMS) return SV_ERR_UNSUPPORTED;
    if (sh->slab_stride < 0 || sh->beam_stride < 0 || sh->head_stride < 0 || sh->position_stride < 0)
        return SV_ERR_INVALID_ARGUMENT;
    const bool empty = sh->positions == 0 || sh->row_bytes == 0;
    if (!empty && !distinct_places(sh, (int64_t)sh->groups * sh->beams)) return SV_ERR_INVALID_ARGUMENT;
    if ((states == nullptr && !empty) || parents == nullptr || !aligned(parents, 4) || !aligned(lengths, 4))
        return SV_ERR_INVALID_ARGUMENT;
    if (empty) return SV_OK;
    // the widest piece that every row divides into; 16-byte pieces need rows on 4-byte places only
    uint64_t places = (uint64_t)(uintptr_t)states;
    if (sh->slabs > 1) places |= (uint64_t)sh->slab_stride;
    if ((int64_t)sh->groups * sh->beams > 1) places |= (uint64_t)sh->beam_stride;
    if (sh->heads > 1) places |= (uint64_t)sh->head_stride;
    if (sh->positions > 1) places |= (uint64_t)sh->position_stride;
    places |= (uint64_t)sh->row_bytes % 16;
    int vecb = places % 2 != 0 ? 1 : places % 4 != 0 ? 2 : sh->row_bytes % 16 != 0 ? 4 : 16;
    // 16 bytes of 64 places take every register of a wave: with more than 16 places 4-byte pieces are faster (190 us
    // against 205 us on 1.07 GB moved between 32 places, 116 against 128 us on 537 MB between 64)
    const double bytes = (double)sh->row_bytes * sh->positions * sh->heads * sh->groups * sh->beams * sh->slabs;
    const bool past = vecb == 16 && bytes > kReorderPastCaches;
    if (sh->beams > 16 && vecb == 16) vecb = 4;
    const int64_t pieces = sh->row_bytes / vecb;
    if (pieces > INT32_MAX) return SV_ERR_UNSUPPORTED;
    const int64_t cols = pieces * sh->positions;
    if (cols > INT32_MAX) return SV_ERR_UNSUPPORTED;
    const int64_t per = (int64_t)sv::kThreads * reorder_cols(sh, vecb);
    const int64_t tiles = (cols + per - 1) / per;
    const double grid = (double)tiles * sh->groups * sh->slabs * sh->heads;
    if (grid > (double)INT32_MAX) return SV_ERR_UNSUPPORTED;
    const sv::ReorderArgs a{static_cast<char*>(states), parents, lengths, sh->beams, sh->heads, sh->positions,
                            sh->slab_stride, sh->beam_stride, sh->head_stride, sh->position_stride,
                            (uint32_t)pieces, (uint32_t)cols, (uint32_t)tiles, sh->slabs};
    const uint32_t n = (uint32_t)(tiles * sh->groups * sh->slabs * sh->heads);
    launch_reorder(sh, vecb, past, a, n, stream, prof);
    return launch_status();
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

sv_status_t spec_state_reorder(const sv_state_shape_t* shape, void* states, const int32_t* parents,
                               const int32_t* lengths, hipStream_t stream)
{
    return state_reorder_common(shape, states, parents, lengths, stream, nullptr);
}

sv_status_t spec_state_reorder_profiled(const sv_profile_events_t* events, const sv_state_shape_t* shape, void* states,
                                        const int32_t* parents, const int32_t* lengths, hipStream_t stream)
{
    return state_reorder_common(shape, states, parents, lengths, stream, events);
}

}  // extern "C"
