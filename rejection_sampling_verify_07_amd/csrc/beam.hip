// C ABI of the beam-decoding calls: argument checks, workspace layout and
// kernel launches.  The operations are documented in include/specverify.h.
#include "specverify.h"
#include "specverify_profile.h"

#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "sv_common.hpp"
#include "sv_host.hpp"
#include "sv_beam.hpp"
#include "sv_reorder.hpp"
#include "sv_attention.hpp"

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

// A launch counts its threads in 32 bits.
bool launchable(double workgroups, int threads) { return workgroups * threads <= (double)UINT32_MAX; }

// ---- beam selection

// 16-byte loads per thread of the streaming pass: 29.8 us on 512 rows of 151936 bf16 logits, against 33.7 us with 2,
// 31.4 with 6 and 31.0 with 8; 1 to 8 within 1 us of one another on 4 to 128 rows of 50304.
constexpr int kBeamLoads = 4;

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
    if (!launchable((double)rows * chunks_for(sh->vocab, vec_of(sh->dtype), kBeamLoads), sv::kThreads) ||
        !launchable(sh->groups, sv::kPickThreads))
        return SV_ERR_UNSUPPORTED;
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
// inside it.  *bytes: the extent of all of them.
bool distinct_places(const sv_state_shape_t* sh, int64_t beams, int64_t* bytes)
{
    int64_t size[4] = {sh->slabs, beams, sh->heads, sh->positions};
    int64_t stride[4] = {sh->slab_stride, sh->beam_stride, sh->head_stride, sh->position_stride};
    int64_t& extent = *bytes;
    extent = sh->row_bytes;
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
    const int64_t batch = (int64_t)sh->groups * sh->beams;
    int64_t extent = 0;
    if (!empty && !distinct_places(sh, batch, &extent)) return SV_ERR_INVALID_ARGUMENT;
    if ((states == nullptr && !empty) || parents == nullptr || !aligned(parents, 4) || !aligned(lengths, 4))
        return SV_ERR_INVALID_ARGUMENT;
    if (empty) return SV_OK;
    // the order is read while states move: it may not lie among them
    const auto inside = [&](const int32_t* p) {
        const uintptr_t a = (uintptr_t)p, b = (uintptr_t)states;
        return p != nullptr && a < b + (uintptr_t)extent && b < a + (uintptr_t)batch * 4;
    };
    if (inside(parents) || inside(lengths)) return SV_ERR_INVALID_ARGUMENT;
    // the widest piece that every row divides into; 16-byte pieces need rows on 4-byte places only
    uint64_t places = (uint64_t)(uintptr_t)states;
    if (sh->slabs > 1) places |= (uint64_t)sh->slab_stride;
    if (batch > 1) places |= (uint64_t)sh->beam_stride;
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
    if (!launchable(grid, sv::kThreads)) return SV_ERR_UNSUPPORTED;
    const sv::ReorderArgs a{static_cast<char*>(states), parents, lengths, sh->beams, sh->heads, sh->positions,
                            sh->slab_stride, sh->beam_stride, sh->head_stride, sh->position_stride,
                            (uint32_t)pieces, (uint32_t)cols, (uint32_t)tiles, sh->slabs};
    const uint32_t n = (uint32_t)(tiles * sh->groups * sh->slabs * sh->heads);
    launch_reorder(sh, vecb, past, a, n, stream, prof);
    return launch_status();
}

// ---- shared-prefix attention

constexpr int32_t kMaxPosStride = 1 << 25;  // bytes: 64 positions stay within a 31-bit offset
constexpr int32_t kMaxPositions = 1 << 30;
constexpr int64_t kMaxRows = INT32_MAX / 2;  // query rows of one key/value head in one group

// Workgroups that the splits of the keys aim at.  Work whose rows fit one workgroup is bound by reading the caches, and
// one workgroup per CU reads them as fast as two while its parts cost half as much to write and join: 194 against
// 214 us on 4 groups of 8 beams with 65536 shared positions, 27 against 31 us for 128 rows per key head on 32768.
// Work of more row tiles is bound by the products, which two workgroups per CU overlap better: 122 against 150 us for
// 1280 rows per key head on 16384 positions.
constexpr int64_t kSplitReading = 256;
constexpr int64_t kSplitProducts = 512;
// Keys that a split keeps at least, one step of the four waves: 7.5 us for 4 single rows on 500 positions, 9.9 us with
// 512; 17 us for 80 rows of 256 columns on 2049 positions, 28 us with 512.
constexpr int32_t kSplitKeys = sv::kKeyRound;

// Caches from which keys that one workgroup alone reads are read past the L2: 57 against 63 us on 285 MB, 48 against
// 52 us on 201 MB; caches that stay in the 256 MB Infinity Cache from step to step lose by it (22.6 against 20.2 us
// on 74 MB).
constexpr double kReadPastCaches = 128e6;

struct AttnPlan {
    bool tiles, past;
    int32_t rows, rep, mtp, mts, ptiles, stiles, psplits, ssplits;
    int64_t punits, pblocks, grid;
    size_t off_acc, off_ml, bytes;
};

int32_t attn_splits(int64_t workgroups, int32_t positions, int64_t target)
{
    if (positions == 0) return 0;
    int64_t n = target / workgroups;
    const int64_t most = (positions + kSplitKeys - 1) / kSplitKeys;
    if (n > most) n = most;
    return n < 1 ? 1 : (int32_t)n;
}

AttnPlan attn_plan(const sv_attention_shape_t* sh)
{
    AttnPlan p{};
    p.rows = sh->total_draft + sh->batch;
    p.rep = sh->q_heads / sh->kv_heads;
    const int64_t per_group = sh->cu_groups != nullptr ? sh->max_group : sh->batch / sh->groups;
    const int64_t prows = per_group * (sh->max_draft + 1) * p.rep;
    const int32_t most = sh->head_dim == 256 ? 1 : 2;  // 16-row tiles per wave that the registers hold
    // More rows than one wave holds: the waves share the rows and the keys pass through LDS.  (64 rows per key head on
    // 8192 positions: 50 us, against 77 us with 64 rows in every wave; 32 rows on 4096: 32 us, against 26 us without.)
    p.tiles = prows > most * 16;
    p.mtp = prows <= 16 ? 1 : most;
    const int32_t wg_rows = p.mtp * 16 * (p.tiles ? sv::kAttnWaves : 1);
    p.ptiles = (int32_t)((prows + wg_rows - 1) / wg_rows);
    // (20 rows per sequence and key head on 300 own positions: 30 us with two tiles per wave, 36 us with one)
    const int64_t srows = (int64_t)(sh->max_draft + 1) * p.rep;
    p.mts = srows <= 16 ? 1 : most;
    p.stiles = (int32_t)((srows + p.mts * 16 - 1) / (p.mts * 16));
    // Row tiles that hold anything, at most: ragged groups have fewer than groups * ptiles.  (2 groups of 40 with K 0..6,
    // 2 key heads of 64, 20000 positions: 49 us against 65 us with the splits that the fullest group would need.)
    const int64_t tiles =
        std::min<int64_t>((int64_t)sh->groups * p.ptiles, (int64_t)p.rows * p.rep / wg_rows + sh->groups);
    p.psplits = attn_splits(tiles * sh->kv_heads, sh->max_prefix,
                            p.ptiles == 1 ? kSplitReading : kSplitProducts);
    p.ssplits = attn_splits((int64_t)sh->batch * sh->kv_heads * p.stiles, sh->max_suffix, kSplitReading);
    const double positions = (double)sh->groups * sh->max_prefix + (double)sh->batch * sh->max_suffix;
    p.past = positions * sh->kv_heads * sh->head_dim * 4 > kReadPastCaches;
    p.punits = (int64_t)sh->groups * sh->kv_heads * p.psplits;
    p.pblocks = (p.punits + 7) / 8 * 8 * p.ptiles;
    p.grid = p.pblocks + (int64_t)sh->batch * sh->kv_heads * p.stiles * p.ssplits;
    const size_t n = (size_t)p.rows * (size_t)sh->q_heads * (size_t)(p.psplits + p.ssplits);
    p.off_acc = 0;
    p.off_ml = align_up(n * (size_t)sh->head_dim * sizeof(float));
    p.bytes = align_up(p.off_ml + n * sizeof(float2));
    if (p.bytes == 0) p.bytes = kAlign;
    return p;
}

sv_status_t check_attention(const sv_attention_shape_t* sh, float scale)
{
    if (sh == nullptr) return SV_ERR_INVALID_ARGUMENT;
    const int32_t dt = dtype_of(sh);
    if (dt != SV_DTYPE_F32 && dt != SV_DTYPE_BF16 && dt != SV_DTYPE_F16) return SV_ERR_INVALID_ARGUMENT;
    if (sh->groups < 1 || sh->batch < 1 || sh->max_draft < 0 || sh->total_draft < 0 || sh->q_heads < 1 ||
        sh->kv_heads < 1 || sh->head_dim < 1 || sh->max_prefix < 0 || sh->max_suffix < 0)
        return SV_ERR_INVALID_ARGUMENT;
    if (sh->q_heads % sh->kv_heads != 0) return SV_ERR_INVALID_ARGUMENT;
    if (sh->cu_groups == nullptr && sh->batch % sh->groups != 0) return SV_ERR_INVALID_ARGUMENT;
    if (sh->cu_groups != nullptr && (sh->max_group < 1 || sh->max_group > sh->batch)) return SV_ERR_INVALID_ARGUMENT;
    const int64_t all = (int64_t)sh->batch * sh->max_draft;
    if (sh->total_draft > all || (sh->cu_draft == nullptr && sh->total_draft != all)) return SV_ERR_INVALID_ARGUMENT;
    if (!aligned(sh->cu_draft, 4) || !aligned(sh->cu_groups, 4) || !aligned(sh->prefix_lengths, 4) ||
        !aligned(sh->suffix_lengths, 4))
        return SV_ERR_INVALID_ARGUMENT;
    if (!(scale > 0.0f) || !isfinite(scale) || !isfinite((float)((double)scale * 1.4426950408889634)))
        return SV_ERR_INVALID_ARGUMENT;
    if (dt == SV_DTYPE_F32) return SV_ERR_UNSUPPORTED;
    if (sh->head_dim != 64 && sh->head_dim != 128 && sh->head_dim != 256) return SV_ERR_UNSUPPORTED;
    if (sh->max_draft > SV_MAX_DRAFT || sh->max_prefix > kMaxPositions || sh->max_suffix > kMaxPositions)
        return SV_ERR_UNSUPPORTED;
    if (((int64_t)sh->total_draft + sh->batch) * sh->q_heads > INT32_MAX / 2) return SV_ERR_UNSUPPORTED;
    const int64_t per_group = sh->cu_groups != nullptr ? sh->max_group : sh->batch / sh->groups;
    if (per_group * (sh->max_draft + 1) > kMaxRows / (sh->q_heads / sh->kv_heads)) return SV_ERR_UNSUPPORTED;
    const AttnPlan p = attn_plan(sh);
    const double join = ((double)p.rows * sh->q_heads + sv::kWaves - 1) / sv::kWaves;
    if (!launchable((double)p.grid, sv::kAttnThreads) || !launchable(join, sv::kThreads)) return SV_ERR_UNSUPPORTED;
    return SV_OK;
}

// A cache's pointer and strides (elements of 2 bytes): 16-byte places.
bool cache_ok(const sv_cache_t* c)
{
    if (c == nullptr || c->data == nullptr || !aligned(c->data, 16)) return false;
    return c->batch_stride >= 0 && c->head_stride >= 0 && c->position_stride >= 0 && c->batch_stride % 8 == 0 &&
           c->head_stride % 8 == 0 && c->position_stride % 8 == 0;
}

// Whether rows of `width` elements at two strides lie apart.
bool distinct_rows(int64_t s0, int64_t n0, int64_t s1, int64_t n1, int64_t width)
{
    if (n0 < 2) s0 = 0;
    if (n1 < 2) s1 = 0;
    const bool first = n1 < 2 || (n0 > 1 && s0 < s1);  // the inner of the two
    const int64_t si = first ? s0 : s1, ni = first ? n0 : n1, so = first ? s1 : s0, no = first ? n1 : n0;
    if (ni > 1 && si < width) return false;
    return no < 2 || (ni < 2 ? so >= width : so >= width && (so - width) / si >= ni - 1);
}

template <int DT, int D>
sv_status_t run_attention(const AttnPlan& p, const sv::AttnArgs& a, hipStream_t stream,
                          const sv_profile_events_t* prof)
{
    const uint32_t grid = (uint32_t)p.grid;
    if (grid > 0) {
        const auto launch = [&](auto kernel) {
            launch_stream_nt(prof, kernel, grid, sv::kAttnThreads, stream, a);
        };
        constexpr int MT = D == 256 ? 1 : 2;
        if (p.tiles && p.mts == 1) launch(sv::attn_part_kernel<DT, D, true, MT, 1>);
        else if (p.tiles) launch(sv::attn_part_kernel<DT, D, true, MT, MT>);
        else if (p.mtp == 1) launch(sv::attn_part_kernel<DT, D, false, 1, 1>);
        else if (p.mts == 1) launch(sv::attn_part_kernel<DT, D, false, MT, 1>);
        else launch(sv::attn_part_kernel<DT, D, false, MT, MT>);
        if (launch_status() != SV_OK) return SV_ERR_HIP;
    }
    const int64_t per = sv::kWaves;  // one wave per (row, head)
    const int64_t n = (int64_t)a.rows * a.q_heads;
    hipLaunchKernelGGL((sv::attn_join_kernel<DT, D>), dim3((uint32_t)((n + per - 1) / per)), dim3(sv::kThreads), 0,
                       stream, a);
    return launch_status();
}

sv_status_t prefix_attention_common(const sv_attention_shape_t* sh, const void* q, const sv_cache_t* prefix_k,
                                    const sv_cache_t* prefix_v, const sv_cache_t* suffix_k, const sv_cache_t* suffix_v,
                                    float scale, void* out, float* out_lse, void* workspace, size_t* workspace_bytes,
                                    hipStream_t stream, const sv_profile_events_t* prof)
{
    if (workspace_bytes == nullptr) return SV_ERR_INVALID_ARGUMENT;
    const sv_status_t st = check_attention(sh, scale);
    if (st != SV_OK) return st;
    const AttnPlan p = attn_plan(sh);
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
    const sv_cache_t none{};
    const sv_cache_t *pk = &none, *pv = &none, *sk = &none, *svc = &none;
    if (sh->max_prefix > 0) {
        if (!cache_ok(prefix_k) || !cache_ok(prefix_v)) return SV_ERR_INVALID_ARGUMENT;
        pk = prefix_k;
        pv = prefix_v;
    }
    if (sh->max_suffix > 0) {
        if (!cache_ok(suffix_k) || !cache_ok(suffix_v)) return SV_ERR_INVALID_ARGUMENT;
        sk = suffix_k;
        svc = suffix_v;
    }
    for (const sv_cache_t* c : {pk, pv, sk, svc})
        if (c->position_stride * 2 > kMaxPosStride) return SV_ERR_UNSUPPORTED;
    if (*workspace_bytes < p.bytes) return SV_ERR_WORKSPACE_TOO_SMALL;
    sv::AttnArgs a{};
    a.q = static_cast<const char*>(q);
    a.pk = static_cast<const char*>(pk->data);
    a.pv = static_cast<const char*>(pv->data);
    a.sk = static_cast<const char*>(sk->data);
    a.sv = static_cast<const char*>(svc->data);
    a.out = static_cast<char*>(out);
    a.lse = out_lse;
    a.q_row = sh->q_row_stride * 2;
    a.q_head = sh->q_head_stride * 2;
    a.out_row = sh->out_row_stride * 2;
    a.out_head = sh->out_head_stride * 2;
    a.pk_group = pk->batch_stride * 2;
    a.pk_head = pk->head_stride * 2;
    a.pk_pos = (int32_t)(pk->position_stride * 2);
    a.pv_group = pv->batch_stride * 2;
    a.pv_head = pv->head_stride * 2;
    a.pv_pos = (int32_t)(pv->position_stride * 2);
    a.sk_seq = sk->batch_stride * 2;
    a.sk_head = sk->head_stride * 2;
    a.sk_pos = (int32_t)(sk->position_stride * 2);
    a.sv_seq = svc->batch_stride * 2;
    a.sv_head = svc->head_stride * 2;
    a.sv_pos = (int32_t)(svc->position_stride * 2);
    a.cu_draft = sh->cu_draft;
    a.cu_groups = sh->cu_groups;
    a.prefix_len = sh->prefix_lengths;
    a.suffix_len = sh->suffix_lengths;
    a.groups = sh->groups;
    a.batch = sh->batch;
    a.rows = p.rows;
    a.max_draft = sh->max_draft;
    a.per_group = sh->batch / sh->groups;
    a.max_prefix = sh->max_prefix;
    a.max_suffix = sh->max_suffix;
    a.q_heads = sh->q_heads;
    a.kv_heads = sh->kv_heads;
    a.rep = p.rep;
    a.c = (float)((double)scale * 1.4426950408889634);
    a.psplits = p.psplits;
    a.ssplits = p.ssplits;
    a.ptiles = p.ptiles;
    a.stiles = p.stiles;
    a.past = p.past;
    a.punits = (uint32_t)p.punits;
    a.pblocks = (uint32_t)p.pblocks;
    a.acc = ws_at<float>(workspace, p.off_acc);
    a.ml = ws_at<float2>(workspace, p.off_ml);
    return by_dtype(sh->dtype, [&](auto dtc) -> sv_status_t {
        constexpr int DT = decltype(dtc)::value;
        if constexpr (DT == sv::DT_F32) {
            return SV_ERR_UNSUPPORTED;
        } else {
            switch (sh->head_dim) {
                case 64: return run_attention<DT, 64>(p, a, stream, prof);
                case 128: return run_attention<DT, 128>(p, a, stream, prof);
                default: return run_attention<DT, 256>(p, a, stream, prof);
            }
        }
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

sv_status_t spec_prefix_attention(const sv_attention_shape_t* shape, const void* q, const sv_cache_t* prefix_k,
                                  const sv_cache_t* prefix_v, const sv_cache_t* suffix_k, const sv_cache_t* suffix_v,
                                  float scale, void* out, float* out_lse, void* workspace, size_t* workspace_bytes,
                                  hipStream_t stream)
{
    return prefix_attention_common(shape, q, prefix_k, prefix_v, suffix_k, suffix_v, scale, out, out_lse, workspace,
                                   workspace_bytes, stream, nullptr);
}

sv_status_t spec_prefix_attention_profiled(const sv_profile_events_t* events, const sv_attention_shape_t* shape,
                                           const void* q, const sv_cache_t* prefix_k, const sv_cache_t* prefix_v,
                                           const sv_cache_t* suffix_k, const sv_cache_t* suffix_v, float scale,
                                           void* out, float* out_lse, void* workspace, size_t* workspace_bytes,
                                           hipStream_t stream)
{
    return prefix_attention_common(shape, q, prefix_k, prefix_v, suffix_k, suffix_v, scale, out, out_lse, workspace,
                                   workspace_bytes, stream, events);
}

}  // extern "C"
