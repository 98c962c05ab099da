// C ABI of the calls on caches in pages: argument checks, workspace layout and
// kernel launches.  The operations are documented in include/specverify.h.
#include "specverify.h"
#include "specverify_profile.h"

#include <stdint.h>

#include <algorithm>

#include "sv_common.hpp"
#include "sv_host.hpp"
#include "sv_pages.hpp"

static_assert(SV_MAX_DRAFT == sv::kCompactMost, "draft limit mismatch");

namespace {

// The pool's checks, its extent in bytes, and the widest piece that every row divides into (16-byte pieces need rows
// on 4-byte places only).
sv_status_t check_pool(const sv_pool_t& p, const void* data, int64_t* extent, int* vecb)
{
    if (p.slabs < 1 || p.pages < 1 || p.page_size < 1 || p.heads < 1 || p.row_bytes < 1) return SV_ERR_INVALID_ARGUMENT;
    if (p.slab_stride < 0 || p.page_stride < 0 || p.head_stride < 0 || p.position_stride < 0)
        return SV_ERR_INVALID_ARGUMENT;
    if (!distinct_places<4>({p.slabs, p.pages, p.heads, p.page_size},
                            {p.slab_stride, p.page_stride, p.head_stride, p.position_stride}, p.row_bytes, extent))
        return SV_ERR_INVALID_ARGUMENT;
    uint64_t places = (uint64_t)(uintptr_t)data | (uint64_t)p.row_bytes % 16;
    if (p.slabs > 1) places |= (uint64_t)p.slab_stride;
    if (p.pages > 1) places |= (uint64_t)p.page_stride;
    if (p.heads > 1) places |= (uint64_t)p.head_stride;
    if (p.page_size > 1) places |= (uint64_t)p.position_stride;
    *vecb = places % 2 != 0 ? 1 : places % 4 != 0 ? 2 : p.row_bytes % 16 != 0 ? 4 : 16;
    return SV_OK;
}

// Pieces of one position in all slabs and heads (-1: too many).
int64_t columns_of(const sv_pool_t& p, int vecb)
{
    const int64_t pieces = p.row_bytes / vecb;
    const double all = (double)pieces * p.slabs * p.heads;
    return all > (double)INT32_MAX ? -1 : pieces * p.slabs * p.heads;
}

sv::Pool pool_args(const sv_pool_t& p, void* data, int vecb)
{
    return sv::Pool{static_cast<char*>(data), p.slab_stride, p.page_stride, p.head_stride, p.position_stride,
                    p.pages, p.page_size, (uint32_t)p.heads, (uint32_t)(p.row_bytes / vecb)};
}

// Whether [a, a + an) and [b, b + bn) share a byte (a null range shares none).
bool overlap(const void* a, int64_t an, const void* b, int64_t bn)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a != nullptr && b != nullptr && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Bytes from a table's first entry to its last one's end (its rows may lie apart).
int64_t table_bytes(int64_t rows, int64_t stride, int64_t entries) { return ((rows - 1) * stride + entries) * 4; }

// Calls fn with std::integral_constant<int, bytes of a piece>.
template <class F>
void by_piece(int vecb, F&& fn)
{
    if (vecb == 16) fn(std::integral_constant<int, 16>{});
    else if (vecb == 4) fn(std::integral_constant<int, 4>{});
    else if (vecb == 2) fn(std::integral_constant<int, 2>{});
    else fn(std::integral_constant<int, 1>{});
}

sv_status_t cache_compact_common(const sv_compact_shape_t* sh, void* data, const int32_t* lengths, const int32_t* path,
                                 const int32_t* num_accepted, int32_t* out_lengths, hipStream_t stream,
                                 const sv_profile_events_t* prof)
{
    if (sh == nullptr) return SV_ERR_INVALID_ARGUMENT;
    int64_t extent = 0;
    int vecb = 1;
    const sv_status_t st = check_pool(sh->pool, data, &extent, &vecb);
    if (st != SV_OK) return st;
    if (sh->batch < 1 || sh->max_draft < 0 || sh->total_draft < 0 || sh->max_pages < 1) return SV_ERR_INVALID_ARGUMENT;
    const int64_t all = (int64_t)sh->batch * sh->max_draft;
    if (sh->total_draft > all || (sh->cu_draft == nullptr && sh->total_draft != all)) return SV_ERR_INVALID_ARGUMENT;
    if (sh->page_table == nullptr ? sh->max_pages != 1 || sh->pool.pages < sh->batch
                                  : sh->batch > 1 && sh->table_stride < sh->max_pages)
        return SV_ERR_INVALID_ARGUMENT;
    if (data == nullptr || path == nullptr || num_accepted == nullptr || out_lengths == nullptr)
        return SV_ERR_INVALID_ARGUMENT;
    for (const int32_t* p : {lengths, path, num_accepted, (const int32_t*)out_lengths, sh->cu_draft, sh->page_table})
        if (!aligned(p, 4)) return SV_ERR_INVALID_ARGUMENT;
    if (sh->max_draft > SV_MAX_DRAFT || (int64_t)sh->max_pages * sh->pool.page_size > kMaxPositions)
        return SV_ERR_UNSUPPORTED;
    const int64_t rows = (int64_t)sh->total_draft + sh->batch;
    if (rows > INT32_MAX || sh->table_stride > INT64_MAX / 8 / sh->batch) return SV_ERR_UNSUPPORTED;
    const struct {
        const int32_t* p;
        int64_t bytes;
    } inputs[] = {{lengths, sh->batch * 4ll}, {path, rows * 4}, {num_accepted, sh->batch * 4ll},
                  {sh->cu_draft, (sh->batch + 1ll) * 4},
                  {sh->page_table,
                   sh->page_table != nullptr ? table_bytes(sh->batch, sh->table_stride, sh->max_pages) : 0}};
    for (const auto& in : inputs)
        if (overlap(in.p, in.bytes, data, extent) || overlap(in.p, in.bytes, out_lengths, sh->batch * 4ll))
            return SV_ERR_INVALID_ARGUMENT;
    if (overlap(out_lengths, sh->batch * 4ll, data, extent)) return SV_ERR_INVALID_ARGUMENT;
    const int64_t cols = columns_of(sh->pool, vecb);
    if (cols < 0) return SV_ERR_UNSUPPORTED;
    const int64_t tiles = (cols + sv::kThreads - 1) / sv::kThreads;
    if (!launchable((double)tiles * sh->batch, sv::kThreads)) return SV_ERR_UNSUPPORTED;
    const sv::CompactArgs a{pool_args(sh->pool, data, vecb), sh->cu_draft, sh->page_table, lengths, path, num_accepted,
                            out_lengths, sh->table_stride, sh->batch, sh->max_draft, sh->total_draft, sh->max_pages,
                            (uint32_t)cols, (uint32_t)tiles};
    by_piece(vecb, [&](auto v) {
        launch_stream(prof, sv::compact_kernel<decltype(v)::value>, (uint32_t)(tiles * sh->batch), stream, a);
    });
    return launch_status();
}

// Table entries, old and new, that one workgroup counts, in LDS: 4 places 7.7 us, 13.4 with the launches for any size, 64
// places of 17 pages 22 and 28.
constexpr int64_t kForkSmall = 1 << 16;
// Workgroups that copy for one place, at most: 64 places of 64 caches 21.4 us with 256, 22.0 with 64, 26.3 with 16.
constexpr int64_t kForkTiles = 256;

struct ForkPlan {
    size_t off_places, off_first, off_fresh, off_left, bytes;
    int64_t fresh;
};

ForkPlan fork_plan(const sv_fork_shape_t* sh)
{
    ForkPlan p{};
    p.fresh = std::min<int64_t>(sh->pool.pages, (int64_t)sh->batch * sh->max_pages);
    p.off_places = 0;
    p.off_first = align_up((size_t)sh->batch * sizeof(sv::ForkPlace));
    p.off_fresh = align_up(p.off_first + (size_t)sh->pool.pages * 4);
    p.off_left = align_up(p.off_fresh + (size_t)p.fresh * 4);
    p.bytes = p.off_left + kAlign;
    return p;
}

sv_status_t page_fork_common(const sv_fork_shape_t* sh, void* data, const int32_t* page_table, const int32_t* lengths,
                             const int32_t* parents, const int32_t* new_lengths, const int32_t* refs,
                             int32_t* out_table, int32_t* out_refs, int32_t* out_free, void* workspace,
                             size_t* workspace_bytes, hipStream_t stream, const sv_profile_events_t* prof)
{
    if (workspace_bytes == nullptr || sh == nullptr) return SV_ERR_INVALID_ARGUMENT;
    int64_t extent = 0;
    int vecb = 1;
    const sv_status_t st = check_pool(sh->pool, data, &extent, &vecb);
    if (st != SV_OK) return st;
    if (sh->old < 1 || sh->batch < 1 || sh->beams < 0 || sh->max_pages < 1) return SV_ERR_INVALID_ARGUMENT;
    if (sh->beams > 0 && (sh->batch % sh->beams != 0 || sh->old % sh->beams != 0)) return SV_ERR_INVALID_ARGUMENT;
    if ((sh->old > 1 && sh->table_stride < sh->max_pages) || (sh->batch > 1 && sh->out_table_stride < sh->max_pages))
        return SV_ERR_INVALID_ARGUMENT;
    if ((int64_t)sh->max_pages * sh->pool.page_size > kMaxPositions ||
        (int64_t)sh->old * sh->max_pages > INT32_MAX || (int64_t)sh->batch * sh->max_pages > INT32_MAX)
        return SV_ERR_UNSUPPORTED;
    if (sh->table_stride > INT64_MAX / 8 / sh->old || sh->out_table_stride > INT64_MAX / 8 / sh->batch)
        return SV_ERR_UNSUPPORTED;
    const int64_t cols = columns_of(sh->pool, vecb);
    if (cols < 0 || cols > INT32_MAX / sh->pool.page_size) return SV_ERR_UNSUPPORTED;
    const int64_t tiles = std::min((cols * sh->pool.page_size + sv::kThreads - 1) / sv::kThreads, kForkTiles);
    if (!launchable((double)tiles * sh->batch, sv::kThreads)) return SV_ERR_UNSUPPORTED;
    const ForkPlan p = fork_plan(sh);
    if (workspace == nullptr) {
        *workspace_bytes = p.bytes;
        return SV_OK;
    }
    if (data == nullptr || page_table == nullptr || lengths == nullptr || refs == nullptr || out_table == nullptr ||
        out_refs == nullptr || out_free == nullptr)
        return SV_ERR_INVALID_ARGUMENT;
    const struct {
        const int32_t* p;
        int64_t bytes;
    } inputs[] = {{page_table, table_bytes(sh->old, sh->table_stride, sh->max_pages)},
                  {lengths, sh->old * 4ll},
                  {parents, sh->batch * 4ll},
                  {new_lengths, sh->batch * 4ll},
                  {refs, sh->pool.pages * 4ll}},
      outputs[] = {{out_table, table_bytes(sh->batch, sh->out_table_stride, sh->max_pages)},
                   {out_refs, sh->pool.pages * 4ll},
                   {out_free, 4}};
    for (const auto& in : inputs) {
        if (!aligned(in.p, 4) || overlap(in.p, in.bytes, data, extent)) return SV_ERR_INVALID_ARGUMENT;
        for (const auto& o : outputs)
            if (!(in.p == refs && o.p == refs) && overlap(in.p, in.bytes, o.p, o.bytes)) return SV_ERR_INVALID_ARGUMENT;
    }
    for (int i = 0; i < 3; ++i) {
        if (!aligned(outputs[i].p, 4) || overlap(outputs[i].p, outputs[i].bytes, data, extent))
            return SV_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (overlap(outputs[i].p, outputs[i].bytes, outputs[j].p, outputs[j].bytes)) return SV_ERR_INVALID_ARGUMENT;
    }
    if (!aligned(workspace, kAlign)) return SV_ERR_INVALID_ARGUMENT;
    if (*workspace_bytes < p.bytes) return SV_ERR_WORKSPACE_TOO_SMALL;
    const sv::ForkArgs a{pool_args(sh->pool, data, vecb), page_table, lengths, parents, new_lengths, refs, out_table,
                         out_refs, out_free, sh->table_stride, sh->out_table_stride, sh->old, sh->batch, sh->beams,
                         sh->max_pages, (uint32_t)(sh->pool.slabs * sh->pool.heads), (uint32_t)tiles,
                         ws_at<sv::ForkPlace>(workspace, p.off_places), ws_at<int32_t>(workspace, p.off_first),
                         ws_at<int32_t>(workspace, p.off_fresh), ws_at<int32_t>(workspace, p.off_left),
                         (int32_t)p.fresh};
    const int64_t entries = ((int64_t)sh->old + sh->batch) * sh->max_pages;
    if (entries <= kForkSmall && sh->pool.pages <= sv::kPlanPages && sh->batch <= sv::kPlanThreads) {
        hipLaunchKernelGGL(sv::fork_small_kernel, dim3(1), dim3(sv::kPlanThreads), 0, stream, a);
    } else {
        const auto grid = [](int64_t n) { return dim3((uint32_t)std::min<int64_t>((n + sv::kThreads - 1) / sv::kThreads, 2048)); };
        if (out_refs != refs) {
            hipLaunchKernelGGL(sv::fork_refs_kernel, grid(sh->pool.pages), dim3(sv::kThreads), 0, stream, a);
            if (launch_status() != SV_OK) return SV_ERR_HIP;
        }
        hipLaunchKernelGGL(sv::fork_count_kernel, grid(entries), dim3(sv::kThreads), 0, stream, a);
        if (launch_status() != SV_OK) return SV_ERR_HIP;
        hipLaunchKernelGGL(sv::fork_plan_kernel, dim3(1), dim3(sv::kPlanThreads), 0, stream, a);
    }
    if (launch_status() != SV_OK) return SV_ERR_HIP;
    by_piece(vecb, [&](auto v) {
        launch_stream(prof, sv::fork_write_kernel<decltype(v)::value>, (uint32_t)(tiles * sh->batch), stream, a);
    });
    return launch_status();
}

}  // namespace

extern "C" {

sv_status_t spec_cache_compact(const sv_compact_shape_t* shape, void* data, const int32_t* lengths, const int32_t* path,
                               const int32_t* num_accepted, int32_t* out_lengths, hipStream_t stream)
{
    return cache_compact_common(shape, data, lengths, path, num_accepted, out_lengths, stream, nullptr);
}

sv_status_t spec_cache_compact_profiled(const sv_profile_events_t* events, const sv_compact_shape_t* shape, void* data,
                                        const int32_t* lengths, const int32_t* path, const int32_t* num_accepted,
                                        int32_t* out_lengths, hipStream_t stream)
{
    return cache_compact_common(shape, data, lengths, path, num_accepted, out_lengths, stream, events);
}

sv_status_t spec_page_fork(const sv_fork_shape_t* shape, void* data, const int32_t* page_table, const int32_t* lengths,
                           const int32_t* parents, const int32_t* new_lengths, const int32_t* refs, int32_t* out_table,
                           int32_t* out_refs, int32_t* out_free, void* workspace, size_t* workspace_bytes,
                           hipStream_t stream)
{
    return page_fork_common(shape, data, page_table, lengths, parents, new_lengths, refs, out_table, out_refs, out_free,
                            workspace, workspace_bytes, stream, nullptr);
}

sv_status_t spec_page_fork_profiled(const sv_profile_events_t* events, const sv_fork_shape_t* shape, void* data,
                                    const int32_t* page_table, const int32_t* lengths, const int32_t* parents,
                                    const int32_t* new_lengths, const int32_t* refs, int32_t* out_table,
                                    int32_t* out_refs, int32_t* out_free, void* workspace, size_t* workspace_bytes,
                                    hipStream_t stream)
{
    return page_fork_common(shape, data, page_table, lengths, parents, new_lengths, refs, out_table, out_refs, out_free,
                            workspace, workspace_bytes, stream, events);
}

}  // extern "C"
