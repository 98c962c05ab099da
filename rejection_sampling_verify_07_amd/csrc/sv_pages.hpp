// Caches in pages: accepted rows moved behind the context (compact), and page
// tables of sequences that continue others (fork).
//
// Both move bytes and are bound by HBM where there are many, by their launches
// where there are few.  compact: 64 sequences of up to 8 taken rows, 64 caches of rows
// of 2 KB, 66 MB read and written: 14 us, 4.7 TB/s; one sequence 4.8 us.  fork: 64 places
// on 859 pages, 89 MB: 24 us (plan 5.6, copies 17 at 5.2 TB/s); 4 places 8.3 us.
#pragma once

#include "sv_common.hpp"
#include "sv_reorder.hpp"

namespace sv {

// pool[slab][page][head][position in page][piece], strides in bytes.
struct Pool {
    char* data;
    int64_t slab, page, head, pos;
    int32_t pages, page_size;
    uint32_t heads, pieces;  // pieces: of VECB bytes per row
};

// ---------------------------------------------------------------------------
// compact: position first + i takes position first + path[i], i = 1 .. n.
// path rises strictly, so path[i] >= i: a thread that owns one column (a piece
// of one slab and head) reads each source before any later store can reach it,
// and needs no scratch.  Leading entries with path[i] = i do not move.
// ---------------------------------------------------------------------------
constexpr int kCompactMost = 128;  // guesses of a sequence
constexpr int kCompactAhead = 8;   // rows in flight per thread

struct CompactArgs {
    Pool pool;
    const int32_t *cu, *table, *lengths, *path, *nacc;
    int32_t* out_lengths;
    int64_t table_stride;
    int32_t batch, kmax, total_draft, max_pages;
    uint32_t cols, tiles;  // columns of a sequence: slabs * heads * pieces; workgroups for them
};

template <int VECB>
__global__ __launch_bounds__(kThreads) void compact_kernel(CompactArgs a)
{
    typedef typename Piece<VECB>::type T;
    __shared__ int64_t s_from[kCompactMost], s_to[kCompactMost];  // byte offsets; s_from < 0: no move
    __shared__ int32_t s_end;                                     // the first path entry that does not rise
    const int32_t b = (int32_t)(blockIdx.x / a.tiles), tile = (int32_t)(blockIdx.x % a.tiles);
    const int tid = (int)threadIdx.x;
    const int64_t most = (int64_t)a.max_pages * a.pool.page_size;
    const int32_t len = a.lengths != nullptr ? (int32_t)min((int64_t)max(a.lengths[b], 0), most) : (int32_t)most;
    int32_t k0 = b * a.kmax, kb = a.kmax, n = a.nacc[b];
    if (a.cu != nullptr) {
        k0 = a.cu[b];
        const int32_t k1 = a.cu[b + 1];
        kb = k1 - k0;
        if (k0 < 0 || kb < 0 || kb > a.kmax || k1 > a.total_draft) n = -1;
    }
    if (n < 0 || n > kb) {
        if (tile == 0 && tid == 0) a.out_lengths[b] = len;
        return;
    }
    const int32_t first = len - 1 - kb;
    if (tile == 0 && tid == 0) a.out_lengths[b] = max(first + 1 + n, 0);
    if (n == 0) return;
    const int32_t* path = a.path + k0 + b;
    if (tid == 0) s_end = n + 1;
    __syncthreads();
    if (tid < n) {  // entry i = tid + 1
        const int32_t i = tid + 1, p = path[i];
        if (p <= path[i - 1] || p > kb || (i == 1 && path[0] != 0)) atomicMin(&s_end, i);
        const int32_t from = first + p, to = first + i;
        int64_t f = -1, t = 0;
        if (to >= 0 && p > i && p <= kb) {
            const int32_t fp = from / a.pool.page_size, tp = to / a.pool.page_size;
            const int32_t* row = a.table + (int64_t)b * a.table_stride;
            const int32_t fpage = a.table != nullptr ? row[fp] : b, tpage = a.table != nullptr ? row[tp] : b;
            if ((uint32_t)fpage < (uint32_t)a.pool.pages && (uint32_t)tpage < (uint32_t)a.pool.pages) {
                f = fpage * a.pool.page + (int64_t)(from - fp * a.pool.page_size) * a.pool.pos;
                t = tpage * a.pool.page + (int64_t)(to - tp * a.pool.page_size) * a.pool.pos;
            }
        }
        s_from[tid] = f;
        s_to[tid] = t;
    }
    __syncthreads();
    const int32_t moves = min(n, s_end - 1);
    const uint32_t col = (uint32_t)tile * kThreads + (uint32_t)tid;
    if (col >= a.cols) return;
    const uint32_t piece = col % a.pool.pieces, sh = col / a.pool.pieces;
    char* base = a.pool.data + (int64_t)(sh / a.pool.heads) * a.pool.slab + (int64_t)(sh % a.pool.heads) * a.pool.head +
                 (int64_t)piece * VECB;
    for (int32_t i0 = 0; i0 < moves; i0 += kCompactAhead) {
        T v[kCompactAhead];
#pragma unroll
        for (int j = 0; j < kCompactAhead; ++j)
            if (i0 + j < moves && s_from[i0 + j] >= 0) v[j] = *(const SV_GLOBAL T*)(base + s_from[i0 + j]);
#pragma unroll
        for (int j = 0; j < kCompactAhead; ++j)
            if (i0 + j < moves && s_from[i0 + j] >= 0) *(SV_GLOBAL T*)(base + s_to[i0 + j]) = v[j];
    }
}

// ---------------------------------------------------------------------------
// fork.  Reference counts change by integer atomics, whose order does not
// matter; pages are given out by prefix sums, so every result is the same on
// every run.  Three steps: counts without the old tables and with the shared
// pages; one workgroup that decides per place and lists the free pages; tables
// and copies.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / kWave;
constexpr int kListAhead = 8;   // counts in flight per thread while free pages are listed
constexpr int kCountAhead = 4;  // table entries in flight per thread while they are counted

struct ForkPlace {
    int32_t source;  // the sequence it continues, -1: none
    int32_t full;    // shared whole pages
    int32_t rest;    // positions in the page that is still written
    int32_t open;    // that page (-1: none)
    int32_t begin;   // pages taken over: full, and the open page where it is kept
    int32_t need;    // pages of the new table
    int32_t start;   // rank of its first fresh page
    int32_t pad;
};

struct ForkArgs {
    Pool pool;
    const int32_t *table, *lengths, *parents, *new_lengths, *refs;
    int32_t *out_table, *out_refs, *out_free;
    int64_t table_stride, out_stride;
    int32_t old, batch, beams, max_pages;
    uint32_t slices, tiles;  // slabs * heads; copying workgroups per place
    ForkPlace* places;
    int32_t *first, *fresh, *left;  // the lowest place of an open page; free pages; how many were listed
    int32_t fresh_most;             // entries of `fresh`
};

__device__ __forceinline__ int32_t fork_source(const ForkArgs& a, int32_t w)
{
    int32_t s = a.parents != nullptr ? a.parents[w] : w;
    if (a.beams > 0 && a.parents != nullptr) s = s >= 0 && s < a.beams ? w / a.beams * a.beams + s : -1;
    return s >= 0 && s < a.old ? s : -1;
}

__device__ __forceinline__ int32_t fork_length(const ForkArgs& a, int32_t s)
{
    return (int32_t)min((int64_t)max(a.lengths[s], 0), (int64_t)a.max_pages * a.pool.page_size);
}

// Values that the workgroup's other waves change by atomics: past the L1.
__device__ __forceinline__ int32_t ld_agent(const int32_t* p)
{
    return __hip_atomic_load((const SV_GLOBAL int32_t*)p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st_agent(int32_t* p, int32_t v)
{
    __hip_atomic_store((SV_GLOBAL int32_t*)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void add_agent(int32_t* p, int32_t v)
{
    __hip_atomic_fetch_add((SV_GLOBAL int32_t*)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void fork_copy_refs(const ForkArgs& a, int64_t i, int64_t threads)
{
    if (a.out_refs == a.refs) return;
    for (; i < a.pool.pages; i += threads) st_agent(a.out_refs + i, a.refs[i]);
}

__device__ __forceinline__ void fork_count(const ForkArgs& a, int64_t i, int64_t threads)
{
    const int64_t gone = (int64_t)a.old * a.max_pages, all = gone + (int64_t)a.batch * a.max_pages;
    for (; i < all; i += threads) {
        int32_t page, by = -1;
        if (i < gone) {
            const int32_t s = (int32_t)(i / a.max_pages);
            page = a.table[(int64_t)s * a.table_stride + (i - (int64_t)s * a.max_pages)];
        } else {
            const int32_t w = (int32_t)((i - gone) / a.max_pages), at = (int32_t)((i - gone) - (int64_t)w * a.max_pages);
            const int32_t s = fork_source(a, w);
            if (s < 0 || at >= fork_length(a, s) / a.pool.page_size) continue;
            page = a.table[(int64_t)s * a.table_stride + at];
            by = 1;
        }
        if ((uint32_t)page < (uint32_t)a.pool.pages) add_agent(a.out_refs + page, by);
    }
}

__global__ __launch_bounds__(kThreads) void fork_refs_kernel(ForkArgs a)
{
    fork_copy_refs(a, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
}
__global__ __launch_bounds__(kThreads) void fork_count_kernel(ForkArgs a)
{
    fork_count(a, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
}

// Exclusive prefix sum over the workgroup, and its total.
__device__ __forceinline__ int32_t plan_scan(int32_t v, int32_t* s_wave, int32_t* total)
{
    const int32_t incl = wave_incl_scan_int(v);
    __syncthreads();  // (s_wave's last readers are done)
    if (lane_id() == kWave - 1) s_wave[wave_id()] = incl;
    __syncthreads();
    int32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
        const int32_t x = s_wave[w];
        before += w < wave_id() ? x : 0;
        all += x;
    }
    *total = all;
    return before + incl - v;
}

// One of up to `steps` runs of 64 pages per wave from page p0 on: lane i keeps the free ones of the wave's i-th run,
// `free(page)` says which are; they are listed behind the `listed` found before, each run by all lanes at once (the lane
// that holds a run writing its up to 64 pages one by one took 3.4 of the small plan's 10 us).  All threads call it.
template <class Free>
__device__ __forceinline__ int32_t list_free(const ForkArgs& a, int64_t p0, int32_t steps, int32_t listed, int32_t* s_wave,
                                             Free free)
{
    const int64_t base = p0 + (int64_t)wave_id() * steps * kWave;
    uint64_t mine = 0;
    for (int i0 = 0; i0 < steps; i0 += kListAhead) {
        bool is[kListAhead];
#pragma unroll
        for (int j = 0; j < kListAhead; ++j) {
            const int64_t page = base + (i0 + j) * kWave + lane_id();
            is[j] = i0 + j < steps && page < a.pool.pages && free((int32_t)page);
        }
#pragma unroll
        for (int j = 0; j < kListAhead; ++j) {
            const uint64_t m = __ballot(is[j]);
            if (lane_id() == i0 + j) mine = m;
        }
    }
    int32_t all;
    const int32_t rank = listed + plan_scan(__popcll(mine), s_wave, &all);
    for (int i = 0; i < steps; ++i) {
        const uint64_t m = (uint64_t)__shfl((long long)mine, i);
        const int32_t at = __shfl(rank, i) + __popcll(m & ((1ull << lane_id()) - 1));
        if ((m >> lane_id() & 1) && at < a.fresh_most) a.fresh[at] = (int32_t)(base + i * kWave + lane_id());
    }
    return all;
}

// The plan where one workgroup holds all counts in LDS and a place per thread: the counts are formed here too.  Its
// steps wait for memory three times (parents, lengths, tables): 64 places of 17 pages, 859 pages: 6 us.
constexpr int kPlanPages = 8192;
__global__ __launch_bounds__(kPlanThreads) void fork_small_kernel(ForkArgs a)
{
    __shared__ int32_t s_refs[kPlanPages], s_first[kPlanPages], s_source[kPlanThreads], s_full[kPlanThreads];
    __shared__ int32_t s_wave[kPlanWaves];
    const int32_t tid = (int32_t)threadIdx.x;
    ForkPlace p{-1, 0, 0, -1, 0, 0, 0, 0};
    if (tid < a.batch) p.source = fork_source(a, tid);
    for (int32_t i = tid; i < a.pool.pages; i += kPlanThreads) {
        s_refs[i] = a.refs[i];
        s_first[i] = INT32_MAX;
    }
    if (p.source >= 0) {
        const int32_t len = fork_length(a, p.source);
        p.full = len / a.pool.page_size;
        p.rest = len - p.full * a.pool.page_size;
        int64_t want = len;
        if (a.new_lengths != nullptr) want = max(want, (int64_t)a.new_lengths[tid]);
        p.need = (int32_t)min((want + a.pool.page_size - 1) / a.pool.page_size, (int64_t)a.max_pages);
    }
    s_source[tid] = p.source;
    s_full[tid] = p.full;
    __syncthreads();
    if (p.rest > 0) {
        const int32_t page = a.table[(int64_t)p.source * a.table_stride + p.full];
        if ((uint32_t)page < (uint32_t)a.pool.pages) p.open = page;
    }
    // the old tables' entries go, those of the shared pages come
    const uint32_t cols = (uint32_t)a.max_pages, all = cols * (uint32_t)(a.old + a.batch);
    for (uint32_t i0 = (uint32_t)tid; i0 < all; i0 += kCountAhead * kPlanThreads) {
        int32_t page[kCountAhead];
        bool gone[kCountAhead];
#pragma unroll
        for (int j = 0; j < kCountAhead; ++j) {
            const uint32_t i = i0 + j * kPlanThreads, row = i / cols, col = i - row * cols;
            page[j] = -1;
            gone[j] = row < (uint32_t)a.old;
            if (i >= all) continue;
            const int32_t s = gone[j] ? (int32_t)row : s_source[row - a.old];
            if (gone[j] || (s >= 0 && (int32_t)col < s_full[row - a.old]))
                page[j] = a.table[(int64_t)s * a.table_stride + col];
        }
#pragma unroll
        for (int j = 0; j < kCountAhead; ++j)
            if ((uint32_t)page[j] < (uint32_t)a.pool.pages) atomicAdd(&s_refs[page[j]], gone[j] ? -1 : 1);
    }
    if (p.open >= 0) atomicMin(&s_first[p.open], tid);
    __syncthreads();
    // a page that is still written stays with the first place that takes it, if nobody else holds it
    const bool keeps = p.open >= 0 && s_first[p.open] == tid && s_refs[p.open] == 0;
    p.begin = p.full + (keeps ? 1 : 0);
    int32_t want;
    p.start = plan_scan(tid < a.batch ? p.need - p.begin : 0, s_wave, &want);
    if (keeps) s_refs[p.open] = 1;
    if (tid < a.batch) a.places[tid] = p;
    __syncthreads();
    const int32_t steps = (a.pool.pages + kPlanThreads - 1) / kPlanThreads;
    const int32_t listed = list_free(a, 0, steps, 0, s_wave, [&](int32_t page) { return s_refs[page] == 0; });
    for (int32_t i = tid; i < a.pool.pages; i += kPlanThreads) a.out_refs[i] = s_refs[i];
    if (tid == 0) {
        *a.out_free = listed - want;
        *a.left = min(listed, a.fresh_most);
    }
}

// The plan of any size, from counts that launches before it have formed.
__global__ __launch_bounds__(kPlanThreads) void fork_plan_kernel(ForkArgs a)
{
    __shared__ int32_t s_wave[kPlanWaves];
    const int32_t tid = (int32_t)threadIdx.x;
    for (int32_t w = tid; w < a.batch; w += kPlanThreads) {
        ForkPlace p{fork_source(a, w), 0, 0, -1, 0, 0, 0, 0};
        if (p.source >= 0) {
            const int32_t len = fork_length(a, p.source);
            p.full = len / a.pool.page_size;
            p.rest = len - p.full * a.pool.page_size;
            int64_t want = len;
            if (a.new_lengths != nullptr) want = max(want, (int64_t)a.new_lengths[w]);
            p.need = (int32_t)min((want + a.pool.page_size - 1) / a.pool.page_size, (int64_t)a.max_pages);
            if (p.rest > 0) {
                const int32_t page = a.table[(int64_t)p.source * a.table_stride + p.full];
                if ((uint32_t)page < (uint32_t)a.pool.pages) {
                    p.open = page;
                    st_agent(a.first + page, INT32_MAX);
                }
            }
        }
        a.places[w] = p;  // (read again by this thread alone, and by later launches)
    }
    wait_stores();
    __syncthreads();
    for (int32_t w = tid; w < a.batch; w += kPlanThreads) {
        const int32_t open = a.places[w].open;
        if (open >= 0)
            __hip_atomic_fetch_min((SV_GLOBAL int32_t*)(a.first + open), w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    wait_stores();
    __syncthreads();
    int32_t want = 0;  // fresh pages of the places so far
    for (int32_t w0 = 0; w0 < a.batch; w0 += kPlanThreads) {
        const int32_t w = w0 + tid;
        int32_t mine = 0, begin = 0;
        if (w < a.batch) {
            const ForkPlace p = a.places[w];
            begin = p.full;
            // (only the lowest place of a page looks at its count: nobody else changes that now)
            if (p.open >= 0 && ld_agent(a.first + p.open) == w && ld_agent(a.out_refs + p.open) == 0) {
                st_agent(a.out_refs + p.open, 1);
                ++begin;
            }
            mine = p.need - begin;
        }
        int32_t all;
        const int32_t before = plan_scan(mine, s_wave, &all);
        if (w < a.batch) {
            a.places[w].begin = begin;
            a.places[w].start = want + before;
        }
        want += all;
    }
    wait_stores();
    __syncthreads();
    // free pages in rising order
    const int32_t steps = min(kWave, (a.pool.pages + kPlanThreads - 1) / kPlanThreads);
    int32_t listed = 0;
    for (int64_t p0 = 0; p0 < a.pool.pages; p0 += (int64_t)steps * kPlanThreads)
        listed += list_free(a, p0, steps, listed, s_wave, [&](int32_t page) { return ld_agent(a.out_refs + page) == 0; });
    if (tid == 0) {
        *a.out_free = listed - want;
        *a.left = min(listed, a.fresh_most);
    }
}

// Tables, counts of the fresh pages, and the copies of pages still written.
template <int VECB>
__global__ __launch_bounds__(kThreads) void fork_write_kernel(ForkArgs a)
{
    typedef typename Piece<VECB>::type T;
    const int32_t w = (int32_t)(blockIdx.x / a.tiles);
    const uint32_t tile = blockIdx.x % a.tiles;
    const ForkPlace p = a.places[w];
    const int32_t left = *a.left;
    if (tile == 0) {
        const int32_t* from = a.table + (int64_t)max(p.source, 0) * a.table_stride;
        int32_t* to = a.out_table + (int64_t)w * a.out_stride;
        for (int32_t i = (int32_t)threadIdx.x; i < a.max_pages; i += kThreads) {
            int32_t page = -1;
            if (i < p.begin) {
                page = from[i];
            } else if (i < p.need) {
                const int32_t rank = p.start + i - p.begin;
                if (rank < left) {
                    page = a.fresh[rank];
                    a.out_refs[page] = 1;
                }
            }
            to[i] = page;
        }
    }
    if (p.open < 0 || p.begin > p.full || p.start >= left) return;
    const int32_t dst = a.fresh[p.start];
    const char* src_page = a.pool.data + p.open * a.pool.page;
    char* dst_page = a.pool.data + dst * a.pool.page;
    const uint32_t per = (uint32_t)p.rest * a.pool.pieces;  // pieces of one slab and head
    const uint64_t all = (uint64_t)per * a.slices;
    constexpr int kAhead = 4;
    const uint64_t step = (uint64_t)a.tiles * kThreads;
    for (uint64_t x0 = (uint64_t)tile * kThreads + threadIdx.x; x0 < all; x0 += kAhead * step) {
        T v[kAhead];
        int64_t at[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint64_t x = x0 + j * step;
            if (x >= all) continue;
            const uint32_t slice = (uint32_t)x / per, in = (uint32_t)x - slice * per;
            const uint32_t pos = in / a.pool.pieces, piece = in - pos * a.pool.pieces;
            at[j] = (int64_t)(slice / a.pool.heads) * a.pool.slab + (int64_t)(slice % a.pool.heads) * a.pool.head +
                    (int64_t)pos * a.pool.pos + (int64_t)piece * VECB;
            v[j] = *(const SV_GLOBAL T*)(src_page + at[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (x0 + j * step < all) *(SV_GLOBAL T*)(dst_page + at[j]) = v[j];
    }
}

}  // namespace sv
