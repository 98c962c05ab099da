// Reorder of beam states, in place: place w of a group takes the state of
// beam parents[w] of the same group,
//     new[slab][g*W + w][head][p][:] = old[slab][g*W + parents[w]][head][p][:]
// for positions p < lengths[g*W + parents[w]]; everything else stays.
//
// One thread owns one column: the same VECB bytes (position p, piece of the
// row) of all W beams.  It loads every source it needs, then stores: no other
// thread touches the column, so the update is in place with no scratch copy,
// each distinct parent's bytes come from HBM once (a parent that several
// places take is read again from L1), and places that keep their state cost
// nothing.  Bound by HBM: distinct moved parents read, moved places written.
// 4.3 GB of caches (8 groups of 8, 5 distinct parents each, of which 4.9 GB are
// read and written): 900 to 960 us, 5.1 to 5.4 TB/s; 162 MB with rows of 180
// bytes (188 MB): 41 us, 4.6 TB/s; 0.9 MB: 4.9 us, the launch.
#pragma once

#include "sv_common.hpp"

namespace sv {

struct ReorderArgs {
    char* states;
    const int32_t* parents;
    const int32_t* lengths;  // nullptr: every beam holds `positions`
    int32_t beams, heads, positions;
    int64_t slab_stride, beam_stride, head_stride, pos_stride;  // bytes
    uint32_t pieces;  // pieces per row
    uint32_t cols;    // positions * pieces
    uint32_t tiles;   // workgroups per (slab, group, head)
    int32_t slabs;
};

// Pieces of 16, 4, 2 or 1 bytes.  The 16-byte one needs 4-byte alignment only.
template <int VECB>
struct Piece;
template <>
struct Piece<16> {
    typedef u32x4 type __attribute__((aligned(4)));
};
template <>
struct Piece<4> {
    typedef uint32_t type;
};
template <>
struct Piece<2> {
    typedef uint16_t type;
};
template <>
struct Piece<1> {
    typedef uint8_t type;
};

// Loads the sources of places W0 .. MAXW-1 for COLS columns, then stores them.
// One value per level of the recursion: an array of them indexed in two loops
// ended up as a copy of the whole array per place (224 registers for 8 places;
// 1494 us against 1072 us on 4.3 GB of states).
// A column at or past a parent's length is loaded (it lies within the state)
// and not stored.
template <int W0, int MAXW, int COLS, bool NT, class T>
__device__ __forceinline__ void move_columns(char* base, const int64_t (&at)[COLS], const uint32_t (&col)[COLS],
                                             const int64_t (&from)[MAXW], const uint32_t (&lim)[MAXW], int64_t stride)
{
    if constexpr (W0 < MAXW) {
        T v[COLS];
        if (lim[W0] != 0) {
#pragma unroll
            for (int i = 0; i < COLS; ++i) {
                const SV_GLOBAL T* p = (const SV_GLOBAL T*)(base + from[W0] + at[i]);
                if constexpr (NT) v[i] = __builtin_nontemporal_load(p);
                else v[i] = *p;
            }
        }
        move_columns<W0 + 1, MAXW, COLS, NT, T>(base, at, col, from, lim, stride);
        if (lim[W0] != 0) {
#pragma unroll
            for (int i = 0; i < COLS; ++i)
                if (col[i] < lim[W0])
                    __builtin_nontemporal_store(v[i], (SV_GLOBAL T*)(base + (int64_t)W0 * stride + at[i]));
        }
    }
}

// Workgroup: COLS * 256 columns of one (slab, group, head), for up to MAXW places.
template <int VECB, int MAXW, int COLS, bool NT>
__global__ __launch_bounds__(kThreads) void state_reorder_kernel(ReorderArgs a)
{
    typedef typename Piece<VECB>::type T;
    const uint32_t tile = blockIdx.x % a.tiles;
    uint32_t rest = blockIdx.x / a.tiles;
    const uint32_t head = rest % (uint32_t)a.heads;
    rest /= (uint32_t)a.heads;
    const uint32_t slab = rest % (uint32_t)a.slabs;
    const uint32_t g = rest / (uint32_t)a.slabs;
    const int W = a.beams;
    const int32_t* par = a.parents + (int64_t)g * W;
    const int32_t* len = a.lengths != nullptr ? a.lengths + (int64_t)g * W : nullptr;
    // place w moves where its parent is another beam of the group, for columns below the parent's length
    int64_t from[MAXW];
    uint32_t lim[MAXW];
    uint32_t most = 0;
#pragma unroll
    for (int w = 0; w < MAXW; ++w) {
        lim[w] = 0;
        from[w] = 0;
        if (w < W) {
            const int32_t q = par[w];
            if (q >= 0 && q < W && q != w) {
                const int32_t l = len != nullptr ? min(max(len[q], 0), a.positions) : a.positions;
                lim[w] = (uint32_t)l * a.pieces;
                from[w] = (int64_t)q * a.beam_stride;
                most = max(most, lim[w]);
            }
        }
    }
    const uint32_t col0 = tile * (kThreads * COLS);
    if (col0 >= most) return;
    int64_t at[COLS];
    uint32_t col[COLS];
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
        col[i] = col0 + i * kThreads + threadIdx.x;
        const uint32_t c = min(col[i], a.cols - 1);  // past the last column: load that one, store nothing
        const uint32_t p = c / a.pieces;
        at[i] = (int64_t)p * a.pos_stride + (int64_t)(c - p * a.pieces) * VECB;
    }
    char* base = a.states + (int64_t)slab * a.slab_stride + (int64_t)g * W * a.beam_stride +
                 (int64_t)head * a.head_stride;
    move_columns<0, MAXW, COLS, NT, T>(base, at, col, from, lim, a.beam_stride);
}

}  // namespace sv
