// Attention of every sequence's newest rows, a tree of guesses, over the
// sequence's cache in pages.
//
// Row k of sequence b (head h, key/value head h / rep) sees the positions before
// the newest rows and, of those rows, the ones on its way up to row 0:
//     a_j = scale * q . k_j,   out = sum_j exp(a_j - z) v_j,   z = log sum_j exp(a_j).
// Sums over parts of the keys join as in sv_attention.hpp, whose products,
// references and fragment orders are used here.
//
// Work is dealt by what the lengths say on the device, not by what the tables could
// hold: the rounds (64 keys) of all (sequence, key head) pairs form one line, and
// each of a fixed number of workgroups takes an equal stretch of it.  A pair that
// lies within one stretch is finished there; one that crosses borders leaves parts,
// at most two per workgroup, which the join adds up.  The workspace therefore does
// not grow with the caches, and sequences of any mix of lengths keep all CUs busy.
// Where the tables hold few positions a pair is one workgroup's, and nothing is dealt.
//
// Positions come in grains of 16, which never cross a page: a wave finds a grain's
// page with scalar loads, a page ahead.  The four waves of a workgroup share the rows
// of a pair and take tiles of keys through LDS, where loads put them by themselves
// (attend_tree_tiles), three tiles ahead of the products.  Rows that one wave alone
// holds go the same way: the other three only move tiles.  (Each wave walking keys of
// its own, from memory to registers, took 165 us where this takes 146: 48 single rows
// of 32/8 heads of 128 on 4500 positions, 885 MB.)
//
// Few rows are bound by the read of the caches: those 48 rows 6.0 TB/s, with 9 rows each
// 5.3, 16 rows of heads of 256 on 16384 positions 6.9; 48 ragged trees on 1000 to 8000
// positions 169 us, 5.4 TB/s.  There the slowest workgroup ends 15% behind the mean (a
// CU's older workgroup leads, and of two neighbouring XCDs one): shorter stretches or a
// second, finer deal cost in parts and starts what they even out.  Many rows are bound by
// what lies between the products: 16 trees of 64 rows, 32/8 heads of 128, 2048 to 16384
// positions 238 us, 680 TFLOP/s, the matrix cores busy for a third of the time, vector
// instructions issued in two fifths of it; 16/4 heads of 256 411 us, 390 TFLOP/s (a wave
// reads all of a tile from LDS for 16 rows).  Few keys are bound by two launches and four
// trips to memory: 2 rows of 8 heads of 64 on 500 positions 10.4 us (7.5 + 3.0).
#pragma once

#include "sv_attention.hpp"
#include "sv_tree_deal.hpp"

namespace sv {

constexpr int kTreeMostGuesses = 128;
constexpr int kTreeWords = 8;  // a row's view of the newest rows: one word of ones before them, 129 bits, zeros

struct TreeArgs {
    const char *q, *k, *v;
    char* out;
    float* lse;
    int64_t q_row, q_head, out_row, out_head;        // bytes
    int64_t k_page, k_head, v_page, v_head;          // bytes
    int32_t k_pos, v_pos;                            // bytes
    const int32_t *cu, *parents, *lengths, *table;
    int64_t table_stride;
    int32_t batch, rows, kmax, pages, capacity;      // capacity: positions a sequence's pages hold
    int32_t grains_shift;                            // grains per page as a multiplication: (g * mul) >> shift
    uint32_t grains_mul;
    int32_t grains;                                  // per page (without a table: all of a sequence's)
    int32_t q_heads, kv_heads, rep;
    float c;                                         // scale * log2(e)
    int32_t groups, tiles;                           // stretches of the line; row tiles
    bool whole;                                      // a stretch is a pair: no parts, no join
    int32_t* plan;                                   // [batch + 1] rounds before each sequence, the stretch, the extra
    float* acc;                                      // [2 * groups][tile][row][D]
    float2* ml;                                      // [2 * groups][tile][row]
};

// First packed row of sequence b (b = batch: the end of the last one's); entries of cu outside the batch are clamped.
__device__ __forceinline__ int32_t tree_row(const TreeArgs& a, int32_t b)
{
    if (a.cu == nullptr) return b * (a.kmax + 1);
    return min(max(a.cu[b], 0), a.rows - a.batch) + b;
}

__device__ __forceinline__ int32_t tree_length(const TreeArgs& a, int32_t b)
{
    return a.lengths != nullptr ? min(max(a.lengths[b], 0), a.capacity) : a.capacity;
}

// Number of the page that grain g of a sequence lies in.
__device__ __forceinline__ int32_t page_of_grain(const TreeArgs& a, int32_t g)
{
    return (int32_t)(((uint64_t)(uint32_t)g * a.grains_mul) >> a.grains_shift);
}

// What one workgroup works on: a stretch of one (sequence, key head) pair.
struct Stretch {
    const char *k, *v;       // the key head's first page
    const int32_t* table;    // the sequence's row, or nullptr: its one page is `b`
    const int32_t* parents;  // its guesses' parents, or nullptr
    int32_t b, hk, row0, nrows;
    int32_t begin, end;      // keys
    int32_t total;           // positions of the sequence
    int32_t pages;           // pages that they take
    int32_t context;         // those before the newest rows (below 0 if the newest rows are not all there)
};

// The page of grain g, for the few that are looked up one by one (-1: none; keys at or past `total` have none).
__device__ __forceinline__ int32_t grain_page(const TreeArgs& a, const Stretch& s, int32_t g, int32_t* in_page)
{
    const int32_t at = page_of_grain(a, g);
    *in_page = (g - at * a.grains) * 16;
    if (g * 16 >= s.total) return -1;
    const int32_t page = s.table != nullptr ? s.table[at] : s.b;
    return (uint32_t)page < (uint32_t)a.pages ? page : -1;
}

// A scalar load: the tables are not written while a kernel reads them.  (A vector load that a loop carries along keeps
// the compiler from letting the tiles' loads run ahead: it waits for all of them.)
__device__ __forceinline__ int32_t scalar_load(const int32_t* p)
{
    return *(const __attribute__((address_space(4))) int32_t*)p;
}

// Walks all grains of a stretch in order: where the next one's keys and values lie.  Within a page a step is an
// addition per pointer; the next page's number is asked for a page ahead.  (Scalar work: it runs beside the products in
// every wave, and with each grain's place worked out anew it was half of the instructions.)
struct KeyWalk {
    const char *k, *v;
    int32_t left;    // grains of the page from here on
    int32_t page;    // -1: none (the pointers then lie in the pool's first page)
    int32_t number;  // of the page after this one
    int32_t asked;   // that page, as the table says

    __device__ __forceinline__ void ask(const Stretch& s)
    {
        if (s.table != nullptr) asked = scalar_load(s.table + min(number, s.pages - 1));
    }
    __device__ __forceinline__ void open(const TreeArgs& a, const Stretch& s)
    {
        page = (uint32_t)asked < (uint32_t)a.pages ? asked : -1;
        const int64_t at = max(page, 0);
        k = s.k + at * a.k_page;
        v = s.v + at * a.v_page;
        left = a.grains;
        ++number;
        ask(s);
    }
    __device__ __forceinline__ void start(const TreeArgs& a, const Stretch& s, int32_t key)
    {
        number = page_of_grain(a, key / 16);
        const int32_t in = key / 16 - number * a.grains;
        asked = s.b;
        ask(s);
        open(a, s);
        k += (int64_t)in * 16 * a.k_pos;
        v += (int64_t)in * 16 * a.v_pos;
        left -= in;
    }
    __device__ __forceinline__ void step(const TreeArgs& a, const Stretch& s)
    {
        if (--left > 0) {
            k += 16 * a.k_pos;
            v += 16 * a.v_pos;
        } else {
            open(a, s);
        }
    }
};

// The rows that rows t0 .. t0 + n - 1 of the sequence see among the newest ones, as
// bits from the sequence's row 0 on.  All threads of the workgroup call it.
__device__ __forceinline__ void tree_views(const Stretch& s, int32_t t0, int32_t n, int32_t* s_up, uint32_t* s_view)
{
    const int tid = (int)threadIdx.x;
    if (s.parents != nullptr) {
        for (int32_t j = tid; j < s.nrows - 1; j += kAttnThreads) s_up[j] = s.parents[j];
        __syncthreads();
    }
    for (int32_t i = tid; i < n; i += kAttnThreads) {
        uint32_t w[kTreeWords] = {~0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
        int32_t r = t0 + i;
        if (s.parents == nullptr) {  // a chain: all rows up to r
#pragma unroll
            for (int x = 0; x < 5; ++x) w[x + 1] = r >= x * 32 + 31 ? ~0u : r >= x * 32 ? (2u << (r % 32)) - 1 : 0u;
        } else {
            while (true) {
#pragma unroll
                for (int x = 0; x < 5; ++x) w[x + 1] |= r / 32 == x ? 1u << (r % 32) : 0u;
                if (r == 0) break;
                const int32_t up = s_up[r - 1];
                r = up >= 0 && up < r ? up : 0;
            }
        }
#pragma unroll
        for (int x = 0; x < kTreeWords; ++x) s_view[i * kTreeWords + x] = w[x];
    }
    __syncthreads();
}

// Four bits: whether a row with view `w` sees keys e .. e + 3, counted from the newest rows' first.
__device__ __forceinline__ uint32_t sees4(const uint32_t* w, int32_t e)
{
    if (e < -3) return 15u;  // before the newest rows: every row sees them
    const int32_t at = min((e >> 5) + 1, kTreeWords - 2);
    return (uint32_t)((((uint64_t)w[at + 1] << 32) | w[at]) >> (e & 31)) & 15u;
}
__device__ __forceinline__ bool sees(const uint32_t* w, int32_t e) { return e < 0 || (sees4(w, e) & 1u) != 0; }

// All loads of this wave have arrived, in a form that the compiler counts: before a loop, so that it does not wait in
// every step for what the first one needs.
__device__ __forceinline__ void loads_done()
{
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
}

// Where a finished or partial result of a workgroup goes.
struct TreeOut {
    bool whole;     // no other workgroup has keys of the pair
    int64_t slot;   // (part * tiles + tile) otherwise
};

// Columns n .. n + 3 of a row, normalised and rounded.
template <int DT>
__device__ __forceinline__ void store4(char* p, float x0, float x1, float x2, float x3)
{
    u32x2 w;
    w.x = pack2<DT>(x0, x1);
    w.y = pack2<DT>(x2, x3);
    *(SV_GLOBAL u32x2*)p = w;
}

// Four waves of MT * 16 rows share tiles of keys through LDS, whose rows lie and are read as in TileAttention.  Four
// tiles (64 columns: of 64 keys, 16 KB; 128: of 32, 16 KB; 256: of 32, 32 KB) are on their way or in use: with two of them
// a step lasted as long as a read of memory.  One workgroup per CU with eight buffers, or with tiles of twice the keys,
// instead of two with four: 200 and 157 us, not 150, on 48 single rows of 4500 positions.
template <int D>
struct TreeTile {
    static constexpr int KT = D == 64 ? 64 : 32;           // keys
    static constexpr int BUFS = 4;
    static constexpr int ROW = D * 2;                      // bytes per key row
    static constexpr int CH = ROW / 16;                    // 16-byte chunks per row
    static constexpr int MASK = CH < 16 ? CH - 1 : 15;     // swizzle
    static constexpr int TILE = KT * ROW;                  // bytes of K (or V)
    static constexpr int LOADS = TILE / 16 / kAttnThreads;  // per thread, of K (or V)
    static constexpr int LDS = BUFS * 2 * TILE;
};

__device__ __forceinline__ uint32_t lds_address(const char* p) { return (uint32_t)(uintptr_t)(const SV_LDS char*)p; }

// 16 bytes from each lane's place `off` behind `base` into LDS, lane i's at `to` + 16 i (`to`: the wave's).  In assembly,
// which the compiler does not count among the loads in flight: it would wait for all of them before every transposed
// read of a tile.  arrived() is the wait for them; a wave has none left when its loop over the tiles ends.  (M0 is not
// kept between instructions that take it: nothing else here does.)
template <bool PAST>
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, uint32_t to)
{
    if constexpr (PAST)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(to), "v"(off),
                     "s"((const SV_GLOBAL char*)base)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off),
                     "s"((const SV_GLOBAL char*)base)
                     : "memory");
}

// All but the newest N of this wave's loads have arrived, and what it read of LDS; then all waves have come here.
template <int N>
__device__ __forceinline__ void arrived()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int DT, int D, int MT>
__device__ __forceinline__ void attend_tree_tiles(const TreeArgs& a, const Stretch& st, int32_t tile, const TreeOut& to,
                                                  int32_t* s_up, uint32_t* s_view, int32_t* s_wild, char* s_kv)
{
    typedef TreeTile<D> TA;
    constexpr int ROWS = kAttnWaves * MT * 16;
    constexpr int DC = D / 32, DT16 = D / 16, KT = TA::KT, SUBS = KT / kKeyBlock, GR = KT / 16;
    static_assert(kWave % TA::CH == 0, "a wave's load stays within a grain");
    const int lane = lane_id(), l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int32_t m_total = st.nrows * a.rep;
    const int32_t r0 = tile * ROWS + wave * (MT * 16), t0 = tile * ROWS / a.rep;
    const bool idle = r0 >= m_total;  // no rows: the wave only moves tiles

    f32x4 o[MT][DT16];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = kNoReference;
        l[mt] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT16; ++d) o[mt][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // A tile goes from memory into LDS by itself (a wave's load fills 1 KB in the order of its lanes); the i-th load of a
    // thread has row (i * 256 + thread) / CH and that place's chunk, which the swizzle has moved.  A wave's rows lie in
    // one grain.
    constexpr int RPL = kAttnThreads / TA::CH;  // rows per load
    const int32_t own_row = (int32_t)threadIdx.x / TA::CH, place = (int32_t)threadIdx.x % TA::CH;
    const int32_t half = RPL == 32 ? wave / 2 : 0;                       // (64 columns: two grains per load)
    const int32_t in_grain = RPL == 32 ? own_row - half * 16 : own_row;  // the row in its grain, of the grain's first load
    constexpr int PER = RPL < 16 ? 16 / RPL : 1;                         // (256 columns: two loads per grain)
    uint32_t koff[PER], voff[PER];
#pragma unroll
    for (int x = 0; x < PER; ++x) {
        const int32_t row = in_grain + x * RPL, ch = place ^ ((own_row + x * RPL) & TA::MASK);
        koff[x] = (uint32_t)(row * a.k_pos + ch * 16);
        voff[x] = (uint32_t)(row * a.v_pos + ch * 16);
    }
    KeyWalk walk;
    int32_t kb = st.begin, ahead = st.begin;  // the tile in use, the next one to load
    int32_t bad_from = INT32_MAX;             // the first tile met that has a grain without a page
    uint32_t there = 0;                       // four bits per buffer: the grains of its tile that have pages
    walk.start(a, st, kb);
    // `past`: where no other row tile reads the same keys they go past the caches (48 ragged trees on up to 8000 positions:
    // 169 us, 194 through them; nothing was slower).
    auto load_tile = [&](int buf, auto past) {
        const uint32_t dst = lds_address(s_kv) + (uint32_t)(buf * (2 * TA::TILE) + wave * (kWave * 16));
        const bool edge = ahead + KT > st.total;
        uint32_t pages = 0;
#pragma unroll
        for (int i = 0; i < TA::LOADS; ++i) {
            // this load's grain: pointers before and after a step where it has two
            const char *k = walk.k, *v = walk.v;
            pages |= walk.page >= 0 ? 1u << (i * RPL / 16) : 0u;
            if constexpr (RPL == 32) {
                walk.step(a, st);
                pages |= walk.page >= 0 ? 2u << (i * 2) : 0u;
                k = half != 0 ? walk.k : k;
                v = half != 0 ? walk.v : v;
            }
            const int x = i % PER;
            uint32_t ko = koff[x], vo = voff[x];
            if (edge) {  // the last key stands in for those behind it, the pool's first where a grain has none (masked below)
                const int32_t first = ahead + (i / PER * (RPL == 32 ? 2 : 1) + half) * 16, last = st.total - 1 - first;
                const int32_t row = max(min(in_grain + x * RPL, last), 0), ch = place ^ ((own_row + x * RPL) & TA::MASK);
                ko = (uint32_t)(row * a.k_pos + ch * 16);
                vo = (uint32_t)(row * a.v_pos + ch * 16);
                k = last < 0 ? st.k : k;
                v = last < 0 ? st.v : v;
            }
            load_to_lds<decltype(past)::value>(k, ko, dst + i * (kAttnThreads * 16));
            load_to_lds<decltype(past)::value>(v, vo, dst + TA::TILE + i * (kAttnThreads * 16));
            if (x == PER - 1) walk.step(a, st);
        }
        if (pages != (1u << GR) - 1) bad_from = min(bad_from, ahead);
        there = (there & ~(15u << (buf * 4))) | pages << (buf * 4);
        ahead += KT;
    };
    auto load_next = [&](int buf) {
        if (ahead < st.end) with_policy(a.tiles == 1, [&](auto past) { load_tile(buf, past); });
    };
    // No value for keys past the last one or without a page; one that is not finite counts as 0 here (times the weight 0
    // of a row that does not see it, it would be NaN) and reaches the rows that see it at the end.
    auto clear = [&](int buf, int32_t kb, uint32_t pages) {
        u32x4* v = (u32x4*)(s_kv + buf * (2 * TA::TILE) + TA::TILE) + threadIdx.x;
        bool any = false;
#pragma unroll
        for (int i = 0; i < TA::LOADS; ++i) {
            const bool there = (pages >> (i * RPL / 16 + half) & 1u) != 0 && kb + i * RPL + own_row < st.total;
            u32x4 w = v[i * kAttnThreads];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t y = there ? w[x] : 0u;
                w[x] = finite_halves<DT>(y);
                any |= w[x] != y;
            }
            v[i * kAttnThreads] = w;
        }
        if (__any(any) && lane == 0) *s_wild = 1;
    };

    if (threadIdx.x == 0) *s_wild = 0;
#pragma unroll
    for (int x = 0; x + 1 < TA::BUFS; ++x) load_next(x);
    if (st.end > st.context) tree_views(st, t0, min(st.nrows, ((tile + 1) * ROWS - 1) / a.rep + 1) - t0, s_up, s_view);
    u32x4 qf[MT][DC];
    const uint32_t* view[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int32_t r = r0 + mt * 16 + l16;
        const int32_t t = r / a.rep, h = st.hk * a.rep + (r - t * a.rep);
        const char* qp = a.q + (int64_t)(st.row0 + t) * a.q_row + (int64_t)h * a.q_head + lg * 16;
#pragma unroll
        for (int c = 0; c < DC; ++c)
            qf[mt][c] = r < m_total ? *(const SV_GLOBAL u32x4*)(qp + c * 64) : u32x4{0u, 0u, 0u, 0u};
        view[mt] = s_view + (r < m_total ? t - t0 : 0) * kTreeWords;
    }
    loads_done();
    const bool younger = blockIdx.x >= gridDim.x / 2;
    int buf = 0;
    uint32_t here = 0;    // a masked tile: which grains have pages
    bool masked = false;  // (uniform) from the first tile on that rows see in part, or whose pages are not all there
    int32_t masked_from = st.end;
    bool far = false;  // (uniform over the wave) a reference lies beyond kFarReference
    // A lane's places in a tile: row l16 (+ 16 per group) of K, its chunk c * 4 + lg behind the swizzle; for the values of
    // 32 keys, four rows (lg * 4 + l16 / 4) and 8 bytes of columns per lane before the exchange.  Another chunk or
    // column is an exclusive or away.
    const uint32_t kplace = (uint32_t)(l16 * TA::ROW + ((lg ^ (l16 & TA::MASK)) * 16));
    const int32_t vrow = lg * 4 + (l16 >> 2);
    const uint32_t vplace =
        (uint32_t)(TA::TILE + vrow * TA::ROW + ((((l16 & 3) >> 1) ^ (vrow & TA::MASK)) * 16) + (l16 & 1) * 8);
    u32x4 kf[2 * SUBS][DC];  // the keys of the tile that is next in use: read while the one before it is
    auto read_keys = [&](int buf) {
        const uint32_t at = (uint32_t)(buf * (2 * TA::TILE)) + kplace;
#pragma unroll
        for (int c = 0; c < DC; ++c)
#pragma unroll
            for (int i = 0; i < 2 * SUBS; ++i)
                kf[i][c] = *(const u32x4*)(s_kv + (at ^ (uint32_t)(c * 64)) + i * 16 * TA::ROW);
    };
    auto use = [&](bool more) {
        u32x4 vf[DT16];
        auto read_values = [&](int u) {
            const uint32_t at = (uint32_t)(buf * (2 * TA::TILE)) + vplace;
#pragma unroll
            for (int d = 0; d < DT16; ++d) {
                const char* p = s_kv + (at ^ (uint32_t)(d * 32)) + u * kKeyBlock * TA::ROW;
                const u32x2 v0 = lds_read_transposed(p), v1 = lds_read_transposed(p + 16 * TA::ROW);
                vf[d] = u32x4{v0.x, v0.y, v1.x, v1.y};
            }
        };
        f32x4 s[SUBS][2][MT];
        read_values(0);
#pragma unroll
        for (int i = 0; i < 2 * SUBS; ++i)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) s[i / 2][i & 1][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < DC; ++c)
#pragma unroll
            for (int i = 0; i < 2 * SUBS; ++i)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    s[i / 2][i & 1][mt] = mfma_16x16x32<DT>(kf[i][c], qf[mt][c], s[i / 2][i & 1][mt]);
        // The wave that is past its products goes first, so that one wave of a SIMD multiplies while the other one takes
        // exponentials (16 trees of 64 rows on 9000 positions: 255 us without, 247 with; fewer rows wait for memory).
        if constexpr (MT == 2) __builtin_amdgcn_s_setprio(1);
        if (more) read_keys((buf + 1) % TA::BUFS);
        if (masked) {
#pragma unroll
            for (int i = 0; i < 2 * SUBS; ++i)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t seen = (here >> i & 1u) == 0 ? 0u : sees4(view[mt], kb + i * 16 + lg * 4 - st.context);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if ((seen >> x & 1u) == 0) s[i / 2][i & 1][mt][x] = neg_inf();
                }
        }
        float top[MT];
        bool over = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float x = s[0][0][mt][0];
#pragma unroll
            for (int i = 1; i < 8 * SUBS; ++i) x = fmaxf(x, s[i / 8][(i / 4) & 1][mt][i & 3]);
            top[mt] = x * a.c;
            over |= top[mt] > m[mt] + (Reference<DT>::kBelow + Reference<DT>::kSlack);
        }
        if (__any(over)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float x = top[mt];
                x = fmaxf(x, __shfl_xor(x, 16, kWave));
                x = fmaxf(x, __shfl_xor(x, 32, kWave));
                x = fmaxf(x - Reference<DT>::kBelow, m[mt]);
                const float f = __builtin_amdgcn_exp2f(m[mt] - x);
                m[mt] = x;
                l[mt] *= f;
#pragma unroll
                for (int d = 0; d < DT16; ++d) o[mt][d] *= f;
            }
            far = far_references<MT>(m);
        }
        if (__builtin_expect(far, 0)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 8 * SUBS; ++i) {
                    f32x4& x = s[i / 8][(i / 4) & 1][mt];
                    x[i & 3] = far_distance(x[i & 3], a.c, m[mt]);
                }
        }
        const float c = far ? 1.0f : a.c;
#pragma unroll
        for (int u = 0; u < SUBS; ++u) {
            u32x4 pf[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float ref = far ? 0.0f : m[mt];
                float p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][i / 4][mt][i & 3], c, -ref));
                    l[mt] += p[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) pf[mt][i] = pack2<DT>(p[2 * i], p[2 * i + 1]);
            }
            if constexpr (MT == 2) __builtin_amdgcn_s_setprio(0);
#pragma unroll
            for (int d = 0; d < DT16; ++d)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) o[mt][d] = mfma_16x16x32<DT>(vf[d], pf[mt], o[mt][d]);
            if (u + 1 < SUBS) read_values(u + 1);
        }
    };
    arrived<0>();  // (the other waves' loads too)
    if (!idle) read_keys(0);
    while (kb < st.end) {
        // the tile after this one has arrived (the one behind it need not have), and all waves have left the one before
        // this, whose place the next load takes
        if (kb + (TA::BUFS - 2) * KT < st.end) arrived<2 * TA::LOADS * (TA::BUFS - 3)>();
        else arrived<0>();
        load_next((buf + TA::BUFS - 1) % TA::BUFS);
        // The older of a CU's two workgroups goes first where both could: the younger one leads in three tiles of four,
        // or it ends 10% later (the line is dealt evenly).  With more rows the products are what counts: no gain.
        if constexpr (MT == 1 && D != 256) {
            if (younger && (kb / KT & 3) != 0) __builtin_amdgcn_s_setprio(1);
            else __builtin_amdgcn_s_setprio(0);
        }
        if (!masked && (kb + KT > st.context || kb >= bad_from)) {
            masked = true;
            masked_from = kb;
        }
        if (masked) {
            here = there >> (buf * 4);
            clear(buf, kb, here);
            __syncthreads();
        }
        if (!idle) use(kb + KT < st.end);
        kb += KT;
        buf = (buf + 1) % TA::BUFS;
    }
    const bool wild = *s_wild != 0;  // (written before a barrier that all waves have passed)
    if (idle) return;
    if (wild) {
#pragma unroll 1
        for (int32_t x = masked_from; x < st.end; ++x) {
            int32_t in;
            const int32_t page = grain_page(a, st, x / 16, &in);
            if (page < 0) continue;
            const char* row = st.v + page * a.v_page + (int64_t)(in + x % 16) * a.v_pos;
            bool see[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) see[mt] = sees(view[mt], x - st.context);
            // accumulator i of tile d holds column d * 16 + lg * 4 + i
#pragma unroll
            for (int d = 0; d < DT16; ++d) {
                const u32x2 w = *(const SV_GLOBAL u32x2*)(row + (d * 16 + lg * 4) * 2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t bad = w[i / 2] ^ finite_halves<DT>(w[i / 2]);
                    const float v = i % 2 ? hi16<DT>(bad) : lo16<DT>(bad);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        if (see[mt]) o[mt][d][i] += v;
                }
            }
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16, kWave);
        l[mt] += __shfl_xor(l[mt], 32, kWave);
        const int32_t r = r0 + mt * 16 + l16;
        if (r >= m_total) continue;
        const int32_t t = r / a.rep, h = st.hk * a.rep + (r - t * a.rep);
        if (to.whole) {
            const float inv = l[mt] != 0.0f ? 1.0f / l[mt] : 0.0f;
            char* dst = a.out + (int64_t)(st.row0 + t) * a.out_row + (int64_t)h * a.out_head + lg * 8;
#pragma unroll
            for (int d = 0; d < DT16; ++d)
                store4<DT>(dst + d * 32, o[mt][d][0] * inv, o[mt][d][1] * inv, o[mt][d][2] * inv, o[mt][d][3] * inv);
            if (a.lse != nullptr && lg == 0)
                a.lse[(int64_t)(st.row0 + t) * a.q_heads + h] =
                    l[mt] != 0.0f ? (m[mt] + __builtin_amdgcn_logf(l[mt])) * 0.69314718055994531f : neg_inf();
        } else {
            const int64_t at = to.slot * ROWS + wave * (MT * 16) + mt * 16 + l16;
            if (lg == 0) a.ml[at] = float2{m[mt], l[mt]};
            SV_GLOBAL f32x4* dst = (SV_GLOBAL f32x4*)(a.acc + at * D + lg * 4);
#pragma unroll
            for (int d = 0; d < DT16; ++d) dst[d * 4] = o[mt][d];
        }
    }
}

constexpr int kTreeRound = 64;  // keys: what the line of all pairs counts
// A pair counts this many rounds beyond its own, for each 16-row tile of a wave, where stretches have at least
// kTreeExtraFrom: what a stretch's start and end cost (6 and 13 us at 2.4 and 2.9 us a round).  48 single rows on 1000 to
// 8000 positions: 160 us without, 158 with 2, 164 with 4; 16 trees of 64 rows on 8192: 201 with 2, 195 with 4, 201 with 6.
constexpr int kTreeExtra = 2, kTreeExtraFrom = 8;

// The line's length and where a stretch begins, by all threads of the workgroup: thread t sums the sequences t * per
// .. t * per + per - 1.
struct TreeStart {
    int32_t total, stretch;  // rounds of the line, and of one workgroup
    int32_t extra;           // rounds that a pair counts beyond its own
    int32_t b, at;           // the sequence that holds the first round, and the rounds of it before that one
    int32_t len, row0, row1;  // its length, its first row and the next sequence's
};
__device__ __forceinline__ TreeStart tree_start(const TreeArgs& a, int32_t group, int32_t per_pair, bool write, int32_t* s_sum,
                                                int32_t* s_found)
{
    const int32_t tid = (int32_t)threadIdx.x, per = (a.batch + kAttnThreads - 1) / kAttnThreads;
    const int32_t b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    int32_t mine = 0, len = 0, row0 = 0, row1 = 0;
    if (b0 < b1) {  // (asked for together: one trip to memory where every thread has one sequence)
        len = tree_length(a, b0);
        row0 = tree_row(a, b0);
        row1 = tree_row(a, b0 + 1);
        mine = (len + kTreeRound - 1) / kTreeRound * a.kv_heads;
    }
    for (int32_t b = b0 + 1; b < b1; ++b) mine += (tree_length(a, b) + kTreeRound - 1) / kTreeRound * a.kv_heads;
    const int32_t incl = wave_incl_scan_int(mine);
    if (lane_id() == kWave - 1) s_sum[wave_id()] = incl;
    __syncthreads();
    int32_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
        const int32_t x = s_sum[w];
        before += w < wave_id() ? x : 0;
        total += x;
    }
    const int32_t more = total >= kTreeExtraFrom * a.groups ? per_pair : 0;  // (a.groups: 512 at most here)
    const int32_t extra = more * a.kv_heads;                                  // per sequence
    before += extra * b0;
    mine += extra * (b1 - b0);
    total += extra * a.batch;
    const int32_t stretch = deal_stretch(total, a.groups);
    const int64_t from = (int64_t)group * stretch;
    if (write) {
        int32_t sum = before;
        for (int32_t b = b0; b < b1; ++b) {
            a.plan[b] = sum;
            if (b + 1 < b1) sum += (tree_length(a, b) + kTreeRound - 1) / kTreeRound * a.kv_heads + extra;
        }
        if (tid == 0) {
            a.plan[a.batch] = total;
            a.plan[a.batch + 1] = stretch;
            a.plan[a.batch + 2] = more;
        }
    }
    if (from >= before && from < before + mine) {
        int32_t sum = before, b = b0;
        while (true) {
            const int32_t n = (len + kTreeRound - 1) / kTreeRound * a.kv_heads + extra;
            if (from < sum + n) break;
            sum += n;
            len = tree_length(a, ++b);
            row0 = row1;
            row1 = tree_row(a, b + 1);
        }
        s_found[0] = b;
        s_found[1] = (int32_t)(from - sum);
        s_found[2] = len;
        s_found[3] = row0;
        s_found[4] = row1;
    }
    __syncthreads();
    return TreeStart{total, stretch, more, s_found[0], s_found[1], s_found[2], s_found[3], s_found[4]};
}

template <int DT, int D, int MT>
__global__ __launch_bounds__(kAttnThreads, D == 256 ? 1 : 2) void tree_part_kernel(TreeArgs a)
{
    constexpr int ROWS = MT * 16 * kAttnWaves, KB = kTreeRound;
    __shared__ __align__(16) char s_mem[TreeTile<D>::LDS];
    __shared__ uint32_t s_view[ROWS * kTreeWords];
    __shared__ int32_t s_up[kTreeMostGuesses], s_sum[kAttnWaves], s_found[5], s_wild;
    // the row tiles of one stretch (the same keys) run on one XCD (workgroups go to the 8 XCDs in turn)
    const uint32_t x = blockIdx.x & 7u, y = blockIdx.x >> 3;
    const int32_t group = a.tiles == 1 ? (int32_t)blockIdx.x : (int32_t)(y / (uint32_t)a.tiles * 8u + x);
    const int32_t tile = a.tiles == 1 ? 0 : (int32_t)(y % (uint32_t)a.tiles);
    if (group >= a.groups) return;
    int64_t at, end;
    int32_t b, in, extra, len, row0, row1;  // in: rounds of sequence b before `at`
    if (a.whole) {                          // one pair per workgroup (an empty one counts a round)
        b = group / a.kv_heads;
        len = __builtin_amdgcn_readfirstlane(tree_length(a, b));
        row0 = __builtin_amdgcn_readfirstlane(tree_row(a, b));
        row1 = __builtin_amdgcn_readfirstlane(tree_row(a, b + 1));
        extra = len == 0 ? 1 : 0;
        at = 0;
        end = (len + KB - 1) / KB + extra;
        in = (group - b * a.kv_heads) * (int32_t)end;
    } else {
        const TreeStart start = tree_start(a, group, MT * kTreeExtra, group == 0 && tile == 0, s_sum, s_found);
        at = (int64_t)group * start.stretch;
        if (at >= start.total) return;
        end = min(at + start.stretch, (int64_t)start.total);
        b = __builtin_amdgcn_readfirstlane(start.b);
        in = __builtin_amdgcn_readfirstlane(start.at);
        extra = start.extra;
        len = __builtin_amdgcn_readfirstlane(start.len);
        row0 = __builtin_amdgcn_readfirstlane(start.row0);
        row1 = __builtin_amdgcn_readfirstlane(start.row1);
    }
    bool first = true;
    while (at < end) {
        const int32_t n = (len + KB - 1) / KB, pair = n + extra;
        if (in >= pair * a.kv_heads) {  // (also the empty sequences)
            in -= pair * a.kv_heads;
            ++b;
            len = __builtin_amdgcn_readfirstlane(tree_length(a, b));
            row0 = row1;
            row1 = __builtin_amdgcn_readfirstlane(tree_row(a, b + 1));
            continue;
        }
        const int32_t hk = in / pair, j = in - hk * pair;
        const int32_t step = (int32_t)min((int64_t)(pair - j), end - at), take = min(step, n - j);
        Stretch st;
        st.b = b;
        st.hk = hk;
        st.row0 = row0;
        st.nrows = min(row1 - row0, a.kmax + 1);
        st.total = len;
        st.context = len - st.nrows;
        st.begin = j * KB;
        st.end = min((j + take) * KB, len);
        st.pages = a.table != nullptr ? page_of_grain(a, (len - 1) / 16) + 1 : 1;
        st.k = a.k + (int64_t)hk * a.k_head;
        st.v = a.v + (int64_t)hk * a.v_head;
        st.table = a.table != nullptr ? a.table + (int64_t)b * a.table_stride : nullptr;
        st.parents = a.parents != nullptr ? a.parents + (st.row0 - b) : nullptr;
        if ((take > 0 || a.whole) && tile * ROWS < st.nrows * a.rep) {
            __syncthreads();  // (the stretch before this one is done with the LDS)
            const TreeOut to{j == 0 && take == n, ((int64_t)group * 2 + (first ? 0 : 1)) * a.tiles + tile};
            attend_tree_tiles<DT, D, MT>(a, st, tile, to, s_up, s_view, &s_wild, s_mem);
        }
        at += step;
        in += step;
        first = false;
    }
}

// Join of the parts: D / 4 lanes over the columns of a (row, head), whose parts come in batches that are on their way at
// once.  With few rows (SPLIT) the wave's other lanes take parts of the same row, with many another row each.  A pair
// that one workgroup finished is left alone; rows that see nothing get zeros.
template <int DT, int D, int ROWS, bool SPLIT>
__global__ __launch_bounds__(kThreads) void tree_join_kernel(TreeArgs a)
{
    constexpr int LPP = D / 4;                        // lanes per part
    constexpr int PPR = SPLIT ? kWave / LPP : 1;      // parts side by side
    constexpr int PER = kWave / LPP / PPR;            // rows per wave
    const int lane = lane_id(), col = (lane % LPP) * 4, sub = SPLIT ? lane / LPP : 0;
    const int32_t i = ((int32_t)blockIdx.x * kWaves + wave_id()) * PER + (SPLIT ? 0 : lane / LPP);
    const int32_t heads = a.q_heads, ik = i / heads, h = i - ik * heads, b = ik / (a.kmax + 1), k = ik - b * (a.kmax + 1);
    if (b >= a.batch) return;
    const int32_t row0 = tree_row(a, b), nrows = min(tree_row(a, b + 1) - row0, a.kmax + 1);
    const int32_t begin = a.plan[b], pair = (a.plan[b + 1] - begin) / a.kv_heads, stretch = a.plan[a.batch + 1];
    const int32_t rounds = pair - a.plan[a.batch + 2];
    if (k >= nrows) return;
    const int32_t hk = h / a.rep, r = k * a.rep + (h - hk * a.rep), tile = r / ROWS;
    const int32_t from = begin + hk * pair;
    const PairParts held = pair_parts(from, rounds, stretch);
    const int32_t parts = held.count;
    if (parts == 1) return;
    auto place = [&](int32_t p) { return (part_place(held, p) * a.tiles + tile) * ROWS + (r - tile * ROWS); };
    float m = kNoReference, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    auto batch = [&](int32_t p0, auto most) {
        constexpr int N = decltype(most)::value;
        float2 ml[N];
        f32x4 v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t at = place(join_part(parts, p0 + j * PPR + sub));
            ml[j] = a.ml[at];
            v[j] = *(const SV_GLOBAL f32x4*)(a.acc + at * D + col);
            if (p0 + j * PPR + sub >= parts) ml[j] = float2{kNoReference, 0.0f};
        }
        float top = m;
#pragma unroll
        for (int j = 0; j < N; ++j) top = fmaxf(top, ml[j].x);
        const float f = __builtin_amdgcn_exp2f(m - top);
        m = top;
        l *= f;
        o *= f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (ml[j].y == 0.0f) continue;  // nothing in this part (l is NaN where a row sees a NaN)
            const float w = __builtin_amdgcn_exp2f(ml[j].x - m);
            l += ml[j].y * w;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] += v[j][e] * w;
        }
    };
    // (an empty sequence has no parts, and nothing of the workspace is its own: it is not read)
    const int32_t most = join_batch(parts, PPR);
    if (most == 2) batch(0, std::integral_constant<int, 2>{});
    else if (most == 4) batch(0, std::integral_constant<int, 4>{});
    else if (most == 8)
        for (int32_t p0 = 0; p0 < parts; p0 += 8 * PPR) batch(p0, std::integral_constant<int, 8>{});
#pragma unroll
    for (int x = LPP; x < LPP * PPR; x <<= 1) {
        const float top = fmaxf(m, __shfl_xor(m, x, kWave)), f = __builtin_amdgcn_exp2f(m - top);
        m = top;
        l *= f;
        l += __shfl_xor(l, x, kWave);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[e] *= f;
            o[e] += __shfl_xor(o[e], x, kWave);
        }
    }
    if (sub != 0) return;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    store4<DT>(a.out + (int64_t)(row0 + k) * a.out_row + (int64_t)h * a.out_head + col * 2, o.x * inv, o.y * inv, o.z * inv,
               o.w * inv);
    if (a.lse != nullptr && col == 0)
        a.lse[(int64_t)(row0 + k) * heads + h] =
            l != 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f : neg_inf();
}

}  // namespace sv
