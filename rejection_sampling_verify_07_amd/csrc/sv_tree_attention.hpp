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
// hold: the rounds (KB keys) of all (sequence, key head) pairs form one line, and
// each of a fixed number of workgroups takes an equal stretch of it.  A pair that lies within
// one stretch is finished there; one that crosses borders leaves parts, at most
// two per workgroup, which the join adds up.  The workspace therefore does not
// grow with the caches, and sequences of any mix of lengths keep all CUs busy.
//
// Positions come in grains of 16, which never cross a page: a wave finds a
// grain's page with scalar loads, a step before the keys' own loads.
//   Few rows per key head (up to 16 or 32): each wave walks its own 32 keys of a
// round with all rows, K and V straight from memory to registers (attend_rows).
//   More: the four waves share the rows and take tiles of 64 keys through LDS
// (attend_tree_tiles).
#pragma once

#include "sv_attention.hpp"

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
    int32_t* plan;                                   // [batch + 1] rounds before each sequence, then the stretch
    float* acc;                                      // [2 * groups][tile][row][D]
    float2* ml;                                      // [2 * groups][tile][row]
};

// First packed row of sequence b; entries of cu outside the batch are clamped.
__device__ __forceinline__ int32_t tree_row(const TreeArgs& a, int32_t b)
{
    if (b >= a.batch) return a.rows;
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
    bool past;               // read past the caches
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

// Where N neighbouring grains lie: page (-1: none) and position in it.
template <int N>
struct Grains {
    int32_t page[N], in[N];
    __device__ __forceinline__ bool sound() const
    {
        int32_t x = 0;
#pragma unroll
        for (int g = 0; g < N; ++g) x |= page[g];
        return x >= 0;
    }
};

// A scalar load: the tables are not written while a kernel reads them.  (A vector load that a loop carries along keeps
// the compiler from letting the tiles' loads run ahead: it waits for all of them.)
__device__ __forceinline__ int32_t scalar_load(const int32_t* p)
{
    return *(const __attribute__((address_space(4))) int32_t*)p;
}

// Walks grains g, g + STEP, ...: N neighbours each time.  Their pages are asked for one step before they are needed.
template <int N, int STEP>
struct GrainCursor {
    int32_t number, rest;  // the next grain's page number, and its place in that page
    int32_t key;           // its first key
    Grains<N> asked;       // those of `key`, as the table says

    __device__ __forceinline__ void ask(const TreeArgs& a, const Stretch& s)
    {
        int32_t n = number, r = rest;
#pragma unroll
        for (int g = 0; g < N; ++g) {
            asked.page[g] = s.table != nullptr ? scalar_load(s.table + min(n, s.pages - 1)) : s.b;
            asked.in[g] = r * 16;
            const bool over = ++r == a.grains;
            n += over ? 1 : 0;
            r = over ? 0 : r;
        }
        if constexpr (STEP == N) {
            number = n;
            rest = r;
        } else {
            const int32_t q = page_of_grain(a, rest + STEP);
            number += q;
            rest += STEP - q * a.grains;
        }
    }
    __device__ __forceinline__ void start(const TreeArgs& a, const Stretch& s, int32_t first_key)
    {
        key = first_key;
        number = page_of_grain(a, key / 16);
        rest = key / 16 - number * a.grains;
        ask(a, s);
    }
    __device__ __forceinline__ Grains<N> next(const TreeArgs& a, const Stretch& s)
    {
        Grains<N> w = asked;
#pragma unroll
        for (int g = 0; g < N; ++g)
            if (key + g * 16 >= s.total || (uint32_t)w.page[g] >= (uint32_t)a.pages) w.page[g] = -1;
        key += STEP * 16;
        ask(a, s);
        return w;
    }
};

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
        while (true) {
#pragma unroll
            for (int x = 0; x < 5; ++x) w[x + 1] |= r / 32 == x ? 1u << (r % 32) : 0u;
            if (r == 0) break;
            const int32_t up = s.parents != nullptr ? s_up[r - 1] : r - 1;
            r = up >= 0 && up < r ? up : 0;
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

template <int D, int MT>
constexpr size_t tree_rows_lds()
{
    return attn_lds_floats(D, MT) * 4;
}

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

// MT tiles of 16 query rows in every wave, 32 keys of each round per wave.
template <int DT, int D, int MT>
__device__ __forceinline__ void attend_rows(const TreeArgs& a, const Stretch& st, int32_t tile, const TreeOut& to,
                                            const uint32_t* s_view, float* s_mem)
{
    constexpr int DC = D / 32;   // 32-wide chunks of the score product
    constexpr int DPL = D / 16;  // columns of V per lane
    constexpr int VW = DPL / 2;  // 32-bit words of a lane's V row
    const int lane = lane_id(), l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int32_t m_total = st.nrows * a.rep;
    const int32_t r0 = tile * (MT * 16), t0 = r0 / a.rep;

    u32x4 qf[MT][DC];  // query rows: column l16 of each tile; rows past the matrix are zero
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
    f32x4 o[MT][DPL];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = kNoReference;
        l[mt] = 0.0f;
#pragma unroll
        for (int d = 0; d < DPL; ++d) o[mt][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // a lane's keys inside a grain: K row l16; V rows 4 lg + j
    const uint32_t koff = (uint32_t)(l16 * a.k_pos + lg * 16);
    uint32_t voff[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) voff[j] = (uint32_t)((lg * 4 + j) * a.v_pos + l16 * (DPL * 2));
    typedef Grains<2> Block;  // 32 keys
    // Rows of a grain that hold keys: the last one stands in for those behind it (masked below), row 0 of the pool for
    // all of a grain without a page.
    auto last_of = [&](const Block& p, int32_t kb, int t) {
        return p.page[t] < 0 ? 0 : min(15, st.total - 1 - (kb + t * 16));
    };
    auto load_k = [&](int32_t kb, const Block& p, u32x4 (&kf)[2][DC], auto edge, auto past) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const char* base = st.k + max(p.page[t], 0) * a.k_page + (int64_t)(p.page[t] < 0 ? 0 : p.in[t]) * a.k_pos;
            uint32_t off = koff;
            if constexpr (decltype(edge)::value) off = (uint32_t)(min(l16, last_of(p, kb, t)) * a.k_pos + lg * 16);
#pragma unroll
            for (int c = 0; c < DC; ++c) kf[t][c] = load16<decltype(past)::value>((const u32x4*)(base + off + c * 64));
        }
    };
    auto load_v = [&](int32_t kb, const Block& p, uint32_t (&vr)[8][VW], auto edge, auto past) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const char* base = st.v + max(p.page[t], 0) * a.v_page + (int64_t)(p.page[t] < 0 ? 0 : p.in[t]) * a.v_pos;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t off = voff[j];
                if constexpr (decltype(edge)::value)
                    off = (uint32_t)(min(lg * 4 + j, last_of(p, kb, t)) * a.v_pos + l16 * (DPL * 2));
                const char* x = base + off;
                if constexpr (VW == 2) {
                    const u32x2 w = *(const SV_GLOBAL u32x2*)x;
                    vr[t * 4 + j][0] = w.x;
                    vr[t * 4 + j][1] = w.y;
                } else {
#pragma unroll
                    for (int y = 0; y < VW / 4; ++y) {
                        const u32x4 w = load16<decltype(past)::value>((const u32x4*)(x + y * 16));
#pragma unroll
                        for (int z = 0; z < 4; ++z) vr[t * 4 + j][y * 4 + z] = w[z];
                    }
                }
            }
        }
    };

    bool wild = false;  // (uniform) a masked block held a value that is not finite
    bool far = false;   // (uniform) a reference lies beyond kFarReference
    int32_t kb = st.begin + wave * kKeyBlock;
    GrainCursor<2, kKeyRound / 16> cursor;
    cursor.start(a, st, kb);
    Block now = cursor.next(a, st);
    u32x4 kf[2][DC];  // the block at hand; the next one's is loaded once the scores have taken it
    auto next_k = [&](int32_t x, const Block& p) {
        if (x >= st.end) return;
        with_policy(st.past, [&](auto past) {
            if (x + kKeyBlock <= st.total && p.sound()) load_k(x, p, kf, std::false_type{}, past);
            else load_k(x, p, kf, std::true_type{}, past);
        });
    };
    bool masked = false;  // (uniform) from the first block on that rows see in part, or whose pages are not all there
    int32_t masked_from = st.end;
    next_k(kb, now);
    loads_done();
    while (kb < st.end) {
        if (!masked && (kb + kKeyBlock > st.context || !now.sound())) {
            masked = true;
            masked_from = kb;
        }
        uint32_t vr[8][VW];
        with_policy(st.past, [&](auto past) {
            if (!masked) load_v(kb, now, vr, std::false_type{}, past);
            else load_v(kb, now, vr, std::true_type{}, past);
        });
        f32x4 s[2][MT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                s[t][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < DC; ++c) s[t][mt] = mfma_16x16x32<DT>(kf[t][c], qf[mt][c], s[t][mt]);
            }
        const Block next = cursor.next(a, st);
        next_k(kb + kKeyRound, next);
        if (masked) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t seen =
                        now.page[t] < 0 ? 0u : sees4(view[mt], kb + t * 16 + lg * 4 - st.context);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((seen >> i & 1u) == 0) s[t][mt][i] = neg_inf();
                }
        }
        // move a reference that a score exceeds by the slack (the first one always does)
        float top[MT];
        bool over = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float x = fmaxf(s[0][mt][0], s[0][mt][1]);
#pragma unroll
            for (int i = 2; i < 8; ++i) x = fmaxf(x, s[i / 4][mt][i & 3]);
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
                for (int d = 0; d < DPL; ++d) o[mt][d] *= f;
            }
            far = far_references<MT>(m);
        }
        if (__builtin_expect(far, 0)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i / 4][mt][i & 3] = far_distance(s[i / 4][mt][i & 3], a.c, m[mt]);
        }
        const float c = far ? 1.0f : a.c;
        u32x4 pf[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float ref = far ? 0.0f : m[mt];
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i / 4][mt][i & 3], c, -ref));
                l[mt] += p[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) pf[mt][i] = pack2<DT>(p[2 * i], p[2 * i + 1]);
        }
        if (masked) {
            // none for keys past the last one, or without a page
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool there = now.page[j / 4] >= 0 && kb + (j < 4 ? 0 : 12) + lg * 4 + j < st.total;
#pragma unroll
                for (int x = 0; x < VW; ++x) vr[j][x] = there ? vr[j][x] : 0u;
            }
            // A value that is not finite times the weight 0 of a row that does not see it would be NaN: such values
            // count as 0 here, and reach the rows that see them after the last block.
            bool any = false;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int x = 0; x < VW; ++x) any |= finite_halves<DT>(vr[j][x]) != vr[j][x];
            if (__any(any)) {
                wild = true;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int x = 0; x < VW; ++x) vr[j][x] = finite_halves<DT>(vr[j][x]);
            }
        }
#pragma unroll
        for (int d = 0; d < DPL; ++d) {
            u32x4 vf;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                vf[i] = __builtin_amdgcn_perm(vr[2 * i + 1][d / 2], vr[2 * i][d / 2], d & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[mt][d] = mfma_16x16x32<DT>(vf, pf[mt], o[mt][d]);
        }
        now = next;
        kb += kKeyRound;
    }
    if (wild) {
#pragma unroll 1
        for (kb = masked_from; kb < st.end; kb += kKeyRound)
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                int32_t in;
                const int32_t page = grain_page(a, st, kb / 16 + t, &in);
                if (page < 0) continue;
                const char* base = st.v + page * a.v_page + (int64_t)in * a.v_pos;
#pragma unroll 1
                for (int32_t x = 0; x < min(16, st.total - (kb + t * 16)); ++x) {
                    // accumulator i of tile d holds column (4 lg + i) * DPL + d
                    const SV_GLOBAL uint32_t* row =
                        (const SV_GLOBAL uint32_t*)(base + (int64_t)x * a.v_pos + lg * (4 * DPL * 2));
                    bool see[MT];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) see[mt] = sees(view[mt], kb + t * 16 + x - st.context);
#pragma unroll
                    for (int e = 0; e < 4 * DPL; e += 2) {
                        const uint32_t w = row[e / 2], bad = w ^ finite_halves<DT>(w);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float v = y ? hi16<DT>(bad) : lo16<DT>(bad);  // 0 where the value was finite
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                if (see[mt]) o[mt][(e + y) % DPL][(e + y) / DPL] += v;
                        }
                    }
                }
            }
    }

    // ---- join the four waves: a common reference, then o summed in a fixed order
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16, kWave);
        l[mt] += __shfl_xor(l[mt], 32, kWave);
    }
    float* s_m = s_mem;                                 // [wave][MT * 16]
    float* s_l = s_m + kAttnWaves * MT * 16;            // [wave][MT * 16]
    f32x4* s_o = (f32x4*)(s_l + kAttnWaves * MT * 16);  // [2][MT * DPL][64]
    if (lg == 0) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            s_m[(wave * MT + mt) * 16 + l16] = m[mt];
            s_l[(wave * MT + mt) * 16 + l16] = l[mt];
        }
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float x = s_m[mt * 16 + l16];
#pragma unroll
        for (int w = 1; w < kAttnWaves; ++w) x = fmaxf(x, s_m[(w * MT + mt) * 16 + l16]);
        const float f = __builtin_amdgcn_exp2f(m[mt] - x);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w)
            sum += s_l[(w * MT + mt) * 16 + l16] * __builtin_amdgcn_exp2f(s_m[(w * MT + mt) * 16 + l16] - x);
        m[mt] = x;
        l[mt] = sum;
#pragma unroll
        for (int d = 0; d < DPL; ++d) o[mt][d] *= f;
    }
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int i = 0; i < MT * DPL; ++i) s_o[((wave - half) * MT * DPL + i) * kWave + lane] = o[i / DPL][i % DPL];
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int i = 0; i < MT * DPL; ++i) o[i / DPL][i % DPL] += s_o[(wave * MT * DPL + i) * kWave + lane];
        }
        __syncthreads();
    }
    if (wave != 0) return;
    // accumulator i of tile d holds column (4 lg + i) * DPL + d
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int32_t r = r0 + mt * 16 + l16;
        if (r >= m_total) continue;
        const int32_t t = r / a.rep, h = st.hk * a.rep + (r - t * a.rep);
        if (to.whole) {
            const float inv = l[mt] != 0.0f ? 1.0f / l[mt] : 0.0f;
            char* dst = a.out + (int64_t)(st.row0 + t) * a.out_row + (int64_t)h * a.out_head + lg * (4 * DPL * 2);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < DPL; d += 4)
                    store4<DT>(dst + (i * DPL + d) * 2, o[mt][d][i] * inv, o[mt][d + 1][i] * inv, o[mt][d + 2][i] * inv,
                               o[mt][d + 3][i] * inv);
            if (a.lse != nullptr && lg == 0)
                a.lse[(int64_t)(st.row0 + t) * a.q_heads + h] =
                    l[mt] != 0.0f ? (m[mt] + __builtin_amdgcn_logf(l[mt])) * 0.69314718055994531f : neg_inf();
        } else {
            const int64_t at = to.slot * (MT * 16) + mt * 16 + l16;
            if (lg == 0) a.ml[at] = float2{m[mt], l[mt]};
            SV_GLOBAL f32x4* dst = (SV_GLOBAL f32x4*)(a.acc + at * D + lg * 4 * DPL);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < DPL; d += 4)
                    dst[(i * DPL + d) / 4] = f32x4{o[mt][d][i], o[mt][d + 1][i], o[mt][d + 2][i], o[mt][d + 3][i]};
        }
    }
}

// ---- many rows per key head: four waves of MT * 16 rows share tiles of keys through LDS, whose rows lie and are read
// as in TileAttention.  Four tiles of 16 KB (64 columns: of 64 keys; 128: of 32) are on their way or in use: with two
// of them a step lasted as long as a read of memory.
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

// 16 bytes from each lane's place `off` behind `base` into LDS, lane i's at `to` + 16 i (`to`: the wave's).  In assembly, which the compiler
// does not count among the loads in flight: it would wait for all of them before every transposed read of a tile.
// arrived() is the wait for them; a wave has none left when its loop over the tiles ends.  (M0 is not kept between
// instructions that take it: nothing else here does.)
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, uint32_t to)
{
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
                                                  const uint32_t* s_view, int32_t* s_wild, char* s_kv)
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
    walk.start(a, st, kb);
    auto load_next = [&](int buf) {
        if (ahead >= st.end) return;
        const uint32_t dst = lds_address(s_kv) + (uint32_t)(buf * (2 * TA::TILE) + wave * (kWave * 16));
        const bool edge = ahead + KT > st.total;
        int32_t pages = 0;
#pragma unroll
        for (int i = 0; i < TA::LOADS; ++i) {
            // this load's grain: pointers before and after a step where it has two
            const char *k = walk.k, *v = walk.v;
            pages |= walk.page;
            if constexpr (RPL == 32) {
                walk.step(a, st);
                pages |= walk.page;
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
            load_to_lds(k, ko, dst + i * (kAttnThreads * 16));
            load_to_lds(v, vo, dst + TA::TILE + i * (kAttnThreads * 16));
            if (x == PER - 1) walk.step(a, st);
        }
        if (pages < 0) bad_from = min(bad_from, ahead);
        ahead += KT;
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
        __builtin_amdgcn_sched_barrier(0);
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
        if (kb + 2 * KT < st.end) arrived<2 * TA::LOADS>();
        else arrived<0>();
        load_next((buf + TA::BUFS - 1) % TA::BUFS);
        if (!masked && (kb + KT > st.context || kb >= bad_from)) {
            masked = true;
            masked_from = kb;
        }
        if (masked) {
            here = 0;
            int32_t in;
#pragma unroll
            for (int g = 0; g < GR; ++g) here |= grain_page(a, st, kb / 16 + g, &in) >= 0 ? 1u << g : 0u;
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

// Rounds of a pair's keys: what the line counts.
template <bool TILES>
constexpr int kTreeRound = TILES ? 64 : kKeyRound;

// The line's length and where a stretch begins, by all threads of the workgroup: thread t sums the sequences t * per
// .. t * per + per - 1.
struct TreeStart {
    int32_t total, stretch;  // rounds of the line, and of one workgroup
    int32_t b, at;           // the sequence that holds the first round, and the rounds of it before that one
};
template <int KB>
__device__ __forceinline__ TreeStart tree_start(const TreeArgs& a, int32_t group, bool write, int32_t* s_sum,
                                                int32_t* s_found)
{
    const int32_t tid = (int32_t)threadIdx.x, per = (a.batch + kAttnThreads - 1) / kAttnThreads;
    const int32_t b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    int32_t mine = 0;
    for (int32_t b = b0; b < b1; ++b) mine += (tree_length(a, b) + KB - 1) / KB * a.kv_heads;
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
    const int32_t stretch = max(1, (total + a.groups - 1) / a.groups);
    const int64_t from = (int64_t)group * stretch;
    if (write) {
        int32_t sum = before;
        for (int32_t b = b0; b < b1; ++b) {
            a.plan[b] = sum;
            sum += (tree_length(a, b) + KB - 1) / KB * a.kv_heads;
        }
        if (tid == 0) {
            a.plan[a.batch] = total;
            a.plan[a.batch + 1] = stretch;
        }
    }
    if (from >= before && from < before + mine) {
        int32_t sum = before, b = b0;
        while (true) {
            const int32_t n = (tree_length(a, b) + KB - 1) / KB * a.kv_heads;
            if (from < sum + n) break;
            sum += n;
            ++b;
        }
        s_found[0] = b;
        s_found[1] = (int32_t)(from - sum);
    }
    __syncthreads();
    return TreeStart{total, stretch, s_found[0], s_found[1]};
}

constexpr double kTreePastCaches = 128e6;  // bytes of keys and values from which they are read past the caches

template <int DT, int D, bool TILES, int MT>
__global__ __launch_bounds__(kAttnThreads, D == 256 ? 1 : 2) void tree_part_kernel(TreeArgs a)
{
    constexpr int ROWS = MT * 16 * (TILES ? kAttnWaves : 1);
    constexpr int KB = kTreeRound<TILES>;
    constexpr size_t kLds = TILES ? (size_t)TreeTile<D>::LDS : tree_rows_lds<D, MT>();
    // The stretches count on two workgroups per CU: more than a third of the 160 KB keeps a third one out.
    constexpr size_t kLdsOfTwo = 52 * 1024, kMem = D != 256 && kLds < kLdsOfTwo ? kLdsOfTwo : kLds;
    __shared__ __align__(16) char s_mem[kMem];
    __shared__ uint32_t s_view[ROWS * kTreeWords];
    __shared__ int32_t s_up[kTreeMostGuesses], s_sum[kAttnWaves], s_found[2], s_wild;
    // the row tiles of one stretch (the same keys) run on one XCD (workgroups go to the 8 XCDs in turn)
    const uint32_t x = blockIdx.x & 7u, y = blockIdx.x >> 3;
    const int32_t group = a.tiles == 1 ? (int32_t)blockIdx.x : (int32_t)(y / (uint32_t)a.tiles * 8u + x);
    const int32_t tile = a.tiles == 1 ? 0 : (int32_t)(y % (uint32_t)a.tiles);
    if (group >= a.groups) return;
    const TreeStart start = tree_start<KB>(a, group, group == 0 && tile == 0, s_sum, s_found);
    int64_t at = (int64_t)group * start.stretch;
    if (at >= start.total) return;
    const int64_t end = min(at + start.stretch, (int64_t)start.total);
    const bool past = a.tiles == 1 && (double)start.total * (KB * D * 4.0) > kTreePastCaches;
    int32_t b = __builtin_amdgcn_readfirstlane(start.b);
    int32_t in = __builtin_amdgcn_readfirstlane(start.at);  // rounds of sequence b before `at`
    bool first = true;
    while (at < end) {
        const int32_t len = __builtin_amdgcn_readfirstlane(tree_length(a, b)), n = (len + KB - 1) / KB;
        if (in >= n * a.kv_heads) {  // (also the empty sequences)
            in -= n * a.kv_heads;
            ++b;
            continue;
        }
        const int32_t hk = in / n, j = in - hk * n;
        const int32_t take = (int32_t)min((int64_t)(n - j), end - at);
        Stretch st;
        st.b = b;
        st.hk = hk;
        st.row0 = __builtin_amdgcn_readfirstlane(tree_row(a, b));
        st.nrows = __builtin_amdgcn_readfirstlane(min(tree_row(a, b + 1) - st.row0, a.kmax + 1));
        st.total = len;
        st.context = len - st.nrows;
        st.begin = j * KB;
        st.end = min((j + take) * KB, len);
        st.pages = a.table != nullptr ? page_of_grain(a, (len - 1) / 16) + 1 : 1;
        st.k = a.k + (int64_t)hk * a.k_head;
        st.v = a.v + (int64_t)hk * a.v_head;
        st.table = a.table != nullptr ? a.table + (int64_t)b * a.table_stride : nullptr;
        st.parents = a.parents != nullptr ? a.parents + (st.row0 - b) : nullptr;
        st.past = past;
        if (tile * ROWS < st.nrows * a.rep) {
            const int32_t t0 = tile * ROWS / a.rep;
            __syncthreads();  // (the stretch before this one is done with the LDS)
            if (st.end > st.context) tree_views(st, t0, min(st.nrows, ((tile + 1) * ROWS - 1) / a.rep + 1) - t0, s_up, s_view);
            const TreeOut to{j == 0 && take == n, ((int64_t)group * 2 + (first ? 0 : 1)) * a.tiles + tile};
            if constexpr (TILES) attend_tree_tiles<DT, D, MT>(a, st, tile, to, s_view, &s_wild, s_mem);
            else attend_rows<DT, D, MT>(a, st, tile, to, s_view, (float*)s_mem);
        }
        at += take;
        in += take;
        first = false;
    }
}

// Join of the parts: one wave per (row, head), D / 4 lanes over the columns of a part and kWave / (D / 4) parts side by
// side.  A pair that one workgroup finished is left alone; rows that see nothing get zeros.
template <int DT, int D, int ROWS>
__global__ __launch_bounds__(kThreads) void tree_join_kernel(TreeArgs a)
{
    constexpr int LPP = D / 4;        // lanes per part
    constexpr int PPR = kWave / LPP;  // parts per round
    const int64_t i = (int64_t)blockIdx.x * kWaves + wave_id();
    const int32_t heads = a.q_heads;
    const int64_t ik = i / heads;
    const int32_t h = (int32_t)(i - ik * heads), b = (int32_t)(ik / (a.kmax + 1)), k = (int32_t)(ik - (int64_t)b * (a.kmax + 1));
    if (b >= a.batch) return;
    const int32_t row0 = tree_row(a, b), nrows = min(tree_row(a, b + 1) - row0, a.kmax + 1);
    if (k >= nrows) return;
    const int32_t begin = a.plan[b], rounds = (a.plan[b + 1] - begin) / a.kv_heads, stretch = a.plan[a.batch + 1];
    const int32_t hk = h / a.rep, r = k * a.rep + (h - hk * a.rep), tile = r / ROWS;
    const int32_t from = begin + hk * rounds;
    const int32_t g0 = from / stretch, parts = rounds > 0 ? (from + rounds - 1) / stretch - g0 + 1 : 0;
    if (parts == 1) return;
    const int lane = lane_id(), col = (lane % LPP) * 4, sub = lane / LPP;
    // the first part lies in its workgroup's second place if the workgroup began with another pair
    auto place = [&](int32_t p) {
        const int64_t slot = (int64_t)(g0 + p) * 2 + (p == 0 && from != g0 * stretch ? 1 : 0);
        return (slot * a.tiles + tile) * ROWS + (r - tile * ROWS);
    };
    float m = kNoReference;
    for (int32_t p = lane; p < parts; p += kWave) m = fmaxf(m, a.ml[place(p)].x);
    m = wave_max_dpp(m);
    float l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int32_t p = sub; p < parts; p += PPR) {
        const int64_t at = place(p);
        const float2 ml = a.ml[at];
        const f32x4 v = *(const SV_GLOBAL f32x4*)(a.acc + at * D + col);
        if (ml.y == 0.0f) continue;  // nothing in this part (l is NaN where a row sees a NaN)
        const float w = __builtin_amdgcn_exp2f(ml.x - m);
        l += ml.y * w;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += v[e] * w;
    }
#pragma unroll
    for (int x = LPP; x < kWave; x <<= 1) {
        l += __shfl_xor(l, x, kWave);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], x, kWave);
    }
    if (sub != 0) return;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    store4<DT>(a.out + (int64_t)(row0 + k) * a.out_row + (int64_t)h * a.out_head + col * 2, o.x * inv, o.y * inv, o.z * inv,
               o.w * inv);
    if (a.lse != nullptr && lane == 0)
        a.lse[(int64_t)(row0 + k) * heads + h] =
            l != 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f : neg_inf();
}

}  // namespace sv
