// Attention of every sequence's newest rows over a prefix that its group
// shares and over the sequence's own suffix.
//
// For query row t of sequence b in group g, head h (key/value head h / rep):
//     a_j = scale * q . k_j over the prefix keys of g and the suffix keys that
//     the row sees,   out = sum_j exp(a_j - z) v_j,   z = log sum_j exp(a_j).
// The sum over keys splits into parts, each kept as (m, l, o): m a reference
// near the part's largest score, l = sum exp2(a c - m), o = sum exp2(a c - m) v
// with c = scale log2 e.  Parts join by rescaling to a common reference.
//
// Part kernel, one workgroup of four waves per (keys, rows) pair.  Prefix
// workgroups take all rows of a group that share a key/value head as one matrix (the
// sequences' rows lie next to each other), so a prefix key is read once for
// the whole group, not once per sequence; suffix workgroups take one sequence's rows.
// Each wave walks its own blocks of 32 keys with all of the rows.  Scores are formed
// transposed, S^T = K Q^T (rows: keys, columns: query rows), which leaves each
// lane four keys of one query row: its exponentials are already the second
// operand of O^T = V^T P^T once both use the key order {4g..4g+3, 16+4g..+3}
// of lane group g.  V is read in rows, 16 lanes over the D columns, and
// pairs of keys are interleaved in registers; neither K, V nor P passes through LDS.
// The reference m moves only when a score exceeds it by some powers of 2
// (Reference), so the accumulators are rescaled rarely.
//
// P is rounded to the element type for the second product, which takes no
// other: at most half a step, 2^-8 (bf16) or 2^-11 (fp16) of each weight (fp16
// weights below 2^-24 of the row's largest in a part: 2^-35 of that one), and
// the weights' errors are independent, so the sum's is about that of rounding
// out itself at the end (both together: up to 1.35 times the error of out's
// rounding alone in bf16, 1.15 times in fp16, measured).  The sum l takes the
// unrounded weights; scores, statistics and accumulators are fp32.
//
// What bounds it.  A group with few rows per key/value head reads its caches:
// 4 groups of 8 beams, 8 key heads of 128, 65536 shared positions: 185 us,
// 5.9 TB/s with the join.  Many rows are bound by the products and the
// exponentials beside them (attend_tiles).  Small calls are two launches and
// their memory latencies: 4 rows of 8 heads on 500 positions 7.5 us in a row of
// calls on a few inputs, 8.1 to 8.6 us on inputs new to the caches.
#pragma once

#include <type_traits>

#include "sv_common.hpp"

namespace sv {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * kWave;
constexpr int kKeyBlock = 32;                            // keys per wave and step
constexpr int kKeyRound = kAttnWaves * kKeyBlock;        // keys per workgroup and step
constexpr float kNoReference = -__FLT_MAX__;             // m of a part without a visible key
// The reference is set kBelow under a row's largest score and moves when a score exceeds it by kSlack more (in log2).
// fp16 weights use the type's range: they reach 2^15, and those down to 2^-24 of the row's largest are normal numbers
// (at 2^0 to 2^8, half of a weight 17 nats below a sink was lost); bf16 has fp32's range.
template <int DT>
struct Reference {
    static constexpr float kBelow = DT == DT_F16 ? 10.0f : 0.0f;
    static constexpr float kSlack = DT == DT_F16 ? 5.0f : 8.0f;
};

struct AttnArgs {
    const char *q, *pk, *pv, *sk, *sv;
    char* out;
    float* lse;
    int64_t q_row, q_head, out_row, out_head;                  // bytes
    int64_t pk_group, pk_head, pv_group, pv_head;              // bytes
    int64_t sk_seq, sk_head, sv_seq, sv_head;                  // bytes
    int32_t pk_pos, pv_pos, sk_pos, sv_pos;                    // bytes
    const int32_t *cu_draft, *cu_groups, *prefix_len, *suffix_len;
    int32_t groups, batch, rows, max_draft, per_group;         // per_group: sequences per group without cu_groups
    int32_t max_prefix, max_suffix;
    int32_t q_heads, kv_heads, rep;
    float c;                                                   // scale * log2(e)
    int32_t psplits, ssplits, ptiles, stiles;
    int32_t past;              // the caches are larger than what stays in the Infinity Cache
    uint32_t punits, pblocks;  // prefix units (group, head, split), and workgroups that serve them
    float* acc;                // [slot][row][head][D]
    float2* ml;                // [row][head][slot]
};

// A score's distance from its reference is fma(s, c, -m): the exact product less the rounded m.  What m lost is common
// to the row and cancels, but beyond 2^22 (|m| 2^-24 > 1/4) it would carry the weights out of their type's range; from
// there on the product is rounded first, as m was.
constexpr float kFarReference = 4194304.0f;
template <int MT>
__device__ __forceinline__ bool far_references(const float (&m)[MT])
{
    bool far = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) far |= fabsf(m[mt]) > kFarReference && m[mt] != kNoReference;
    return __any(far);
}
__device__ __forceinline__ float far_distance(float s, float c, float m)
{
#pragma clang fp contract(off)
    return s * c - m;
}

template <int DT>
__device__ __forceinline__ f32x4 mfma_16x16x32(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// Two fp32 values rounded to nearest, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (DT == DT_BF16) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 v = {(__bf16)a, (__bf16)b};
        return __builtin_bit_cast(uint32_t, v);
    } else {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const f16x2 v = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
}

// A word's two elements, an infinity or a NaN replaced by 0.
template <int DT>
__device__ __forceinline__ uint32_t finite_halves(uint32_t w)
{
    constexpr uint32_t E = DT == DT_BF16 ? 0x7f80u : 0x7c00u;
    const uint32_t lo = (w & E) == E ? 0u : w & 0xffffu;
    const uint32_t hi = (w & (E << 16)) == E << 16 ? 0u : w & 0xffff0000u;
    return lo | hi;
}

// First query row of sequence b, and the row count of a sequence; entries of
// cu_draft outside the batch are clamped, so no row index leaves [0, rows].
__device__ __forceinline__ int32_t first_row(const AttnArgs& a, int32_t b)
{
    if (b >= a.batch) return a.rows;
    if (a.cu_draft == nullptr) return b * (a.max_draft + 1);
    return min(max(a.cu_draft[b], 0), a.rows - a.batch) + b;
}

// The keys that one workgroup's rows meet, and where.
struct KeyRange {
    const char *k, *v;
    int32_t k_pos, v_pos;   // bytes between positions
    int32_t begin, end;     // this workgroup's positions
    int32_t total;          // positions of the cache (the last row's view)
    bool past;              // read past the caches: nothing else will read these keys
};

// Runs load(true) or load(false) as `past`, uniform over the workgroup, says.  The empty asm statements keep the
// compiler from merging the two arms' loads, which differ in nothing but the cache policy, into plain ones.
template <class Load>
__device__ __forceinline__ void with_policy(bool past, Load load)
{
    if (past) {
        asm volatile("");
        load(std::true_type{});
        asm volatile("");
    } else {
        load(std::false_type{});
    }
}

// MT tiles of 16 query rows.  row0, nrows: the packed query rows of the matrix;
// tile: which MT * 16 of its nrows * rep rows; seen_short: how many keys
// before `total` the first query row stops (suffix: K_b, each next row one
// later; prefix: every row sees all).
template <int DT, int D, int MT>
__device__ __forceinline__ void attend(const AttnArgs& a, const KeyRange& kr, int32_t row0, int32_t nrows, int32_t hk,
                                       int32_t tile, int32_t seen_short, int32_t slot, float* s_mem)
{
    constexpr int DC = D / 32;   // 32-wide chunks of the score product
    constexpr int DPL = D / 16;  // columns of V per lane
    constexpr int VW = DPL / 2;  // 32-bit words of a lane's V row
    const int lane = lane_id(), wave = wave_id(), l16 = lane & 15, lg = lane >> 4;
    const int32_t m_total = nrows * a.rep;
    const int32_t r0 = tile * (MT * 16);

    // query rows: column l16 of each tile; rows past the matrix are zero
    u32x4 qf[MT][DC];
    int32_t lim[MT];  // keys from here on are masked for this lane's row
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int32_t r = r0 + mt * 16 + l16;
        const int32_t t = r / a.rep, h = hk * a.rep + (r - t * a.rep);
        const char* qp = a.q + (int64_t)(row0 + t) * a.q_row + (int64_t)h * a.q_head + lg * 16;
#pragma unroll
        for (int c = 0; c < DC; ++c)
            qf[mt][c] = r < m_total ? *(const SV_GLOBAL u32x4*)(qp + c * 64) : u32x4{0u, 0u, 0u, 0u};
        lim[mt] = min(kr.end, kr.total - max(seen_short - t, 0));
    }
    const int32_t whole = min(kr.end, kr.total - seen_short);  // keys below are seen by every row

    f32x4 o[MT][DPL];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = kNoReference;
        l[mt] = 0.0f;
#pragma unroll
        for (int d = 0; d < DPL; ++d) o[mt][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // a lane's keys inside a block: K rows l16 and 16 + l16; V rows 4 lg + j and 16 + 4 lg + j.
    // Offsets of a whole block are kept; a block that the range ends in takes the last key for those past it (masked
    // below).
    uint32_t koff[2], voff[8];
#pragma unroll
    for (int t = 0; t < 2; ++t) koff[t] = (uint32_t)((t * 16 + l16) * kr.k_pos + lg * 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) voff[j] = (uint32_t)(((j < 4 ? 0 : 12) + lg * 4 + j) * kr.v_pos + l16 * (DPL * 2));
    auto load_k = [&](int32_t kb, u32x4 (&kf)[2][DC], auto masked, auto past) {
        const char* base = kr.k + (int64_t)kb * kr.k_pos;
        const int32_t last = kr.end - 1 - kb;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t off = koff[t];
            if constexpr (decltype(masked)::value) off = (uint32_t)(min(t * 16 + l16, last) * kr.k_pos + lg * 16);
#pragma unroll
            for (int c = 0; c < DC; ++c) kf[t][c] = load16<decltype(past)::value>((const u32x4*)(base + off + c * 64));
        }
    };
    auto load_v = [&](int32_t kb, uint32_t (&vr)[8][VW], auto masked, auto past) {
        const char* base = kr.v + (int64_t)kb * kr.v_pos;
        const int32_t last = kr.end - 1 - kb;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t off = voff[j];
            if constexpr (decltype(masked)::value)
                off = (uint32_t)(min((j < 4 ? 0 : 12) + lg * 4 + j, last) * kr.v_pos + l16 * (DPL * 2));
            const char* p = base + off;
            if constexpr (VW == 2) {
                const u32x2 w = *(const SV_GLOBAL u32x2*)p;
                vr[j][0] = w.x;
                vr[j][1] = w.y;
            } else {
#pragma unroll
                for (int x = 0; x < VW / 4; ++x) {
                    const u32x4 w = load16<decltype(past)::value>((const u32x4*)(p + x * 16));
#pragma unroll
                    for (int y = 0; y < 4; ++y) vr[j][x * 4 + y] = w[y];
                }
            }
        }
    };

    bool wild = false;  // (uniform) a masked block held a value that is not finite
    bool far = false;   // (uniform) a reference lies beyond kFarReference
    u32x4 kf[2][DC];  // the block at hand; the next one's is loaded once the scores have taken it
    auto next_k = [&](int32_t kb) {
        if (kb >= kr.end) return;
        with_policy(kr.past, [&](auto past) {
            if (kb + kKeyBlock <= kr.end) load_k(kb, kf, std::false_type{}, past);
            else load_k(kb, kf, std::true_type{}, past);
        });
    };
    auto step = [&](int32_t kb, auto masked) {
        constexpr bool MASKED = decltype(masked)::value;
        uint32_t vr[8][VW];
        with_policy(kr.past, [&](auto past) { load_v(kb, vr, masked, past); });
        f32x4 s[2][MT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                s[t][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < DC; ++c) s[t][mt] = mfma_16x16x32<DT>(kf[t][c], qf[mt][c], s[t][mt]);
            }
        next_k(kb + kKeyRound);
        if constexpr (MASKED) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (kb + t * 16 + lg * 4 + i >= lim[mt]) s[t][mt][i] = neg_inf();
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
        if constexpr (MASKED) {
            // the last key's value may be infinite: none for keys past the range
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int x = 0; x < VW; ++x)
                    vr[j][x] = kb + (j < 4 ? 0 : 12) + lg * 4 + j < kr.end ? vr[j][x] : 0u;
            // A value that is not finite times the weight 0 of a row that does not see it would be NaN: such values
            // count as 0 here, and reach the rows that see them after the last block.
            if (seen_short > 0) {
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
    };
    int32_t kb = kr.begin + wave * kKeyBlock;
    next_k(kb);
    for (; kb + kKeyBlock <= whole; kb += kKeyRound) step(kb, std::false_type{});
    const int32_t kb_masked = kb;
    for (; kb < kr.end; kb += kKeyRound) step(kb, std::true_type{});
    if (wild) {
#pragma unroll 1
        for (kb = kb_masked; kb < kr.end; kb += kKeyRound)
#pragma unroll 1
            for (int32_t x = kb; x < min(kr.end, kb + kKeyBlock); ++x) {
                // accumulator i of tile d holds column (4 lg + i) * DPL + d
                const SV_GLOBAL uint32_t* row =
                    (const SV_GLOBAL uint32_t*)(kr.v + (int64_t)x * kr.v_pos + lg * (4 * DPL * 2));
#pragma unroll
                for (int e = 0; e < 4 * DPL; e += 2) {
                    const uint32_t w = row[e / 2], bad = w ^ finite_halves<DT>(w);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float v = y ? hi16<DT>(bad) : lo16<DT>(bad);  // 0 where the value was finite
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            if (x < lim[mt]) o[mt][(e + y) % DPL][(e + y) / DPL] += v;
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
    float* s_m = s_mem;                                   // [wave][MT * 16]
    float* s_l = s_m + kAttnWaves * MT * 16;              // [wave][MT * 16]
    f32x4* s_o = (f32x4*)(s_l + kAttnWaves * MT * 16);    // [2][MT * DPL][64]
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
        const int32_t t = r / a.rep, h = hk * a.rep + (r - t * a.rep);
        const int64_t rh = (int64_t)(row0 + t) * a.q_heads + h;
        const int64_t at = (int64_t)slot * a.rows * a.q_heads + rh;
        if (lg == 0) a.ml[rh * (a.psplits + a.ssplits) + slot] = float2{m[mt], l[mt]};
        SV_GLOBAL f32x4* dst = (SV_GLOBAL f32x4*)(a.acc + at * D + lg * 4 * DPL);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 0; d < DPL; d += 4)
                dst[(i * DPL + d) / 4] = f32x4{o[mt][d][i], o[mt][d + 1][i], o[mt][d + 2][i], o[mt][d + 3][i]};
    }
}

// ---- many rows per key/value head: keys and values through LDS
//
// Four waves of MT * 16 rows each share tiles of KT keys.  At these row counts
// the products bound the kernel, and what feeds them: with each wave reading
// its own keys (attend above) 64 rows per wave hold all registers and leave one
// wave per SIMD; 32 rows and two workgroups per CU let one wave's exponentials
// run beside another's products, and LDS serves a key row to four waves.
//
// A tile's 16-byte chunks are stored at chunk ^ (row mod 16) (mod 8 for D = 64): the score
// product reads 16 rows at one column, which would otherwise all lie in the same banks.
// V is read transposed (each 16 lanes exchange a 4 x 16 block), so that lane
// l16 of tile d holds four keys of column d * 16 + l16.
// The next tile travels in registers while the present one is used.
//
// 320 rows of 32 heads on 65536 positions (8 key heads of 128): 366 to 379 us,
// 0.91 to 0.94 PFLOP/s with the join.  Per 64 keys and 32 rows a wave spends
// 1024 cycles of matrix instructions and about 1250 of vector ones (32
// exponentials at a quarter rate, 32 each of scale-and-subtract, sum, maximum),
// and the two waves of a SIMD overlap them little: counters show the vector
// units busy 47% and the matrix units 33% of the time, LDS 33%.  (128 columns
// hold all 256 registers; 8 more are spilled, outside the loop.)  Three waves
// per SIMD leave 168 registers, which spills inside it; 64 rows per wave leave
// one wave.  Scores of the next 32 keys formed beside the exponentials of the
// present ones (keys a tile ahead of values, 80 KB of LDS) took 400 us, however
// the two were interleaved.
template <int DT, int D, int MT>
struct TileAttention {
    static constexpr int DC = D / 32, DT16 = D / 16;
    static constexpr int KT = 64;                         // keys per tile
    static constexpr int ROW = D * 2;                     // bytes per key row
    static constexpr int CH = ROW / 16;                   // 16-byte chunks per row
    static constexpr int MASK = CH < 16 ? CH - 1 : 15;    // swizzle
    static constexpr int TILE = KT * ROW;                 // bytes of K (or V) per tile
    static constexpr int LOADS = TILE / 16 / kAttnThreads;
    static constexpr int LDS = 4 * TILE;                  // K and V, two tiles each
    static constexpr int ROWS = kAttnWaves * MT * 16;     // query rows per workgroup
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
#define SV_LDS __attribute__((address_space(3)))

__device__ __forceinline__ u32x2 lds_read_transposed(const char* p)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SV_LDS s16x4*)p));
}

template <int DT, int D, int MT>
__device__ __forceinline__ void attend_tiles(const AttnArgs& a, const KeyRange& kr, int32_t row0, int32_t nrows,
                                             int32_t hk, int32_t tile, int32_t slot, char* s_kv)
{
    typedef TileAttention<DT, D, MT> TA;
    constexpr int DC = TA::DC, DT16 = TA::DT16, KT = TA::KT, SUBS = KT / kKeyBlock;
    const int lane = lane_id(), wave = wave_id(), l16 = lane & 15, lg = lane >> 4;
    const int32_t m_total = nrows * a.rep;
    const int32_t r0 = tile * TA::ROWS + wave * (MT * 16);
    const bool idle = r0 >= m_total;  // no rows: the wave only moves tiles

    u32x4 qf[MT][DC];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int32_t r = r0 + mt * 16 + l16;
        const int32_t t = r / a.rep, h = hk * a.rep + (r - t * a.rep);
        const char* qp = a.q + (int64_t)(row0 + t) * a.q_row + (int64_t)h * a.q_head + lg * 16;
#pragma unroll
        for (int c = 0; c < DC; ++c)
            qf[mt][c] = r < m_total ? *(const SV_GLOBAL u32x4*)(qp + c * 64) : u32x4{0u, 0u, 0u, 0u};
    }
    f32x4 o[MT][DT16];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = kNoReference;
        l[mt] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT16; ++d) o[mt][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // this thread's chunks of a tile: row and column, and the place in LDS
    u32x4 kreg[TA::LOADS], vreg[TA::LOADS];
    uint32_t koff[TA::LOADS], voff[TA::LOADS];
#pragma unroll
    for (int i = 0; i < TA::LOADS; ++i) {
        const int32_t x = i * kAttnThreads + (int32_t)threadIdx.x;
        koff[i] = (uint32_t)(x / TA::CH * kr.k_pos + x % TA::CH * 16);
        voff[i] = (uint32_t)(x / TA::CH * kr.v_pos + x % TA::CH * 16);
    }
    auto fetch = [&](int32_t kb) {
        const char* kbase = kr.k + (int64_t)kb * kr.k_pos;
        const char* vbase = kr.v + (int64_t)kb * kr.v_pos;
        const int32_t last = kr.end - 1 - kb;
        if (last >= KT - 1) {
#pragma unroll
            for (int i = 0; i < TA::LOADS; ++i) {
                kreg[i] = *(const SV_GLOBAL u32x4*)(kbase + koff[i]);
                vreg[i] = *(const SV_GLOBAL u32x4*)(vbase + voff[i]);
            }
        } else {  // the range ends in this tile: the last key in place of those past it, masked below
#pragma unroll
            for (int i = 0; i < TA::LOADS; ++i) {
                const int32_t x = i * kAttnThreads + (int32_t)threadIdx.x;
                const int32_t row = min(x / TA::CH, last), ch = x % TA::CH;
                kreg[i] = *(const SV_GLOBAL u32x4*)(kbase + (uint32_t)(row * kr.k_pos + ch * 16));
                vreg[i] = *(const SV_GLOBAL u32x4*)(vbase + (uint32_t)(row * kr.v_pos + ch * 16));
            }
        }
    };
    auto keep = [&](int buf, int32_t kb) {
        char* dst = s_kv + buf * (2 * TA::TILE);
        if (kb + KT > kr.end) {  // the last key's value may be infinite: none for keys past the range
#pragma unroll
            for (int i = 0; i < TA::LOADS; ++i)
                if (kb + (i * kAttnThreads + (int32_t)threadIdx.x) / TA::CH >= kr.end) vreg[i] = u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int i = 0; i < TA::LOADS; ++i) {
            const int32_t x = i * kAttnThreads + (int32_t)threadIdx.x;
            const int32_t row = x / TA::CH, ch = x % TA::CH;
            const int32_t at = row * TA::ROW + ((ch ^ (row & TA::MASK)) * 16);
            *(u32x4*)(dst + at) = kreg[i];
            *(u32x4*)(dst + TA::TILE + at) = vreg[i];
        }
    };

    if (kr.begin < kr.end) {
        fetch(kr.begin);
        keep(0, kr.begin);
    }
    __syncthreads();
    int buf = 0;
    bool far = false;  // (uniform over the wave) a reference lies beyond kFarReference
    // one tile; MASKED: the range ends inside it
    auto use = [&](int32_t kb, auto masked) {
        constexpr bool MASKED = decltype(masked)::value;
        const char* s_k = s_kv + buf * (2 * TA::TILE);
        const char* s_v = s_k + TA::TILE;
        // The fragments that a group of products needs are read while the group before it runs (the barriers keep the
        // scheduler from moving a read down to its use, which exposed the LDS latency once per product).
        auto k_rows = [&](int i, u32x4 (&kf)[DC]) {  // 16 keys
            const int32_t row = i * 16 + l16;
#pragma unroll
            for (int c = 0; c < DC; ++c)
                kf[c] = *(const u32x4*)(s_k + row * TA::ROW + (((c * 4 + lg) ^ (l16 & TA::MASK)) * 16));
        };
        auto v_columns = [&](int u, u32x4 (&vf)[DT16]) {  // 32 keys: four (lg * 4 + l16 / 4) and 8 bytes of columns per
                                                          // lane before the exchange
            const int32_t vrow = u * kKeyBlock + lg * 4 + (l16 >> 2);
#pragma unroll
            for (int d = 0; d < DT16; ++d) {
                const int32_t at =
                    vrow * TA::ROW + (((d * 2 + ((l16 & 3) >> 1)) ^ (vrow & TA::MASK)) * 16) + (l16 & 1) * 8;
                const u32x2 v0 = lds_read_transposed(s_v + at), v1 = lds_read_transposed(s_v + at + 16 * TA::ROW);
                vf[d] = u32x4{v0.x, v0.y, v1.x, v1.y};
            }
        };
        f32x4 s[SUBS][2][MT];
        u32x4 kf[2][DC], vf[DT16];
        k_rows(0, kf[0]);
#pragma unroll
        for (int i = 0; i < 2 * SUBS; ++i) {
            const int u = i / 2, t = i & 1;
            if (i + 1 < 2 * SUBS) k_rows(i + 1, kf[(i + 1) & 1]);
            else v_columns(0, vf);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) s[u][t][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < DC; ++c)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) s[u][t][mt] = mfma_16x16x32<DT>(kf[i & 1][c], qf[mt][c], s[u][t][mt]);
            if constexpr (MASKED) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i2 = 0; i2 < 4; ++i2)
                        if (kb + u * kKeyBlock + t * 16 + lg * 4 + i2 >= kr.end) s[u][t][mt][i2] = neg_inf();
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
            if (u + 1 < SUBS) v_columns(u + 1, vf);
        }
    };
    int32_t kb = kr.begin;
    for (; kb + KT < kr.end; kb += KT, buf ^= 1) {
        fetch(kb + KT);
        if (!idle) use(kb, std::false_type{});
        keep(buf ^ 1, kb + KT);
        __syncthreads();
    }
    if (kb < kr.end && !idle) use(kb, std::true_type{});
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16, kWave);
        l[mt] += __shfl_xor(l[mt], 32, kWave);
        const int32_t r = r0 + mt * 16 + l16;
        if (r >= m_total) continue;
        const int32_t t = r / a.rep, h = hk * a.rep + (r - t * a.rep);
        const int64_t rh = (int64_t)(row0 + t) * a.q_heads + h;
        const int64_t at = (int64_t)slot * a.rows * a.q_heads + rh;
        if (lg == 0) a.ml[rh * (a.psplits + a.ssplits) + slot] = float2{m[mt], l[mt]};
        // accumulator i of tile d holds column d * 16 + lg * 4 + i
        SV_GLOBAL f32x4* dst = (SV_GLOBAL f32x4*)(a.acc + at * D + lg * 4);
#pragma unroll
        for (int d = 0; d < DT16; ++d) dst[d * 4] = o[mt][d];
    }
}

constexpr size_t attn_lds_floats(int D, int MT)
{
    return 2 * kAttnWaves * MT * 16 + 2 * (size_t)MT * (D / 16) * kWave * 4;
}

__device__ __forceinline__ int32_t div_up(int32_t x, int32_t y) { return (x + y - 1) / y; }

// A share of [0, total) for split i of n, in whole steps of `keys`.
template <int keys>
__device__ __forceinline__ void share(int32_t total, int32_t i, int32_t n, int32_t* begin, int32_t* end)
{
    const int32_t chunk = div_up(div_up(total, n), keys) * keys;
    *begin = (int32_t)min((int64_t)total, (int64_t)i * chunk);
    *end = (int32_t)min((int64_t)total, (int64_t)*begin + chunk);
}

// MTP, MTS: 16-row tiles per wave for prefix and suffix work.  TILES: prefix
// work goes through attend_tiles.
// Two waves per SIMD where 256 registers hold a wave's rows.
template <int DT, int D, bool TILES, int MTP, int MTS>
__global__ __launch_bounds__(kAttnThreads, D == 256 ? 1 : 2) void attn_part_kernel(AttnArgs a)
{
    constexpr size_t kLdsPrefix = TILES ? TileAttention<DT, D, MTP>::LDS : attn_lds_floats(D, MTP) * 4;
    constexpr size_t kLdsSuffix = attn_lds_floats(D, MTS) * 4;
    constexpr int kRowsPrefix = TILES ? TileAttention<DT, D, MTP>::ROWS : MTP * 16;
    constexpr size_t kLds = kLdsPrefix > kLdsSuffix ? kLdsPrefix : kLdsSuffix;
    // The splits of tiled work count on two workgroups per CU: more than a third of the 160 KB keeps a third one out where
    // the registers would hold it (58 against 48 us on 2 groups of 40 with K 0..6, 2 key heads of 64, 20000 positions).
    constexpr size_t kLdsOfTwo = 56 * 1024;
    __shared__ __align__(16) char s_mem[TILES && kLds < kLdsOfTwo ? kLdsOfTwo : kLds];
    KeyRange kr;
    if (blockIdx.x < a.pblocks) {
        // the tiles of one unit (the same keys) run on one XCD (workgroups go to the 8 XCDs in turn)
        const uint32_t x = blockIdx.x & 7u, y = blockIdx.x >> 3;
        const uint32_t unit = (y / (uint32_t)a.ptiles) * 8u + x;
        const int32_t tile = (int32_t)(y % (uint32_t)a.ptiles);
        if (unit >= a.punits) return;
        const int32_t hk = (int32_t)(unit % (uint32_t)a.kv_heads);
        const uint32_t rest = unit / (uint32_t)a.kv_heads;
        const int32_t g = (int32_t)(rest % (uint32_t)a.groups), split = (int32_t)(rest / (uint32_t)a.groups);
        int32_t b0 = g * a.per_group, b1 = b0 + a.per_group;
        if (a.cu_groups != nullptr) {
            b0 = min(max(a.cu_groups[g], 0), a.batch);
            b1 = min(max(a.cu_groups[g + 1], 0), a.batch);
        }
        const int32_t row0 = first_row(a, b0), nrows = b1 > b0 ? first_row(a, b1) - row0 : 0;
        if (tile * kRowsPrefix >= nrows * a.rep) return;
        const int32_t total = a.prefix_len != nullptr ? min(max(a.prefix_len[g], 0), a.max_prefix) : a.max_prefix;
        share<TILES ? TileAttention<DT, D, MTP>::KT : kKeyRound>(total, split, a.psplits, &kr.begin, &kr.end);
        kr.total = total;
        kr.past = a.past != 0;  // (one wave's rows: no other workgroup reads these keys; attend_tiles ignores it)
        kr.k = a.pk + (int64_t)g * a.pk_group + (int64_t)hk * a.pk_head;
        kr.v = a.pv + (int64_t)g * a.pv_group + (int64_t)hk * a.pv_head;
        kr.k_pos = a.pk_pos;
        kr.v_pos = a.pv_pos;
        if constexpr (TILES) attend_tiles<DT, D, MTP>(a, kr, row0, nrows, hk, tile, split, s_mem);
        else attend<DT, D, MTP>(a, kr, row0, nrows, hk, tile, 0, split, (float*)s_mem);
    } else {
        uint32_t y = blockIdx.x - a.pblocks;
        const int32_t tile = (int32_t)(y % (uint32_t)a.stiles);
        y /= (uint32_t)a.stiles;
        const int32_t hk = (int32_t)(y % (uint32_t)a.kv_heads);
        y /= (uint32_t)a.kv_heads;
        const int32_t b = (int32_t)(y % (uint32_t)a.batch), split = (int32_t)(y / (uint32_t)a.batch);
        const int32_t row0 = first_row(a, b), nrows = min(first_row(a, b + 1) - row0, a.max_draft + 1);
        if (tile * (MTS * 16) >= nrows * a.rep) return;
        const int32_t total = a.suffix_len != nullptr ? min(max(a.suffix_len[b], 0), a.max_suffix) : a.max_suffix;
        share<kKeyRound>(total, split, a.ssplits, &kr.begin, &kr.end);
        kr.total = total;
        kr.past = a.past != 0 && a.stiles == 1;
        kr.k = a.sk + (int64_t)b * a.sk_seq + (int64_t)hk * a.sk_head;
        kr.v = a.sv + (int64_t)b * a.sv_seq + (int64_t)hk * a.sv_head;
        kr.k_pos = a.sk_pos;
        kr.v_pos = a.sv_pos;
        attend<DT, D, MTS>(a, kr, row0, nrows, hk, tile, nrows - 1, a.psplits + split, (float*)s_mem);
    }
}

// Join of the parts: one wave per (row, head).  D / 4 lanes take the columns
// of a part, so kWave / (D / 4) parts are read side by side, kJoinRounds times
// without waiting: those loads go out before the parts' (m, l), one per lane,
// have arrived, and before it is known which parts hold anything (a part
// without a visible key has l = 0 and is dropped; l is NaN where a row sees a NaN).
// 10240 (row, head) pairs of 128 columns in 7 parts: 9.6 us, 4.1 TB/s; 32 pairs
// of 4 parts: 3.5 us, latency.
constexpr int kJoinRounds = 4;
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnArgs a)
{
    constexpr int LPP = D / 4;         // lanes per part
    constexpr int PPR = kWave / LPP;   // parts per round
    const int64_t n = (int64_t)a.rows * a.q_heads;
    const int64_t i = (int64_t)blockIdx.x * kWaves + wave_id();
    if (i >= n) return;
    const int lane = lane_id(), col = (lane % LPP) * 4, sub = lane / LPP;
    const int slots = a.psplits + a.ssplits;
    const float2* ml = a.ml + i * slots;
    const int64_t part = n * (D * 4);  // bytes from a part to the next
    const SV_GLOBAL char* acc = (const SV_GLOBAL char*)(a.acc + i * D + col) + sub * part;
    f32x4 v[kJoinRounds];
    auto bring = [&](int s0) {
        const SV_GLOBAL char* p = acc + s0 * part;
#pragma unroll
        for (int r = 0; r < kJoinRounds; ++r, p += PPR * part)
            v[r] = s0 + r * PPR + sub < slots ? *(const SV_GLOBAL f32x4*)p : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    bring(0);
    float2 own = lane < slots ? ml[lane] : float2{kNoReference, 0.0f};  // this lane's part of the current 64
    float m = own.x;
    for (int s = kWave + lane; s < slots; s += kWave) m = fmaxf(m, ml[s].x);
    m = wave_max_dpp(m);
    float l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < slots; s0 += kWave) {
        if (s0 > 0) own = s0 + lane < slots ? ml[s0 + lane] : float2{kNoReference, 0.0f};
        const float w = own.y != 0.0f ? __builtin_amdgcn_exp2f(own.x - m) : -1.0f;  // -1: nothing in this part
        l += own.y * w;
#pragma unroll 1
        for (int q = 0; q < kWave && s0 + q < slots; q += kJoinRounds * PPR) {
            if (s0 + q > 0) bring(s0 + q);
#pragma unroll
            for (int r = 0; r < kJoinRounds; ++r) {
                const float f = __shfl(w, q + r * PPR + sub, kWave);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] += f < 0.0f ? 0.0f : v[r][e] * f;
            }
        }
    }
#pragma unroll
    for (int x = kWave / 2; x > 0; x >>= 1) l += __shfl_xor(l, x, kWave);
#pragma unroll
    for (int x = LPP; x < kWave; x <<= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], x, kWave);
    }
    if (sub != 0) return;
    const int32_t t = (int32_t)(i / a.q_heads), h = (int32_t)(i - (int64_t)t * a.q_heads);
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    u32x2 w;
    w.x = pack2<DT>(o.x * inv, o.y * inv);
    w.y = pack2<DT>(o.z * inv, o.w * inv);
    *(SV_GLOBAL u32x2*)(a.out + (int64_t)t * a.out_row + (int64_t)h * a.out_head + col * 2) = w;
    if (a.lse != nullptr && lane == 0)
        a.lse[i] = l != 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f : neg_inf();
}

}  // namespace sv
