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
// The reference m moves only when a score exceeds it by 8 (in log2): then p is
// at most 2^8, and the accumulators are rescaled rarely.
//
// P is rounded to the element type for the second product (half a unit:
// 2^-9 of a bf16 value's binade, averaged over the keys), as out itself is at
// the end; scores, statistics and accumulators are fp32.
#pragma once

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
constexpr float kNoReference = -1e30f;                   // m of a part without a visible key
constexpr float kReferenceSlack = 8.0f;

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
    uint32_t punits, pblocks;  // prefix units (group, head, split), and workgroups that serve them
    float* acc;                // [slot][row][head][D]
    float2* ml;                // [slot][row][head]
};

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
};

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

    // a lane's keys inside a block: K rows l16 and 16 + l16; V rows 4 lg + j and 16 + 4 lg + j
    auto load_k = [&](int32_t kb, u32x4 (&kf)[2][DC]) {
        const char* base = kr.k + (int64_t)kb * kr.k_pos;
        const int32_t last = kr.end - 1 - kb;  // (a key past the end: the last one, masked below)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t off = (uint32_t)(min(t * 16 + l16, last) * kr.k_pos + lg * 16);
#pragma unroll
            for (int c = 0; c < DC; ++c) kf[t][c] = *(const SV_GLOBAL u32x4*)(base + off + c * 64);
        }
    };
    auto load_v = [&](int32_t kb, uint32_t (&vr)[8][VW]) {
        const char* base = kr.v + (int64_t)kb * kr.v_pos;
        const int32_t last = kr.end - 1 - kb;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t key = (j < 4 ? 0 : 12) + lg * 4 + j;
            const char* p = base + (uint32_t)(min(key, last) * kr.v_pos + l16 * (DPL * 2));
            if constexpr (VW == 2) {
                const u32x2 w = *(const SV_GLOBAL u32x2*)p;
                vr[j][0] = w.x;
                vr[j][1] = w.y;
            } else {
#pragma unroll
                for (int x = 0; x < VW / 4; ++x) {
                    const u32x4 w = *(const SV_GLOBAL u32x4*)(p + x * 16);
#pragma unroll
                    for (int y = 0; y < 4; ++y) vr[j][x * 4 + y] = w[y];
                }
            }
        }
    };

    u32x4 kf[2][DC];
    int32_t kb = kr.begin + wave * kKeyBlock;
    if (kb < kr.end) load_k(kb, kf);
    for (; kb < kr.end; kb += kKeyRound) {
        uint32_t vr[8][VW];
        load_v(kb, vr);
        f32x4 s[2][MT];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                s[t][mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < DC; ++c) s[t][mt] = mfma_16x16x32<DT>(kf[t][c], qf[mt][c], s[t][mt]);
            }
        if (kb + kKeyRound < kr.end) load_k(kb + kKeyRound, kf);
        if (kb + kKeyBlock > whole) {
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
            over |= top[mt] > m[mt] + kReferenceSlack;
        }
        if (__any(over)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float x = top[mt];
                x = fmaxf(x, __shfl_xor(x, 16, kWave));
                x = fmaxf(x, __shfl_xor(x, 32, kWave));
                x = fmaxf(x, m[mt]);
                const float f = __builtin_amdgcn_exp2f(m[mt] - x);
                m[mt] = x;
                l[mt] *= f;
#pragma unroll
                for (int d = 0; d < DPL; ++d) o[mt][d] *= f;
            }
        }
        u32x4 pf[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i / 4][mt][i & 3], a.c, -m[mt]));
                l[mt] += p[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) pf[mt][i] = pack2<DT>(p[2 * i], p[2 * i + 1]);
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
        const int64_t at = ((int64_t)slot * a.rows + row0 + t) * a.q_heads + h;
        if (lg == 0) a.ml[at] = float2{m[mt], l[mt]};
        SV_GLOBAL f32x4* dst = (SV_GLOBAL f32x4*)(a.acc + at * D + lg * 4 * DPL);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 0; d < DPL; d += 4)
                dst[(i * DPL + d) / 4] = f32x4{o[mt][d][i], o[mt][d + 1][i], o[mt][d + 2][i], o[mt][d + 3][i]};
    }
}

constexpr size_t attn_lds_floats(int D, int MT)
{
    return 2 * kAttnWaves * MT * 16 + 2 * (size_t)MT * (D / 16) * kWave * 4;
}

__device__ __forceinline__ int32_t div_up(int32_t x, int32_t y) { return (x + y - 1) / y; }

// A share of [0, total) for split i of n, in whole rounds of the workgroup's keys.
__device__ __forceinline__ void share(int32_t total, int32_t i, int32_t n, int32_t* begin, int32_t* end)
{
    const int32_t chunk = div_up(div_up(total, n), kKeyRound) * kKeyRound;
    *begin = (int32_t)min((int64_t)total, (int64_t)i * chunk);
    *end = (int32_t)min((int64_t)total, (int64_t)*begin + chunk);
}

template <int DT, int D, int MTP, int MTS>
__global__ __launch_bounds__(kAttnThreads) void attn_part_kernel(AttnArgs a)
{
    __shared__ __align__(16) float s_mem[attn_lds_floats(D, MTP > MTS ? MTP : MTS)];
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
        if (tile * (MTP * 16) >= nrows * a.rep) return;
        const int32_t total = a.prefix_len != nullptr ? min(max(a.prefix_len[g], 0), a.max_prefix) : a.max_prefix;
        share(total, split, a.psplits, &kr.begin, &kr.end);
        kr.total = total;
        kr.k = a.pk + (int64_t)g * a.pk_group + (int64_t)hk * a.pk_head;
        kr.v = a.pv + (int64_t)g * a.pv_group + (int64_t)hk * a.pv_head;
        kr.k_pos = a.pk_pos;
        kr.v_pos = a.pv_pos;
        attend<DT, D, MTP>(a, kr, row0, nrows, hk, tile, 0, split, s_mem);
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
        share(total, split, a.ssplits, &kr.begin, &kr.end);
        kr.total = total;
        kr.k = a.sk + (int64_t)b * a.sk_seq + (int64_t)hk * a.sk_head;
        kr.v = a.sv + (int64_t)b * a.sv_seq + (int64_t)hk * a.sv_head;
        kr.k_pos = a.sk_pos;
        kr.v_pos = a.sv_pos;
        attend<DT, D, MTS>(a, kr, row0, nrows, hk, tile, nrows - 1, a.psplits + split, s_mem);
    }
}

// Join of the parts: one thread per 4 columns of a (row, head).
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnArgs a)
{
    constexpr int TPR = D / 4;
    const int64_t n = (int64_t)a.rows * a.q_heads;
    const int64_t i = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    if (i >= n) return;
    const int d = (threadIdx.x % TPR) * 4;
    const int slots = a.psplits + a.ssplits;
    float m = kNoReference;
    for (int s = 0; s < slots; ++s) m = fmaxf(m, a.ml[s * n + i].x);
    float l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < slots; ++s) {
        const float2 p = a.ml[s * n + i];
        if (p.y == 0.0f) continue;  // a part without a visible key
        const float f = __builtin_amdgcn_exp2f(p.x - m);
        l += p.y * f;
        o += *(const SV_GLOBAL f32x4*)(a.acc + (s * n + i) * D + d) * f;
    }
    const int32_t t = (int32_t)(i / a.q_heads), h = (int32_t)(i - (int64_t)t * a.q_heads);
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    u32x2 w;
    w.x = pack2<DT>(o.x * inv, o.y * inv);
    w.y = pack2<DT>(o.z * inv, o.w * inv);
    *(SV_GLOBAL u32x2*)(a.out + (int64_t)t * a.out_row + (int64_t)h * a.out_head + d * 2) = w;
    if (a.lse != nullptr && d == 0)
        a.lse[i] = l > 0.0f ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f : neg_inf();
}

}  // namespace sv
