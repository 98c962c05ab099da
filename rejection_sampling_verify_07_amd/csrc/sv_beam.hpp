// Beam search's selection: for every group of W beams, the n candidates
// (beam w, token v) of largest score
//     s(w, v) = cum_w + l_wv / T - lse_w,   lse_w = log sum_u exp(l_wu / T),
// ties to the lowest w * V + v.
//
// Two kernels.  beam_stream_kernel reads every logit once (HBM bound) and
// leaves, per 512-byte block of a row, the block's largest logit (1/128 of the
// bytes read), and per wave's tile its
// maximum and sum of exponentials.  beam_pick_kernel, one workgroup per group,
// merges the sums into lse_w and needs only those n blocks that come first by
// (largest score, position): blocks are contiguous runs of w * V + v, so a
// candidate outside them has n block maxima ahead of it.  It reads the n
// blocks again (they are a few kB) and ranks their elements.
//
// The score is formed as (cum_w - log S_w) + (l - m_w) / T with m_w the row's
// largest logit and S_w = sum_u exp((l_wu - m_w) / T): the difference is exact
// in fp64 and no large terms cancel.
//
// 512 rows of 151936 bf16 logits (64 groups of 8, 16 kept): streaming pass 31 us,
// 5.0 TB/s; pick 13 us.  4 rows of 50304 fp32: 3 and 9 us.  The pick is a
// chain of latencies: offsets 2 us (two memory rounds, one fp64 log), then
// scores, bound, gather, block ranking, element loads and ranking, 0.7 to 1 us each.
//
// Which candidate of two beams is ahead may hang on the last bits of two
// lse_w.  Scores are formed in fp64; the streaming sums carry fp32 terms.
// With x = (m - l) / T >= 0 for the maximum m, one term exp2(-x log2 e) is off
// by at most (3 x + 2) 2^-24 relative (difference, log2(e) / T and product
// each rounded once; exp2 good to one ulp), eight of them are added in fp32
// (7 * 2^-24), everything after that in fp64.  The mean of x under the softmax
// is at most ln V <= 13.9, so lse_w is off by at most
// (3 * 13.9 + 9) 2^-24 < 3.1e-6.  Two candidates of different beams whose
// scores lie within twice that (kBeamWindow) and a few of the scores' own fp64
// steps are not decided by these sums: the pick then recomputes the log sums
// concerned in fp64 from the rows and selects again, so the order is always the
// fp64 scores' order.  A group that
// needs it takes 32 us more per beam of 151936 logits; on random logits that is
// rare (two scores of different beams have to lie within the window).
#pragma once

#include "sv_common.hpp"
#include "sv_stats.hpp"
#include "sv_stream.hpp"

namespace sv {

constexpr int kBeamMaxBeams = 64;
constexpr int kBeamMaxSelect = 128;
constexpr int kBeamBlockBytes = 512;  // 32 lanes' 16-byte loads
// The pick's workgroup.  The pick is a chain of short steps, 0.5 to 1 us each, between barriers; 256 threads take
// longer for it even where a group has few blocks (12.8 against 10.2 us for 4 beams of 50304 logits), 512 as long.
constexpr int kPickThreads = 1024;
constexpr int kPickWaves = kPickThreads / kWave;
constexpr int kPickCap = 1024;  // candidate blocks, and candidate elements, held in LDS
constexpr int kPickBins = 256;   // maxima the pick's lower bound is taken from (at least kBeamMaxSelect)
constexpr int kPickHeld = 8;     // block maxima a thread holds at a time
constexpr double kBeamWindow = 6.4e-6;
static_assert(kPickBins >= kBeamMaxSelect, "the bound needs one bin per selected candidate");

struct BeamPart {  // one wave's share of a row: its maximum and sum of exp((l - m) / T)
    double s;
    float m;
    int32_t pad;
};

// A beam takes part with its row's logits when its score is finite and it has not ended.
__device__ __forceinline__ bool beam_streams(const float* cum, const uint8_t* finished, int32_t row)
{
    const float s = cum[row];
    return s - s == 0.0f && !(finished != nullptr && finished[row] != 0);
}

// One workgroup per (row, chunk) tile.  blkmax[row][chunk * LOADS * 8 + i]:
// the largest logit of the tile's i-th 512-byte block (-inf outside the row);
// parts[row][chunk * 4 + wave].  Rows that do not take part are not read.
template <int DT, int LOADS>
__global__ __launch_bounds__(kThreads) void beam_stream_kernel(RowSet rs, const float* __restrict__ cum,
                                                               const uint8_t* __restrict__ finished, int32_t vocab,
                                                               int32_t nchunk, int32_t nblkp, float c,
                                                               float* __restrict__ blkmax, BeamPart* __restrict__ parts)
{
    constexpr int VEC = Dt<DT>::kVec;
    const u32x4* base;
    u32x4 raw[LOADS];
    const Tile t = make_tile<DT>(rs, vocab, nchunk, (int32_t)blockIdx.x, LOADS, &base);
    if (!beam_streams(cum, finished, t.row)) return;
    issue_tile<DT, LOADS, true>(t, base, raw);
    sanitize_edge<DT, LOADS>(t, vocab, raw);
    float tm = neg_inf();
    float* bm = blkmax + (int64_t)t.row * nblkp + t.cb0 / 32 + (threadIdx.x >> 5);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        float f[VEC];
        unpack<DT>(raw[i], f);
        float b = f[0];
#pragma unroll
        for (int e = 1; e < VEC; ++e) b = fmaxf(b, f[e]);
        const int ninf = __float_as_int(neg_inf());
        b = fmaxf(b, __int_as_float(dpp_mov<kDppQuad1032>(ninf, __float_as_int(b))));
        b = fmaxf(b, __int_as_float(dpp_mov<kDppQuad2301>(ninf, __float_as_int(b))));
        b = fmaxf(b, __int_as_float(dpp_mov<kDppHalfMirror>(ninf, __float_as_int(b))));
        b = fmaxf(b, __int_as_float(dpp_mov<kDppMirror>(ninf, __float_as_int(b))));
        // row_bcast:15 brings row 0's maximum to row 1 and row 2's to row 3
        b = fmaxf(b, __int_as_float(dpp_mov<kDppBcast15, 0xa>(ninf, __float_as_int(b))));
        if ((threadIdx.x & 31) == 31) bm[i * (kThreads / 32)] = b;
        tm = fmaxf(tm, b);
    }
    const float wm = wave_max_dpp(tm);
    // an all -inf tile keeps a finite reference, so that a NaN among its elements still reaches the sum
    const float m = wm == neg_inf() ? 0.0f : wm;
    double acc = 0.0;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        float f[VEC];
        unpack<DT>(raw[i], f);
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += __builtin_amdgcn_exp2f((f[e] - m) * c);
        acc += (double)s;
    }
    acc = wave_sum_dpp(acc);
    if (lane_id() == 0) {
        BeamPart* out = parts + (int64_t)t.index * kWaves + wave_id();
        out->s = acc;
        out->m = wm;
    }
}

struct PickArgs {
    RowSet rs;
    const float* cum;
    const uint8_t* finished;
    int32_t beams, vocab, nsel;
    int32_t nparts;  // BeamPart entries per row
    int32_t nblk;    // blocks per row that the streaming pass wrote
    int32_t nblkp;   // blocks per row in memory, a multiple of 64
    int32_t pad_token;
    float temperature;
    const float* blkmax;
    const BeamPart* parts;
    float* out_scores;
    int32_t* out_tokens;
    int32_t* out_parents;
};

// (score, position) order: larger score first, then the lower position.
__device__ __forceinline__ bool ahead(double sa, int32_t ia, double sb, int32_t ib)
{
    return sa > sb || (sa == sb && ia < ib);
}

// exp(x) in fp64 for x <= 0 (and NaN): 2^(n / 32) from a table and exp of the
// rest, at most ln 2 / 64 = 0.0109, by its series to the 6th power (the next
// term is below 4e-18 relative).  The form of P. T. P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point
// arithmetic", ACM TOMS 15 (1989), with a Taylor series for its polynomial.
// About a dozen fp64 instructions; the library's exp took four times as long
// over a row.
constexpr int kExpTable = 32;
static __device__ const double kExp2Of32nds[kExpTable] = {  // 2^(j / 32)
    0x1.0000000000000p+0, 0x1.059b0d3158574p+0, 0x1.0b5586cf9890fp+0, 0x1.11301d0125b51p+0,
    0x1.172b83c7d517bp+0, 0x1.1d4873168b9aap+0, 0x1.2387a6e756238p+0, 0x1.29e9df51fdee1p+0,
    0x1.306fe0a31b715p+0, 0x1.371a7373aa9cbp+0, 0x1.3dea64c123422p+0, 0x1.44e086061892dp+0,
    0x1.4bfdad5362a27p+0, 0x1.5342b569d4f82p+0, 0x1.5ab07dd485429p+0, 0x1.6247eb03a5585p+0,
    0x1.6a09e667f3bcdp+0, 0x1.71f75e8ec5f74p+0, 0x1.7a11473eb0187p+0, 0x1.82589994cce13p+0,
    0x1.8ace5422aa0dbp+0, 0x1.93737b0cdc5e5p+0, 0x1.9c49182a3f090p+0, 0x1.a5503b23e255dp+0,
    0x1.ae89f995ad3adp+0, 0x1.b7f76f2fb5e47p+0, 0x1.c199bdd85529cp+0, 0x1.cb720dcef9069p+0,
    0x1.d5818dcfba487p+0, 0x1.dfc97337b9b5fp+0, 0x1.ea4afa2a490dap+0, 0x1.f50765b6e4540p+0,
};
__device__ __forceinline__ double exp_f64(double x, const double* table)
{
    const double n = __builtin_rint(x * (kExpTable * 1.4426950408889634));
    // ln 2 / 32 in two parts, the first of 25 bits: its product with n (16 bits where the result is not 0) is exact
    const double r = __builtin_fma(n, -0x1.f473de6af278fp-35, __builtin_fma(n, -0x1.62e42fep-6, x));
    double p = __builtin_fma(r, 1.0 / 720, 1.0 / 120);
    p = __builtin_fma(r, p, 1.0 / 24);
    p = __builtin_fma(r, p, 1.0 / 6);
    p = __builtin_fma(r, p, 0.5);
    p = __builtin_fma(r, p, 1.0);
    p = __builtin_fma(r, p, 1.0);
    const int k = (int)n;
    const double e = __builtin_ldexp(p * table[k & (kExpTable - 1)], k >> 5);
    return x < -800.0 ? 0.0 : e;
}

// What the fp32 pass over the block maxima needs of a beam: a block's score is
// off + (m - top) / T for blocks first .. last, -inf elsewhere.  (An ended
// beam: off at its pad token's block, with scale 0 for whatever m holds there.)
struct BeamView {
    float off, top;
    int32_t first, last;
};

template <int DT>
__global__ __launch_bounds__(kPickThreads) void beam_pick_kernel(PickArgs a)
{
    constexpr int ES = Dt<DT>::kSize;
    constexpr int BE = kBeamBlockBytes / ES;  // elements per block
    __shared__ double s_off[kBeamMaxBeams];   // score = s_off + (l - s_top) / T; -inf: the beam gives no candidate
    __shared__ __align__(16) BeamView s_view[kBeamMaxBeams];
    __shared__ float s_top[kBeamMaxBeams];    // the row's largest logit
    __shared__ int32_t s_end[kBeamMaxBeams];  // ended beam: 1
    __shared__ float s_bin[kPickThreads];
    __shared__ double s_bs[kPickCap];
    __shared__ int32_t s_bi[kPickCap];
    __shared__ float s_bm[kPickCap];
    __shared__ int32_t s_br[kPickCap];
    __shared__ double s_es[kPickCap];
    __shared__ int32_t s_ei[kPickCap];
    __shared__ int32_t s_er[kPickCap];
    __shared__ double s_ss[kBeamMaxSelect];   // the selected blocks, later the selected candidates
    __shared__ int32_t s_si[kBeamMaxSelect];
    __shared__ int32_t s_cnt, s_ecnt;
    __shared__ float s_bound;
    __shared__ uint32_t s_mark[2];
    __shared__ double s_red[kPickWaves];
    __shared__ int32_t s_redi[kPickWaves];
    __shared__ double s_exp[kExpTable];

    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
    const int32_t g = (int32_t)blockIdx.x, W = a.beams, V = a.vocab, n = a.nsel;
    const int32_t row0 = g * W;
    const double T = (double)a.temperature;
    const double ninf = -__builtin_inf();

    auto mis_of = [&](int32_t w) { return (int32_t)(((uintptr_t)row_ptr(a.rs, row0 + w) & 15u) / ES); };
    // an ended beam's only block with a candidate
    auto pad_block = [&](int32_t w) { return (a.pad_token + mis_of(w)) / BE; };

    // ---- the block maxima, before anything that their scores wait for (blocks of beams that were not streamed hold
    // old bytes, which block_score ignores)
    const int32_t per_row = a.nblkp / kWave;  // runs of 64 blocks per row: a wave's run lies in one row
    const int32_t runs = W * per_row;
    // A wave's runs wave, wave + 16, ... as (beam, run of its row).  The quotient by a multiplication: runs < 2^14 and
    // per_row <= 2^8, so the rounded-up reciprocal's excess, below 2^-24 per run, never reaches the next integer.
    struct Run {
        int32_t q, w, r;
    };
    const uint32_t recip = per_row > 1 ? (uint32_t)(0xffffffffu / (uint32_t)per_row) + 1u : 0u;
    // (the empty asm keeps the compiler from computing every run once, up front, and holding all of them: that spilled
    // 588 bytes a lane)
    auto run_at = [&](int32_t q) {
        asm volatile("" : "+s"(q));
        const int32_t w = per_row > 1 ? (int32_t)__umulhi((uint32_t)q, recip) : q;
        return Run{q, w, q - w * per_row};
    };
    auto next_run = [&](Run& c) { c = run_at(c.q + kPickWaves); };
    const float* blkmax = a.blkmax + (int64_t)row0 * a.nblkp;
    constexpr int kGroupRuns = kPickHeld * kPickWaves;  // runs that the workgroup's registers hold at a time
    float held[kPickHeld];
    auto bring = [&](int32_t q0) {
#pragma unroll
        for (int j = 0; j < kPickHeld; ++j) {
            const int32_t q = q0 + wave + j * kPickWaves;
            held[j] = q < runs ? blkmax[q * kWave + lane] : 0.0f;
        }
    };
    bring(0);

    if (tid < kExpTable) s_exp[tid] = kExp2Of32nds[tid];
    __syncthreads();

    // ---- the beams' offsets: cum - log S, one wave per beam in turn
    for (int32_t w = wave; w < W; w += kPickWaves) {
        const int32_t row = row0 + w;
        // (parts of a beam that was not streamed hold old bytes and are not used)
        const BeamPart* p = a.parts + (int64_t)row * a.nparts;
        BeamPart first{0.0, neg_inf(), 0};  // this lane's first part stays in registers
        if (lane < a.nparts) first = p[lane];
        const float cum = a.cum[row];
        double off = ninf;
        float top = neg_inf();
        int32_t ended = 0;
        if (beam_streams(a.cum, a.finished, row)) {
            float m = first.m;
            for (int32_t i = lane + kWave; i < a.nparts; i += kWave) m = fmaxf(m, p[i].m);
            top = wave_max_dpp(m);
            // a part with no finite logit holds 0 (or NaN, from a NaN logit)
            auto share = [&](float pm, double ps) {
                return pm == neg_inf() ? ps : ps * exp_f64(((double)pm - (double)top) / T, s_exp);
            };
            double s = share(first.m, first.s);
            for (int32_t i = lane + kWave; i < a.nparts; i += kWave) s += share(p[i].m, p[i].s);
            s = wave_sum_dpp(s);
            off = (double)cum - log(s);
            if (!(off - off == 0.0)) off = ninf;  // no finite logit, or NaN or +inf among them
        } else if (cum - cum == 0.0f) {
            ended = 1;
            off = (double)cum;
        }
        if (lane == 0) {
            s_off[w] = off;
            s_top[w] = top;
            s_view[w] = off == ninf ? BeamView{0.0f, 0.0f, 1, 0}
                        : ended     ? BeamView{(float)off, __builtin_nanf(""), pad_block(w), pad_block(w)}
                                    : BeamView{(float)off, top, 0, a.nblk - 1};
            s_end[w] = ended;
        }
    }
    if (tid < 2) s_mark[tid] = 0u;
    __syncthreads();

    // the largest score of block `blk` of beam w, and its fp32 form
    auto block_score = [&](int32_t w, int32_t blk, float m) -> double {
        const double off = s_off[w];
        if (off == ninf || blk >= a.nblk) return ninf;
        if (s_end[w] != 0) return blk == pad_block(w) ? off : ninf;
        return off + ((double)m - (double)s_top[w]) / T;
    };
    // (fp32 may overflow where fp64 does not: only a logit of -inf is no candidate, so everything else stays finite here,
    // and the fp64 scores decide)
    const float inv_t = 1.0f / a.temperature;
    auto block_score_f = [&](int32_t w, int32_t blk, float m) -> float {
        const BeamView v = s_view[w];
        const bool ended = v.top != v.top;
        const float x = ended ? 0.0f : (m - v.top) * inv_t;
        return blk >= v.first && blk <= v.last && (ended || m > neg_inf()) ? fmaxf(v.off + x, -__FLT_MAX__) : neg_inf();
    };
    // The places of the first `count` entries (s, i) of two lists: place(entry, its place), called by one thread per
    // entry.  16 threads share an entry's comparisons.
    auto rank = [&](const double* ls, const int32_t* li, int32_t count, auto place) {
        for (int32_t c0 = 0; c0 < count; c0 += kPickThreads / 16) {
            const int32_t c = c0 + tid / 16, at = min(c, count - 1);
            const double s = ls[at];
            const int32_t i = li[at];
            int32_t r = 0;
#pragma unroll 4
            for (int32_t j = tid & 15; j < count; j += 16) r += ahead(ls[j], li[j], s, i) ? 1 : 0;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) r += __shfl_xor(r, o, kWave);
            if (c < count && (tid & 15) == 0) place(c, r);
        }
    };
    // the score of element j of block `blk` of beam w, and its position in the group
    auto element_score = [&](int32_t w, int32_t blk, int32_t j, int32_t* pos) -> double {
        const int32_t v = blk * BE + j - mis_of(w);
        if (v < 0 || v >= V) return ninf;
        *pos = w * V + v;
        if (s_end[w] != 0) return v == a.pad_token ? s_off[w] : ninf;
        return s_off[w] + ((double)load_one<DT>(row_ptr(a.rs, row0 + w), v) - (double)s_top[w]) / T;
    };
    auto mark = [&](int32_t w) { atomicOr(&s_mark[w >> 5], 1u << (w & 31)); };
    // the workgroup's first of the (s, i) that its threads bring, in s_red / s_redi[0]
    auto reduce_first = [&](double s, int32_t i) {
        for (int o = kWave / 2; o > 0; o >>= 1) {
            const double os = __shfl_xor(s, o, kWave);
            const int32_t oi = __shfl_xor(i, o, kWave);
            if (ahead(os, oi, s, i)) {
                s = os;
                i = oi;
            }
        }
        __syncthreads();
        if (lane == 0) {
            s_red[wave] = s;
            s_redi[wave] = i;
        }
        __syncthreads();
        if (tid == 0) {
            for (int k = 1; k < kPickWaves; ++k)
                if (ahead(s_red[k], s_redi[k], s_red[0], s_redi[0])) {
                    s_red[0] = s_red[k];
                    s_redi[0] = s_redi[k];
                }
        }
        __syncthreads();
    };

    int32_t nout = 0;
    for (int pass = 0;; ++pass) {
        const double win = pass == 0 ? kBeamWindow : 0.0;
        // ---- a lower bound of the n-th best block: the n-th largest of kPickBins bins' maxima, in fp32, by its
        // distance below the largest to 5 mantissa bits
        if (tid == 0) s_cnt = s_ecnt = 0;
        float km = neg_inf(), near[kPickHeld];
        auto score_group = [&](int32_t q0) {
            Run c = run_at(q0 + wave);
#pragma unroll
            for (int j = 0; j < kPickHeld; ++j) {
                near[j] = c.q < runs ? block_score_f(c.w, c.r * kWave + lane, held[j]) : neg_inf();
                km = fmaxf(km, near[j]);
                next_run(c);
            }
        };
        for (int32_t q0 = 0; q0 < runs; q0 += kGroupRuns) {
            if (q0 > 0) bring(q0);
            score_group(q0);
        }
        s_bin[tid] = km;
        float most = lane < W && s_view[lane].first <= s_view[lane].last ? fmaxf(s_view[lane].off, 0.0f) : 0.0f;
        most = wave_max_dpp(most);
        __syncthreads();
        if (wave == 0) {
            constexpr int KEYS = kPickBins / kWave;
            float v[KEYS], best = neg_inf();
#pragma unroll
            for (int j = 0; j < KEYS; ++j) {
                v[j] = neg_inf();
#pragma unroll
                for (int i = 0; i < kPickThreads / kPickBins; ++i)
                    v[j] = fmaxf(v[j], s_bin[(i * KEYS + j) * kWave + lane]);
                best = fmaxf(best, v[j]);
            }
            best = wave_max_dpp(best);
            uint32_t k[KEYS];
#pragma unroll
            for (int j = 0; j < KEYS; ++j) k[j] = __float_as_uint(best - v[j]) >> 18;
            uint32_t cur = 0u;  // the least prefix that n bins do not exceed
#pragma unroll
            for (int b = 12; b >= 0; --b) {
                const uint32_t t = cur + (1u << b);
                int cnt = 0;
#pragma unroll
                for (int j = 0; j < KEYS; ++j) cnt += __popcll(__ballot(k[j] < t));
                if (cnt < n) cur = t;
            }
            // An fp32 score is off by less than 2^-21 (|score| + |offset|): difference, 1 / T, product, offset and sum each
            // rounded once, (m - top) / T at most |score| + |offset| (a subnormal 1 / T keeps 2^-22).  No score exceeds its
            // beam's offset, so an offset below 0 is at most |score|: e = 2^-21 (2 |score| + the largest offset above 0),
            // and a beam at -1e9, a place not yet in use, widens no margin but its own.  The n bins are at least best - d
            // in fp32 (two roundings here), so at least that less e in fp64, and a block that reaches this less the window
            // has an fp32 score another e lower.  (A bound near fp32's lowest value becomes -inf here: every block with a
            // candidate passes.)
            const float d = __uint_as_float((cur << 18) | 0x3ffffu);
            float low = neg_inf();
            if (best != neg_inf() && d < __builtin_inff()) {
                const float bound = best - d;
                low = bound - 0x1p-20f * (3.0f * fabsf(bound) + 2.0f * most + fabsf(best)) - 1e-30f -
                      (float)(win * 1.01);
            }
            if (lane == 0) s_bound = low;
        }
        __syncthreads();
        const float low = s_bound;
        // ---- the blocks at or above it
        auto take = [&](const Run& c, float m) {
            const int32_t at = atomicAdd(&s_cnt, 1);
            if (at < kPickCap) {
                s_bm[at] = m;
                s_bi[at] = (c.w << 16) | (c.r * kWave + lane);  // in the order of positions
            }
        };
        for (int32_t q0 = 0; q0 < runs; q0 += kGroupRuns) {
            if (runs > kGroupRuns) {
                bring(q0);
                score_group(q0);
            }
            Run c = run_at(q0 + wave);
#pragma unroll
            for (int j = 0; j < kPickHeld; ++j) {
                if (near[j] >= low && near[j] > neg_inf()) take(c, held[j]);
                next_run(c);
            }
        }
        __syncthreads();
        const int32_t cnt = s_cnt;
        int32_t nblocks = min(cnt, n);
        bool overflow = cnt > kPickCap;
        if (!overflow) {
            for (int32_t c = tid; c < cnt; c += kPickThreads)
                s_bs[c] = block_score(s_bi[c] >> 16, s_bi[c] & 0xffff, s_bm[c]);
            __syncthreads();
            rank(s_bs, s_bi, cnt, [&](int32_t c, int32_t r) {
                s_br[c] = r;
                if (r < n) {
                    s_ss[r] = s_bs[c];
                    s_si[r] = s_bi[c];
                }
            });
            __syncthreads();
        } else if (pass > 0) {
            // more ties than the list holds: take the first n blocks one after another
            double ps = __builtin_inf();
            int32_t pi = -1;
            for (nblocks = 0; nblocks < n; ++nblocks) {
                double bs = ninf;
                int32_t bi = INT32_MAX;
                for (Run c = run_at(wave); c.q < runs; next_run(c)) {
                    const int32_t blk = c.r * kWave + lane, i = (c.w << 16) | blk;
                    const double s = block_score(c.w, blk, blkmax[c.q * kWave + lane]);
                    if (ahead(ps, pi, s, i) && ahead(s, i, bs, bi)) {
                        bs = s;
                        bi = i;
                    }
                }
                reduce_first(bs, bi);
                ps = s_red[0];
                pi = s_redi[0];
                if (ps == ninf) break;
                if (tid == 0) {
                    s_ss[nblocks] = ps;
                    s_si[nblocks] = pi;
                }
            }
            __syncthreads();
        }
        // ---- the elements of those blocks that can be among the first n
        if (!overflow || pass > 0) {
            // What may lie ahead of a score: the window, and what the fp64 roundings of two offsets and two scores make of
            // an offset that the window holds, half a step each (|offset| as in e above).
            auto reach = [&](double s) {
                return pass == 0 ? s - (kBeamWindow + 0x1p-50 * (2.0 * fabs(s) + (double)most)) : s;
            };
            const double elow = nblocks == n ? reach(s_ss[n - 1]) : ninf;
            // (fp32 scores first, with the margin of the bound above)
            const float elowf =
                elow == ninf ? neg_inf() : (float)elow - 0x1p-20f * (2.0f * fabsf((float)elow) + most) - 1e-30f;
            for (int32_t e0 = tid; e0 < nblocks * BE; e0 += 4 * kPickThreads) {
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t e = e0 + j * kPickThreads;
                    x[j] = neg_inf();
                    if (e < nblocks * BE) {
                        const int32_t bi = s_si[e / BE], w = bi >> 16;
                        const int32_t v = (bi & 0xffff) * BE + e % BE - mis_of(w);
                        if (v >= 0 && v < V && (s_end[w] == 0 || v == a.pad_token))
                            x[j] = s_end[w] != 0 ? 0.0f : load_one<DT>(row_ptr(a.rs, row0 + w), v);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t e = e0 + j * kPickThreads;
                    if (x[j] == neg_inf()) continue;
                    const int32_t bi = s_si[e / BE], w = bi >> 16;
                    if (block_score_f(w, bi & 0xffff, x[j]) < elowf) continue;
                    const double s = s_end[w] != 0 ? s_off[w] : s_off[w] + ((double)x[j] - (double)s_top[w]) / T;
                    if (!(s >= elow && s > ninf)) continue;
                    const int32_t at = atomicAdd(&s_ecnt, 1);
                    if (at < kPickCap) {
                        s_es[at] = s;
                        s_ei[at] = w * V + (bi & 0xffff) * BE + e % BE - mis_of(w);
                    }
                }
            }
            __syncthreads();
            const int32_t ecnt = s_ecnt;
            nout = min(ecnt, n);
            if (ecnt <= kPickCap) {
                rank(s_es, s_ei, ecnt, [&](int32_t c, int32_t r) {
                    s_er[c] = r;
                    if (r < n) {
                        s_ss[r] = s_es[c];  // (the blocks' places are no longer needed: see the barrier above)
                        s_si[r] = s_ei[c];
                    }
                });
                __syncthreads();
                if (pass == 0) {
                    // candidates of different beams closer than the window, in the list or just outside it
                    if (tid + 1 < nout) {
                        const int32_t w0 = s_si[tid] / V, w1 = s_si[tid + 1] / V;
                        if (w0 != w1 && s_ss[tid + 1] >= reach(s_ss[tid])) {
                            mark(w0);
                            mark(w1);
                        }
                    }
                    if (nout == n) {
                        const double edge = reach(s_ss[n - 1]);
                        const int32_t wl = s_si[n - 1] / V;
                        for (int32_t c = tid; c < ecnt; c += kPickThreads)
                            if (s_er[c] >= n && s_es[c] >= edge && s_ei[c] / V != wl) {
                                mark(wl);
                                mark(s_ei[c] / V);
                            }
                        // (a block that was not read: its largest element is outside)
                        for (int32_t c = tid; c < cnt; c += kPickThreads)
                            if (s_br[c] >= n && s_bs[c] >= edge && s_bi[c] >> 16 != wl) {
                                mark(wl);
                                mark(s_bi[c] >> 16);
                            }
                    }
                }
            } else if (pass > 0) {
                double ps = __builtin_inf();
                int32_t pi = -1;
                // (the selected blocks stay in s_ss / s_si; the candidates go to s_es / s_ei)
                for (nout = 0; nout < n; ++nout) {
                    double bs = ninf;
                    int32_t bi = INT32_MAX;
                    for (int32_t e = tid; e < nblocks * BE; e += kPickThreads) {
                        const int32_t blk = s_si[e / BE];
                        int32_t pos = 0;
                        const double s = element_score(blk >> 16, blk & 0xffff, e % BE, &pos);
                        if (s > ninf && ahead(ps, pi, s, pos) && ahead(s, pos, bs, bi)) {
                            bs = s;
                            bi = pos;
                        }
                    }
                    reduce_first(bs, bi);
                    ps = s_red[0];
                    pi = s_redi[0];
                    if (ps == ninf) break;
                    if (tid == 0) {
                        s_es[nout] = ps;
                        s_ei[nout] = pi;
                    }
                }
                __syncthreads();
                if (tid < nout) {
                    s_ss[tid] = s_es[tid];
                    s_si[tid] = s_ei[tid];
                }
            } else {
                overflow = true;
            }
        }
        __syncthreads();
        if (pass > 0) break;
        const uint64_t marked = overflow ? ~0ull : ((uint64_t)s_mark[1] << 32 | s_mark[0]);
        if (marked == 0) break;
        // ---- the marked beams' lse in fp64, from the rows
        for (int32_t w = 0; w < W; ++w) {
            if (!(marked >> w & 1) || s_end[w] != 0 || s_off[w] == ninf) continue;
            const char* row = row_ptr(a.rs, row0 + w);
            const double m = (double)s_top[w], inv = 1.0 / T;
            double s = 0.0;
            // Chunks of 16 bytes counted from the row's start wherever it lies (the loads need no alignment): the
            // same terms go to the same thread in the same order in every row, so rows that are copies of one
            // another get the same bits and tie.
            constexpr int VEC = Dt<DT>::kVec;
            typedef u32x4 loose __attribute__((aligned(2)));
            auto chunk = [&](int32_t k) { return *(const SV_GLOBAL loose*)(row + (int64_t)k * 16); };
            const int32_t nk = V / VEC;
            u32x4 ahead1{}, ahead2{};
            if (tid < nk) ahead1 = chunk(tid);
            if (tid + kPickThreads < nk) ahead2 = chunk(tid + kPickThreads);
            for (int32_t k = tid; k < nk; k += kPickThreads) {
                float x[VEC];
                unpack<DT>(ahead1, x);
                ahead1 = ahead2;
                if (k + 2 * kPickThreads < nk) ahead2 = chunk(k + 2 * kPickThreads);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    s += exp_f64(((double)x[j] - m) * inv, s_exp);
                    if (j & 1) __builtin_amdgcn_sched_barrier(0);  // more side by side spills registers
                }
            }
            for (int32_t v = nk * VEC + tid; v < V; v += kPickThreads)
                s += exp_f64(((double)load_one<DT>(row, v) - m) * inv, s_exp);
            s = wave_sum_dpp(s);
            __syncthreads();
            if (lane == 0) s_red[wave] = s;
            __syncthreads();
            if (tid == 0) {
                double t = 0.0;
                for (int k = 0; k < kPickWaves; ++k) t += s_red[k];
                s_off[w] = (double)a.cum[row0 + w] - log(t);
                s_view[w].off = (float)s_off[w];
            }
        }
        bring(0);  // (not held across the sums)
        __syncthreads();
    }
    if (tid < n) {
        const int64_t at = (int64_t)g * n + tid;
        const bool live = tid < nout;
        const int32_t pos = live ? s_si[tid] : 0;
        a.out_scores[at] = live ? (float)s_ss[tid] : neg_inf();
        a.out_tokens[at] = live ? pos % V : -1;
        a.out_parents[at] = live ? pos / V : -1;
    }
}

}  // namespace sv
