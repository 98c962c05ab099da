// Beam search's selection: for every group of W beams, the n candidates
// (beam w, token v) of largest score
//     s(w, v) = cum_w + l_wv / T - lse_w,   lse_w = log sum_u exp(l_wu / T),
// ties to the lowest w * V + v.
//
// Two kernels.  beam_stream_kernel reads every logit once (HBM bound) and
// leaves, per 256-byte block of a row, the block's largest logit (1/64 of the
// bytes read for 16-bit logits, 1/64 for fp32), and per wave's tile its
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
// Which candidate of two beams is ahead may hang on the last bits of two
// lse_w.  Scores are formed in fp64; the streaming sums carry fp32 terms.
// With x = (m - l) / T >= 0 for the maximum m, one term exp2(-x log2 e) is off
// by at most (3 x + 2) 2^-24 relative (difference, log2(e) / T and product
// each rounded once; exp2 good to one ulp), eight of them are added in fp32
// (7 * 2^-24), everything after that in fp64.  The mean of x under the softmax
// is at most ln V <= 13.9, so lse_w is off by at most
// (3 * 13.9 + 9) 2^-24 < 3.1e-6.  Two candidates of different beams whose
// scores lie within twice that (kBeamWindow) are not decided by these sums:
// the pick then recomputes the lse_w concerned in fp64 from the rows and
// selects again, so the order is always the fp64 scores' order.
#pragma once

#include "sv_common.hpp"
#include "sv_stats.hpp"
#include "sv_stream.hpp"

namespace sv {

constexpr int kBeamMaxBeams = 64;
constexpr int kBeamMaxSelect = 128;
constexpr int kBeamBlockBytes = 256;  // 16 lanes' 16-byte loads
constexpr int kPickThreads = 1024;
constexpr int kPickWaves = kPickThreads / kWave;
constexpr int kPickCap = 1024;   // candidate blocks, and candidate elements, held in LDS
constexpr int kPickBins = 256;   // maxima the pick's lower bound is taken from (at least kBeamMaxSelect)
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

// One workgroup per (row, chunk) tile.  blkmax[row][chunk * LOADS * 16 + i]:
// the largest logit of the tile's i-th 256-byte block (-inf outside the row);
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
    float* bm = blkmax + (int64_t)t.row * nblkp + t.cb0 / 16 + (threadIdx.x >> 4);
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
        if ((threadIdx.x & 15) == 0) bm[i * (kThreads / 16)] = b;
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

template <int DT>
__global__ __launch_bounds__(kPickThreads) void beam_pick_kernel(PickArgs a)
{
    constexpr int ES = Dt<DT>::kSize;
    constexpr int BE = kBeamBlockBytes / ES;  // elements per block
    __shared__ double s_off[kBeamMaxBeams];   // score = s_off + (l - s_top) / T; -inf: the beam gives no candidate
    __shared__ float s_top[kBeamMaxBeams];    // the row's largest logit
    __shared__ int32_t s_end[kBeamMaxBeams];  // ended beam: 1
    __shared__ uint32_t s_key[kPickThreads];
    __shared__ double s_bs[kPickCap];
    __shared__ int32_t s_bi[kPickCap];
    __shared__ double s_es[kPickCap];
    __shared__ int32_t s_ei[kPickCap];
    __shared__ double s_ss[kBeamMaxSelect];   // the selected blocks, later the selected candidates
    __shared__ int32_t s_si[kBeamMaxSelect];
    __shared__ int32_t s_cnt, s_ecnt, s_bound;
    __shared__ uint32_t s_mark[2];
    __shared__ double s_red[kPickWaves];
    __shared__ int32_t s_redi[kPickWaves];

    const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
    const int32_t g = (int32_t)blockIdx.x, W = a.beams, V = a.vocab, n = a.nsel;
    const int32_t row0 = g * W;
    const double T = (double)a.temperature;
    const double ninf = -__builtin_inf();

    auto mis_of = [&](int32_t w) { return (int32_t)(((uintptr_t)row_ptr(a.rs, row0 + w) & 15u) / ES); };
    // an ended beam's only block with a candidate
    auto pad_block = [&](int32_t w) { return (a.pad_token + mis_of(w)) / BE; };

    // ---- the beams' offsets: cum - lse, one wave per beam in turn
    for (int32_t w = wave; w < W; w += kPickWaves) {
        const int32_t row = row0 + w;
        const float cum = a.cum[row];
        double off = ninf;
        float top = neg_inf();
        int32_t ended = 0;
        if (beam_streams(a.cum, a.finished, row)) {
            const BeamPart* p = a.parts + (int64_t)row * a.nparts;
            float m = neg_inf();
            for (int32_t i = lane; i < a.nparts; i += kWave) m = fmaxf(m, p[i].m);
            top = wave_max_dpp(m);
            double s = 0.0;
            for (int32_t i = lane; i < a.nparts; i += kWave) {
                const float pm = p[i].m;
                const double ps = p[i].s;
                // a part with no finite logit holds 0 (or NaN, from a NaN logit)
                s += pm == neg_inf() ? ps : ps * exp(((double)pm - (double)top) / T);
            }
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
            s_end[w] = ended;
        }
    }
    if (tid < 2) s_mark[tid] = 0u;
    __syncthreads();

    const int32_t per_row = a.nblkp / kWave;  // runs of 64 blocks per row: a wave's run lies in one row
    // the largest score of block `blk` of beam w
    auto block_score = [&](int32_t w, int32_t blk) -> double {
        const double off = s_off[w];
        if (off == ninf || blk >= a.nblk) return ninf;
        if (s_end[w] != 0) return blk == pad_block(w) ? off : ninf;
        return off + ((double)a.blkmax[(int64_t)(row0 + w) * a.nblkp + blk] - (double)s_top[w]) / T;
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
        // ---- a lower bound of the n-th best block: the n-th largest of kPickBins bins' maxima (fp32 keys: the
        // rounding keeps the order, so every block at or above the n-th best has a key at or above the bound)
        if (tid == 0) s_cnt = s_ecnt = 0;
        float km = neg_inf();
        for (int32_t q = wave; q < W * per_row; q += kPickWaves) {
            const int32_t w = q / per_row;
            km = fmaxf(km, (float)block_score(w, (q - w * per_row) * kWave + lane));
        }
        s_key[tid] = order_key(km);
        __syncthreads();
        if (wave == 0) {
            uint32_t k[kPickBins / kWave];
#pragma unroll
            for (int j = 0; j < kPickBins / kWave; ++j) {
                k[j] = 0u;
#pragma unroll
                for (int i = 0; i < kPickThreads / kPickBins; ++i)
                    k[j] = max(k[j], s_key[(i * (kPickBins / kWave) + j) * kWave + lane]);
            }
            uint32_t cur = 0u;
            for (int b = 31; b >= 0; --b) {
                const uint32_t t = cur | (1u << b);
                int cnt = 0;
#pragma unroll
                for (int j = 0; j < kPickBins / kWave; ++j) cnt += __popcll(__ballot(k[j] >= t));
                if (cnt >= n) cur = t;
            }
            if (lane == 0) s_bound = (int32_t)cur;
        }
        __syncthreads();
        const uint32_t bound = (uint32_t)s_bound;
        // one fp32 step below the bound, less the window: an fp64 score under it cannot matter
        const double low = bound <= order_key(neg_inf())
                               ? ninf
                               : (double)key_to_float(bound) - fabs((double)key_to_float(bound)) * 0x1p-23 - 1e-30 - win;
        // ---- the blocks at or above it
        for (int32_t q = wave; q < W * per_row; q += kPickWaves) {
            const int32_t w = q / per_row;
            const int32_t blk = (q - w * per_row) * kWave + lane;
            const double s = block_score(w, blk);
            if (s >= low && s > ninf) {
                const int32_t at = atomicAdd(&s_cnt, 1);
                if (at < kPickCap) {
                    s_bs[at] = s;
                    s_bi[at] = w * a.nblkp + blk;
                }
            }
        }
        __syncthreads();
        const int32_t cnt = s_cnt;
        int32_t nblocks = min(cnt, n);
        bool overflow = cnt > kPickCap;
        int32_t rb = 0;  // this thread's block's place
        if (!overflow) {
            if (tid < cnt) {
                const double s = s_bs[tid];
                const int32_t i = s_bi[tid];
                for (int32_t j = 0; j < cnt; ++j) rb += ahead(s_bs[j], s_bi[j], s, i) ? 1 : 0;
                if (rb < n) {
                    s_ss[rb] = s;
                    s_si[rb] = i;
                }
            }
            __syncthreads();
        } else if (pass > 0) {
            // more ties than the list holds: take the first n blocks one after another
            double ps = __builtin_inf();
            int32_t pi = -1;
            for (nblocks = 0; nblocks < n; ++nblocks) {
                double bs = ninf;
                int32_t bi = INT32_MAX;
                for (int32_t q = wave; q < W * per_row; q += kPickWaves) {
                    const int32_t w = q / per_row;
                    const int32_t blk = (q - w * per_row) * kWave + lane;
                    const double s = block_score(w, blk);
                    const int32_t i = w * a.nblkp + blk;
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
            const double elow = nblocks == n ? s_ss[n - 1] - win : ninf;
            for (int32_t e = tid; e < nblocks * BE; e += kPickThreads) {
                const int32_t bi = s_si[e / BE];
                const int32_t w = bi / a.nblkp;
                int32_t pos = 0;
                const double s = element_score(w, bi - w * a.nblkp, e % BE, &pos);
                if (s >= elow && s > ninf) {
                    const int32_t at = atomicAdd(&s_ecnt, 1);
                    if (at < kPickCap) {
                        s_es[at] = s;
                        s_ei[at] = pos;
                    }
                }
            }
            __syncthreads();
            const int32_t ecnt = s_ecnt;
            nout = min(ecnt, n);
            if (ecnt <= kPickCap) {
                int32_t r = n;
                if (tid < ecnt) {
                    const double s = s_es[tid];
                    const int32_t i = s_ei[tid];
                    r = 0;
                    for (int32_t j = 0; j < ecnt; ++j) r += ahead(s_es[j], s_ei[j], s, i) ? 1 : 0;
                    if (r < n) {
                        s_ss[r] = s;  // (the blocks' places are no longer needed: see the barrier above)
                        s_si[r] = i;
                    }
                }
                __syncthreads();
                if (pass == 0) {
                    // candidates of different beams closer than the window, in the list or just outside it
                    if (tid + 1 < nout) {
                        const int32_t w0 = s_si[tid] / V, w1 = s_si[tid + 1] / V;
                        if (w0 != w1 && s_ss[tid] - s_ss[tid + 1] <= win) {
                            mark(w0);
                            mark(w1);
                        }
                    }
                    if (nout == n) {
                        const double last = s_ss[n - 1];
                        const int32_t wl = s_si[n - 1] / V;
                        if (tid < ecnt && r >= n && s_es[tid] >= last - win && s_ei[tid] / V != wl) {
                            mark(wl);
                            mark(s_ei[tid] / V);
                        }
                        // (a block that was not read: its largest element is outside)
                        if (tid < cnt && rb >= n && s_bs[tid] >= last - win && s_bi[tid] / a.nblkp != wl) {
                            mark(wl);
                            mark(s_bi[tid] / a.nblkp);
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
                        const int32_t w = blk / a.nblkp;
                        int32_t pos = 0;
                        const double s = element_score(w, blk - w * a.nblkp, e % BE, &pos);
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
            const double m = (double)s_top[w];
            double s = 0.0;
#pragma unroll 4
            for (int32_t v = tid; v < V; v += kPickThreads) s += exp(((double)load_one<DT>(row, v) - m) / T);
            s = wave_sum_dpp(s);
            __syncthreads();
            if (lane == 0) s_red[wave] = s;
            __syncthreads();
            if (tid == 0) {
                double t = 0.0;
                for (int k = 0; k < kPickWaves; ++k) t += s_red[k];
                s_off[w] = (double)a.cum[row0 + w] - log(t);
            }
        }
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
