// Verify of a tree of guesses: every row's own token (the argmax of the row, or
// a draw from it) is known; the walk from row 0 takes, at each row, the first
// guess that extends the row and equals the row's token.
//
// One workgroup per sequence.  The rows' tokens are found side by side (16 lanes
// per row merge its chunks' maxima) and kept in LDS, so a step of the walk costs
// an LDS read and two ballots, not a trip to memory.  The logits' one read bounds
// the call: 64 ragged trees of up to 24 guesses, 755 rows of 128256 bf16 logits
// (194 MB): 35 us; one tree of 12 guesses on 50304 fp32 logits: 7.7 us, latency.
#pragma once

#include "sv_common.hpp"

namespace sv {

constexpr int kTreeMostRows = 129;  // guesses of a sequence, and row 0
constexpr int kTreeGroup = 16;      // lanes that merge a row's chunks

struct TreeWalkArgs {
    const int32_t *cu, *ids, *parents;  // parents nullptr: the chain
    int32_t batch, kmax, total_draft, vocab, nchunk;
    const PartialArg* partials;   // greedy: [row][chunk]
    const int32_t* row_tokens;    // sampling: [row]
    int32_t *out_tokens, *out_nacc, *out_path;
};

template <bool GREEDY>
__global__ __launch_bounds__(kThreads) void tree_walk_kernel(TreeWalkArgs a)
{
    __shared__ int32_t s_tok[kTreeMostRows + 7], s_path[kTreeMostRows + 7];
    __shared__ int32_t s_n;
    const int32_t b = (int32_t)blockIdx.x, tid = (int32_t)threadIdx.x;
    int32_t k0 = b * a.kmax, kb = a.kmax;
    if (a.cu != nullptr) {
        k0 = a.cu[b];
        const int32_t k1 = a.cu[b + 1];
        kb = k1 - k0;
        if (k0 < 0 || kb < 0 || kb > a.kmax || k1 > a.total_draft) {
            if (tid == 0) a.out_nacc[b] = -1;
            return;
        }
    }
    const int32_t row0 = k0 + b;
    // this wave's own copy of the guesses, two per lane (every wave holds it; the first one walks)
    int32_t id[2] = {-1, -1}, up[2] = {-1, -1};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int32_t j = lane_id() + i * kWave;
        if (j < kb) {
            id[i] = a.ids[k0 + j];
            up[i] = a.parents != nullptr ? a.parents[k0 + j] : j;
            bad |= id[i] < 0 || id[i] >= a.vocab || up[i] < 0 || up[i] > j;
        }
    }
    if constexpr (GREEDY) {
        const int32_t l = tid % kTreeGroup;
        for (int32_t r = tid / kTreeGroup; r <= kb; r += kThreads / kTreeGroup) {
            const PartialArg* pp = a.partials + (int64_t)(row0 + r) * a.nchunk;
            float v = neg_inf();
            int32_t ix = INT32_MAX;
            for (int32_t ch = l; ch < a.nchunk; ch += kTreeGroup) argmax_merge(v, ix, pp[ch].m, pp[ch].idx);
#pragma unroll
            for (int o = kTreeGroup / 2; o > 0; o >>= 1) {
                const float ov = __shfl_xor(v, o, kWave);
                const int32_t oi = __shfl_xor(ix, o, kWave);
                argmax_merge(v, ix, ov, oi);
            }
            if (l == 0) s_tok[r] = ix;
        }
    } else {
        for (int32_t r = tid; r <= kb; r += kThreads) s_tok[r] = a.row_tokens[row0 + r];
    }
    __syncthreads();
    if (wave_id() == 0) {
        const bool any = __any(bad);
        int32_t n = 0, r = 0;
        while (!any) {  // (r rises: at most kb steps)
            if (lane_id() == 0) s_path[n] = r;
            const int32_t t = s_tok[r];
            const uint64_t lo = __ballot(up[0] == r && id[0] == t), hi = __ballot(up[1] == r && id[1] == t);
            if ((lo | hi) == 0) break;
            r = lo != 0 ? __builtin_ctzll(lo) + 1 : __builtin_ctzll(hi) + kWave + 1;
            ++n;
        }
        if (lane_id() == 0) {
            s_n = any ? -1 : n;
            a.out_nacc[b] = any ? -1 : n;
        }
    }
    __syncthreads();
    const int32_t n = s_n;
    if (n < 0) return;
    for (int32_t i = tid; i <= kb; i += kThreads) {
        const int32_t at = i <= n ? s_path[i] : -1;
        a.out_tokens[row0 + i] = i <= n ? s_tok[at] : -1;  // (an accepted guess is the token of the row it extends)
        if (a.out_path != nullptr) a.out_path[row0 + i] = at;
    }
}

}  // namespace sv
