// Edits of logits before any selection: penalties for tokens already written,
// biases and grammar masks, in place or into another tensor.
//
//     x = l > 0 ? l / rep : l * rep   where the token was seen
//     x = x - freq n - pres [n > 0]   n: how often it was written
//     x = x + bias
//     x = -inf                        where the row's mask has no bit
//
// One workgroup takes CT neighbouring tokens of one sequence and a run of its
// rows.  It counts the sequence's history into a table of those tokens in LDS
// (integer atomics: any order gives the same counts) and lists the tokens met.
// Then two passes over its rows.  The first, in vectors of 16 bytes, copies
// (out of place) and masks: in place it touches only vectors with a masked token,
// and writes those that are masked whole without reading them.  The second goes
// through the list, all rows side by side, and edits single elements.  The
// guesses on a row's own path are few: a listed token that is a guess at all is
// compared with them one by one, so table and list are the same for all rows.  The
// history is read once per run of rows and CT tokens, from the caches; nothing needs
// a workspace.
//
// 320 rows of 151936 bf16 logits, texts of up to 8000 tokens, three of four sequences
// under masks, in place (97 MB): 45 us where the 256 MB cache holds the logits, 49 with
// three such sets in turn, 59 with four.  The masks alone take 21 and 28 of the 45 and 59
// (almost every line of a masked row is written), the penalties and biases alone 32 and
// 34: elements scattered over lines, and before them the chain of the text's read, the
// counts and the list.  43 ragged rows of 32003 fp16 logits, apart: 9.0 us; one row of
// 50304 fp32 logits, in place: 4.8 us, a launch and that chain.
//
// Arithmetic is fp32, each step rounded, the result rounded to the element type once.
#pragma once

#include "sv_common.hpp"

namespace sv {

constexpr int kAdjustMost = 128;  // guesses of a sequence
// A table entry: how often the token was written (below 2^30: the entry points refuse longer texts), and
constexpr uint32_t kSeen = 0x80000000u;    // it is in the prompt
constexpr uint32_t kBiased = 0x40000000u;  // it has a bias

// Whether tokens may have biases, and the width of the table that holds each token's last entry.
enum { BIAS_NONE = 0, BIAS_16 = 1, BIAS_32 = 2 };
template <int BIAS>
struct BiasTable {
    typedef uint16_t type;
};
template <>
struct BiasTable<BIAS_32> {
    typedef uint32_t type;
};

// table[slot] = max(table[slot], n): the half of a word by comparing and swapping the word.
__device__ __forceinline__ void table_max(uint32_t* table, uint32_t slot, uint32_t n) { atomicMax(table + slot, n); }
__device__ __forceinline__ void table_max(uint16_t* table, uint32_t slot, uint32_t n)
{
    uint32_t* word = (uint32_t*)table + slot / 2;
    const uint32_t sh = slot % 2 * 16;
    uint32_t old = *word;
    while ((old >> sh & 0xffffu) < n) {  // (a swap that fails has met another's that went in: at most one per entry)
        const uint32_t was = atomicCAS(word, old, (old & ~(0xffffu << sh)) | n << sh);
        if (was == old) break;
        old = was;
    }
}

struct AdjustArgs {
    const char* in;
    char* out;
    int64_t in_stride, out_stride;  // bytes
    const int32_t *cu, *ids, *parents;
    int32_t batch, kmax, total_draft, vocab;
    int32_t nchunk, runs, run_rows;  // workgroups over the vocabulary and over a sequence's rows; rows of one
    const int32_t *tokens, *lengths, *prompt;
    int64_t token_stride;
    int32_t max_tokens;
    const float *repetition, *presence, *frequency;
    const int32_t *bias_ids, *cu_bias;
    const float* bias_values;
    int32_t total_bias;
    const uint8_t* masks;  // bit v % 8 of byte v / 8: token v is allowed
    int64_t mask_stride;   // bytes
    int32_t num_masks;
    const int32_t* mask_rows;
    bool past;  // whole vectors are stored past the caches
};

// 16 bytes of a row, aligned to its elements only.
template <int DT>
struct RowVec;
template <>
struct RowVec<DT_F32> {
    typedef u32x4 type __attribute__((aligned(4)));
};
template <>
struct RowVec<DT_BF16> {
    typedef u32x4 type __attribute__((aligned(2)));
};
template <>
struct RowVec<DT_F16> {
    typedef u32x4 type __attribute__((aligned(2)));
};

template <int DT>
__device__ __forceinline__ uint32_t narrow(float x)  // rounded to nearest, the type's bits
{
    if constexpr (DT == DT_F32) return __float_as_uint(x);
    else if constexpr (DT == DT_BF16) return __builtin_bit_cast(uint16_t, (__bf16)x);
    else return __builtin_bit_cast(uint16_t, (_Float16)x);
}

struct Penalty {
    float rep, pres, freq;
};

// One token's penalties.  entry: its count (kSeen: in the prompt too).
__device__ __forceinline__ float edited(float x, uint32_t entry, const Penalty& p)
{
#pragma clang fp contract(off)
    if (entry != 0) x = x > 0.0f ? x / p.rep : x * p.rep;
    const uint32_t n = entry & ~kSeen;
    if (n != 0) {
        x = x - p.freq * (float)n;
        x = x - p.pres;
    }
    return x;
}

template <int DT, bool INPLACE, int BIAS, int CT, int NT>
__global__ __launch_bounds__(NT) void adjust_kernel(AdjustArgs a)
{
    typedef typename RowVec<DT>::type Vec;
    constexpr int VEC = Dt<DT>::kVec, ES = Dt<DT>::kSize;
    constexpr int NV = CT / VEC / NT;  // vectors per thread and row
    constexpr uint32_t FULL = (1u << VEC) - 1;
    constexpr uint32_t kGuess = 0x8000u;  // in the list: the token is a guess
    static_assert(NV >= 1 && CT % NT == 0 && CT <= (int)kGuess, "tokens per workgroup");
    __shared__ __align__(16) uint32_t s_count[CT];
    __shared__ __align__(16) typename BiasTable<BIAS>::type s_bias[BIAS != BIAS_NONE ? CT : 8];  // 1 + the last entry
    __shared__ uint16_t s_list[CT];        // tokens with any edit
    __shared__ uint32_t s_guess[CT / 32];  // tokens that are guesses
    __shared__ int32_t s_mask[kAdjustMost + 1];  // the rows' masks, -1: none
    __shared__ int32_t s_id[kAdjustMost], s_up[kAdjustMost], s_listed;
    __shared__ uint32_t s_path[kAdjustMost + 1][4];
    const int tid = (int)threadIdx.x;
    const int32_t chunk = (int32_t)(blockIdx.x % (uint32_t)a.nchunk);
    uint32_t rest = blockIdx.x / (uint32_t)a.nchunk;
    const int32_t run = (int32_t)(rest % (uint32_t)a.runs), b = (int32_t)(rest / (uint32_t)a.runs);
    int32_t k0 = b * a.kmax, kb = a.kmax;
    if (a.cu != nullptr) {
        k0 = a.cu[b];
        const int32_t k1 = a.cu[b + 1];
        kb = k1 - k0;
        if (k0 < 0 || kb < 0 || kb > a.kmax || k1 > a.total_draft) return;
    }
    const int32_t r0 = run * a.run_rows, r1 = min(r0 + a.run_rows, kb + 1);
    if (r0 >= r1) return;
    const int32_t lo = chunk * CT, width = min(a.vocab - lo, CT);

    const Penalty p{a.repetition != nullptr ? a.repetition[b] : 1.0f, a.presence != nullptr ? a.presence[b] : 0.0f,
                    a.frequency != nullptr ? a.frequency[b] : 0.0f};
    const bool pen = p.rep != 1.0f || p.pres != 0.0f || p.freq != 0.0f;
    const bool guesses = pen && a.ids != nullptr && kb > 0;
    int32_t b0 = 0, b1 = BIAS != BIAS_NONE ? a.total_bias : 0;
    if (BIAS != BIAS_NONE && a.cu_bias != nullptr) {
        b0 = max(a.cu_bias[b], 0);
        b1 = min(a.cu_bias[b + 1], a.total_bias);
    }
    const bool edits = pen || b0 < b1;  // (uniform) any token may be met
    const auto mask_of = [&](int32_t at) -> const SV_GLOBAL uint8_t* {  // of the run's row `at`
        return (const SV_GLOBAL uint8_t*)(a.masks + s_mask[at] * a.mask_stride + lo / 8);
    };
    if (a.masks != nullptr && tid < r1 - r0) {
        const int64_t row = (int64_t)k0 + b + r0 + tid;
        const int32_t m = a.mask_rows != nullptr ? a.mask_rows[row] : (int32_t)row;
        s_mask[tid] = m >= 0 && m < a.num_masks ? m : -1;
    }

    if (edits) {
        for (int i = tid; i < CT / 32; i += NT) s_guess[i] = 0;
#pragma unroll
        for (int i = tid; i < CT / 4; i += NT) ((u32x4*)s_count)[i] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (BIAS != BIAS_NONE) {
#pragma unroll
            for (int i = tid; i < (int)(sizeof(s_bias) / 16); i += NT) ((u32x4*)s_bias)[i] = u32x4{0u, 0u, 0u, 0u};
        }
        if (tid == 0) s_listed = 0;
        if (guesses && tid < kb) {
            s_id[tid] = a.ids[k0 + tid];
            s_up[tid] = a.parents != nullptr ? a.parents[k0 + tid] : tid;
        }
        __syncthreads();
        if (pen && a.tokens != nullptr) {
            const int32_t len = a.lengths != nullptr ? min(max(a.lengths[b], 0), a.max_tokens) : a.max_tokens;
            const int32_t prompt = a.prompt != nullptr ? a.prompt[b] : 0;
            const int32_t* row = a.tokens + (int64_t)b * a.token_stride;
            typedef u32x4 Four __attribute__((aligned(4)));
            // tokens [from, to) of the text, `hit` for those of this workgroup
            auto scan = [&](int32_t from, int32_t to, auto hit) {
                auto meet = [&](uint32_t token) {
                    const uint32_t slot = token - (uint32_t)lo;
                    if (slot < (uint32_t)width) hit(slot);
                };
                constexpr int kAhead = 4096 / NT / 4 > 4 ? 4 : 4096 / NT / 4 > 0 ? 4096 / NT / 4 : 1;  // 16-byte loads
                constexpr int kStep = kAhead * NT * 4;
                int32_t i0 = from;
                for (; i0 + kStep <= to; i0 += kStep) {
                    u32x4 t[kAhead];
#pragma unroll
                    for (int x = 0; x < kAhead; ++x) t[x] = *(const SV_GLOBAL Four*)(row + i0 + (x * NT + tid) * 4);
#pragma unroll
                    for (int x = 0; x < kAhead; ++x)
#pragma unroll
                        for (int j = 0; j < 4; ++j) meet(t[x][j]);
                }
                uint32_t t[kAhead * 4];  // the rest, one by one
#pragma unroll
                for (int x = 0; x < kAhead * 4; ++x) {
                    t[x] = UINT32_MAX;
                    if (i0 + x * NT >= to) continue;
                    const int32_t i = i0 + x * NT + tid;
                    if (i < to) t[x] = (uint32_t)((const SV_GLOBAL int32_t*)row)[i];
                }
#pragma unroll
                for (int x = 0; x < kAhead * 4; ++x)
                    if (i0 + x * NT < to) meet(t[x]);
            };
            const int32_t cut = min(max(prompt, 0), len);
            scan(0, cut, [&](uint32_t slot) { atomicOr(&s_count[slot], kSeen); });
            scan(cut, len, [&](uint32_t slot) { atomicAdd(&s_count[slot], 1u); });
        }
        if constexpr (BIAS != BIAS_NONE) {
            for (int32_t i = b0 + tid; i < b1; i += NT) {
                const uint32_t slot = (uint32_t)a.bias_ids[i] - (uint32_t)lo;
                if (slot >= (uint32_t)width) continue;
                atomicOr(&s_count[slot], kBiased);
                table_max(s_bias, slot, (uint32_t)(i - b0) + 1u);
            }
        }
        if (guesses && tid < kb) {
            const uint32_t slot = (uint32_t)s_id[tid] - (uint32_t)lo;
            if (slot < (uint32_t)width) atomicOr(&s_guess[slot / 32], 1u << (slot % 32));
        }
        if (guesses && tid < r1 - r0) {  // the guesses on the way up from row r0 + tid
            uint32_t set[4] = {0u, 0u, 0u, 0u};
            for (int32_t r = r0 + tid; r > 0;) {
                const int32_t g = r - 1, up = s_up[g];
#pragma unroll
                for (int w = 0; w < 4; ++w) set[w] |= g / 32 == w ? 1u << (g % 32) : 0u;
                r = up >= 0 && up < r ? up : 0;
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) s_path[tid][w] = set[w];
        }
        __syncthreads();
        // the list, in any order: each thread looks at runs of four tokens, a wave's places come from one addition
        constexpr int RUNS = CT / 4 / NT;
        uint32_t found[RUNS];  // bits 0..3: met, 4..7: of these, guesses
        int32_t mine = 0;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
            const int slot = (i * NT + tid) * 4;
            const u32x4 c = *(const u32x4*)(s_count + slot);
            const uint32_t g = s_guess[slot / 32] >> (slot % 32) & 15u;
            found[i] = g | (c.x != 0 ? 1u : 0u) | (c.y != 0 ? 2u : 0u) | (c.z != 0 ? 4u : 0u) | (c.w != 0 ? 8u : 0u) | g << 4;
            mine += __builtin_popcount(found[i] & 15u);
        }
        const int32_t incl = wave_incl_scan_int(mine);
        int32_t base = 0;
        if (lane_id() == kWave - 1 && incl != 0) base = atomicAdd(&s_listed, incl);
        base = __builtin_amdgcn_readlane(base, kWave - 1) + incl - mine;
        if (mine != 0) {
#pragma unroll
            for (int i = 0; i < RUNS; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if ((found[i] >> x & 1u) != 0)
                        s_list[base++] = (uint16_t)((uint32_t)((i * NT + tid) * 4 + x) |
                                                    ((found[i] >> (4 + x) & 1u) != 0 ? kGuess : 0u));
        }
    }
    __syncthreads();  // (the list, and the masks' numbers)

    const auto vectors = [&](auto past) {
        for (int32_t r = r0; r < r1; ++r) {
            const bool masked = a.masks != nullptr && s_mask[r - r0] >= 0;
            if (INPLACE && !masked) continue;
            const int64_t at = (int64_t)k0 + b + r;
            const char* in = a.in + at * a.in_stride + (int64_t)lo * ES;
            char* out = a.out + at * a.out_stride + (int64_t)lo * ES;
            uint32_t allowed[NV];
            u32x4 raw[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int32_t e = (i * NT + tid) * VEC;
                allowed[i] = masked && e < width ? mask_of(r - r0)[e / 8] : 255u;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int32_t e = (i * NT + tid) * VEC;
                allowed[i] = allowed[i] >> (VEC == 8 ? 0 : e % 8) & FULL;
                raw[i] = u32x4{0u, 0u, 0u, 0u};
                if (e + VEC <= width && allowed[i] != 0 && (!INPLACE || allowed[i] != FULL))
                    raw[i] = *(const SV_GLOBAL Vec*)(in + (int64_t)e * ES);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int32_t e = (i * NT + tid) * VEC;
                const uint32_t may = allowed[i];
                if (e >= width || (INPLACE && may == FULL)) continue;
                if (e + VEC <= width) {
                    u32x4 v = raw[i];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if constexpr (ES == 4) {
                            if ((may >> q & 1u) == 0) v[q] = 0xff800000u;
                        } else {
                            const uint32_t drop = (may >> (2 * q) & 1u ? 0u : 0xffffu) |
                                                  (may >> (2 * q + 1) & 1u ? 0u : 0xffff0000u);
                            v[q] = (v[q] & ~drop) | (Dt<DT>::kNegInf * 0x10001u & drop);
                        }
                    }
                    SV_GLOBAL Vec* to = (SV_GLOBAL Vec*)(out + (int64_t)e * ES);
                    if constexpr (decltype(past)::value) __builtin_nontemporal_store((Vec)v, to);
                    else *to = v;
                } else {  // the vocabulary ends in this vector
#pragma unroll 1
                    for (int x = 0; e + x < width; ++x) {
                        if constexpr (ES == 4)
                            ((SV_GLOBAL uint32_t*)out)[e + x] =
                                may >> x & 1u ? ((const SV_GLOBAL uint32_t*)in)[e + x] : 0xff800000u;
                        else
                            ((SV_GLOBAL uint16_t*)out)[e + x] =
                                may >> x & 1u ? ((const SV_GLOBAL uint16_t*)in)[e + x] : (uint16_t)Dt<DT>::kNegInf;
                    }
                }
            }
        }
    };
    if (!INPLACE || a.masks != nullptr) {
        if (a.past) vectors(std::true_type{});
        else vectors(std::false_type{});
    }
    if (!edits) return;
    if (!INPLACE || a.masks != nullptr) __syncthreads();  // (the first pass's stores, which share vectors with the second's)
    const int32_t n = s_listed, all = n * (r1 - r0);
    constexpr int kItems = 4;  // elements in flight per thread
    for (int32_t it0 = tid; it0 < all; it0 += kItems * NT) {
        float x[kItems];
        uint32_t token[kItems], may[kItems];  // UINT32_MAX: none, or masked; the mask's byte
        int32_t at[kItems];                   // the row's place in the run
        bool guess[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int32_t it = it0 + j * NT;
            token[j] = UINT32_MAX;
            x[j] = 0.0f;
            if (it >= all) continue;
            at[j] = it / n;
            const uint32_t listed = s_list[it - at[j] * n];
            token[j] = listed & (kGuess - 1);
            guess[j] = (listed & kGuess) != 0;
            may[j] = 0xffu;
            if (a.masks != nullptr && s_mask[at[j]] >= 0) may[j] = mask_of(at[j])[token[j] / 8];
        }
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            if (token[j] == UINT32_MAX) continue;
            if ((may[j] >> (token[j] % 8) & 1u) == 0) token[j] = UINT32_MAX;
            else x[j] = load_one<DT>(a.in + ((int64_t)k0 + b + r0 + at[j]) * a.in_stride, lo + (int64_t)token[j]);
        }
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            if (token[j] == UINT32_MAX) continue;
            uint32_t entry = s_count[token[j]];
            const bool biased = BIAS != BIAS_NONE && (entry & kBiased) != 0;
            entry &= ~kBiased;
            if (guess[j]) {
                for (int32_t g = 0; g < kb; ++g)
                    entry += s_id[g] == lo + (int32_t)token[j] ? s_path[at[j]][g / 32] >> (g % 32) & 1u : 0u;
            }
            if (entry == 0 && !biased) continue;  // (a guess on another row's path)
            float f = edited(x[j], entry, p);
            if constexpr (BIAS != BIAS_NONE) {
                if (biased) f += a.bias_values[b0 + (int32_t)s_bias[token[j]] - 1];
            }
            char* out = a.out + ((int64_t)k0 + b + r0 + at[j]) * a.out_stride + ((int64_t)lo + token[j]) * ES;
            if constexpr (ES == 4) *(SV_GLOBAL uint32_t*)out = narrow<DT>(f);
            else *(SV_GLOBAL uint16_t*)out = (uint16_t)narrow<DT>(f);
        }
    }
}

}  // namespace sv
