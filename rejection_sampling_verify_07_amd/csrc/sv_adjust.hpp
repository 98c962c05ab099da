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
// (integer atomics: any order gives the same counts) and marks the tokens met in
// a bitmap, then walks the rows in vectors of 16 bytes: the bitmap and the mask
// say which vectors change, and only those are touched in place; a vector whose
// tokens are all masked is written without being read.  The guesses on a row's own path enter
// the table before the row and leave it after.  The history is read once per run
// of rows and CT tokens, from the caches; nothing needs a workspace.
//
// Arithmetic is fp32, each step rounded, the result rounded to the element type once.
#pragma once

#include "sv_common.hpp"

namespace sv {

constexpr int kAdjustMost = 128;  // guesses of a sequence
constexpr uint32_t kSeen = 0x80000000u;

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

// One token's edits but for the mask.  entry: its count (kSeen: in the prompt too); bias: its value or 0.
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

template <int DT, bool INPLACE, bool BIAS, int CT>
__global__ __launch_bounds__(kThreads) void adjust_kernel(AdjustArgs a)
{
    typedef typename RowVec<DT>::type Vec;
    constexpr int VEC = Dt<DT>::kVec, ES = Dt<DT>::kSize;
    constexpr int NV = CT / VEC / kThreads;  // vectors per thread and row
    constexpr uint32_t FULL = (1u << VEC) - 1;
    static_assert(NV >= 1 && CT % 32 == 0, "tokens per workgroup");
    __shared__ __align__(16) uint32_t s_count[CT];
    __shared__ __align__(16) uint32_t s_bias[BIAS ? CT : 4];  // 1 + the last entry of the token, 0: none
    __shared__ __align__(16) uint32_t s_met[CT / 32];
    __shared__ int32_t s_id[kAdjustMost], s_up[kAdjustMost];
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
    int32_t b0 = 0, b1 = BIAS ? a.total_bias : 0;
    if (BIAS && a.cu_bias != nullptr) {
        b0 = max(a.cu_bias[b], 0);
        b1 = min(a.cu_bias[b + 1], a.total_bias);
    }
    const bool edits = pen || b0 < b1;  // (uniform) any token may be met
    if (edits) {
        for (int i = tid; i < CT / 32; i += kThreads) s_met[i] = 0;
        for (int i = tid; i < CT / 4; i += kThreads) ((u32x4*)s_count)[i] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (BIAS)
            for (int i = tid; i < CT / 4; i += kThreads) ((u32x4*)s_bias)[i] = u32x4{0u, 0u, 0u, 0u};
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
            auto meet = [&](uint32_t token, int32_t at) {
                const uint32_t slot = token - (uint32_t)lo;
                if (slot >= (uint32_t)width) return;
                if (at < prompt) atomicOr(&s_count[slot], kSeen);
                else atomicAdd(&s_count[slot], 1u);
                atomicOr(&s_met[slot / 32], 1u << (slot % 32));
            };
            int32_t i = tid * 4;
#pragma unroll 2
            for (; i + 4 <= len; i += kThreads * 4) {
                const u32x4 t = *(const SV_GLOBAL Four*)(row + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) meet(t[j], i + j);
            }
            for (; i < len; ++i) meet((uint32_t)row[i], i);  // (one thread: the last 1 to 3)
        }
        if constexpr (BIAS) {
            for (int32_t i = b0 + tid; i < b1; i += kThreads) {
                const uint32_t slot = (uint32_t)a.bias_ids[i] - (uint32_t)lo;
                if (slot >= (uint32_t)width) continue;
                atomicMax(&s_bias[slot], (uint32_t)(i - b0) + 1u);
                atomicOr(&s_met[slot / 32], 1u << (slot % 32));
            }
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
    }

    for (int32_t r = r0; r < r1; ++r) {
        const int64_t row = (int64_t)k0 + b + r;
        uint32_t own = UINT32_MAX;  // the slot of this thread's guess, where it is on the row's path
        if (guesses) {
            if (tid < kb && (s_path[r - r0][tid / 32] >> (tid % 32) & 1u) != 0) {
                own = (uint32_t)s_id[tid] - (uint32_t)lo;
                if (own < (uint32_t)width) {
                    atomicAdd(&s_count[own], 1u);
                    atomicOr(&s_met[own / 32], 1u << (own % 32));
                }
            }
            __syncthreads();
        }
        const uint8_t* mask = nullptr;
        if (a.masks != nullptr) {
            const int64_t m = a.mask_rows != nullptr ? a.mask_rows[row] : row;
            if (m >= 0 && m < a.num_masks) mask = a.masks + m * a.mask_stride;
        }
        const char* in = a.in + row * a.in_stride + (int64_t)lo * ES;
        char* out = a.out + row * a.out_stride + (int64_t)lo * ES;
        u32x4 raw[NV];
        uint32_t allowed[NV], met[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int32_t e = (i * kThreads + tid) * VEC;
            allowed[i] = FULL;
            if (mask != nullptr && e < width) allowed[i] = (uint32_t)mask[(lo + e) / 8] >> (e % 8) & FULL;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int32_t e = (i * kThreads + tid) * VEC;
            met[i] = 0;
            if (edits) met[i] = s_met[e / 32] >> (e % 32) & allowed[i];
            raw[i] = u32x4{0u, 0u, 0u, 0u};
            const bool read = allowed[i] != 0 && (!INPLACE || met[i] != 0 || allowed[i] != FULL);
            if (read && e + VEC <= width) {
                raw[i] = *(const SV_GLOBAL Vec*)(in + (int64_t)e * ES);
            } else if (read && e < width) {  // the vocabulary ends in this vector
                for (int x = 0; x < width - e; ++x) {
                    const uint32_t v = ES == 4 ? ((const SV_GLOBAL uint32_t*)in)[e + x]
                                               : (uint32_t)((const SV_GLOBAL uint16_t*)in)[e + x] << (x % 2 * 16);
                    const int q = ES == 4 ? x : x / 2;
#pragma unroll
                    for (int w = 0; w < 4; ++w) raw[i][w] |= w == q ? v : 0u;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int32_t e = (i * kThreads + tid) * VEC;
            if (e >= width || (INPLACE && allowed[i] == FULL && met[i] == 0)) continue;
            if (met[i] != 0) {
#pragma unroll
                for (int x = 0; x < VEC; ++x) {
                    if ((met[i] >> x & 1u) == 0) continue;
                    const int q = ES == 4 ? x : x / 2, sh = ES == 4 ? 0 : x % 2 * 16;
                    const uint32_t bits = ES == 4 ? raw[i][q] : raw[i][q] >> sh & 0xffffu;
                    float v;
                    if constexpr (DT == DT_F32) v = __uint_as_float(bits);
                    else v = lo16<DT>(bits);
                    v = edited(v, s_count[e + x], p);
                    if constexpr (BIAS) {
                        const uint32_t n = s_bias[e + x];
                        if (n != 0) v += a.bias_values[b0 + (int32_t)n - 1];
                    }
                    const uint32_t keep = ES == 4 ? 0u : 0xffffu << (16 - sh);
                    raw[i][q] = (raw[i][q] & keep) | narrow<DT>(v) << sh;
                }
            }
            if (allowed[i] != FULL) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (ES == 4) {
                        if ((allowed[i] >> q & 1u) == 0) raw[i][q] = 0xff800000u;
                    } else {
                        const uint32_t drop = (allowed[i] >> (2 * q) & 1u ? 0u : 0xffffu) |
                                              (allowed[i] >> (2 * q + 1) & 1u ? 0u : 0xffff0000u);
                        raw[i][q] = (raw[i][q] & ~drop) | (Dt<DT>::kNegInf * 0x10001u & drop);
                    }
                }
            }
            if (e + VEC <= width) {
                *(SV_GLOBAL Vec*)(out + (int64_t)e * ES) = raw[i];
            } else {
                for (int x = 0; x < width - e; ++x) {
                    const int q = ES == 4 ? x : x / 2;
                    uint32_t v = 0;
#pragma unroll
                    for (int w = 0; w < 4; ++w) v |= w == q ? raw[i][w] : 0u;
                    if constexpr (ES == 4) ((SV_GLOBAL uint32_t*)out)[e + x] = v;
                    else ((SV_GLOBAL uint16_t*)out)[e + x] = (uint16_t)(v >> (x % 2 * 16));
                }
            }
        }
        if (guesses) {
            __syncthreads();
            if (own < (uint32_t)width) atomicSub(&s_count[own], 1u);
        }
    }
}

}  // namespace sv
