// Host-side helpers shared by the entry points: alignment, element types,
// workspace offsets and kernel launches.
#pragma once

#include "specverify.h"
#include "specverify_profile.h"

#include <hip/hip_ext.h>

#include <stdint.h>
#include <string.h>

#include <array>
#include <type_traits>

#include "sv_common.hpp"

namespace {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int vec_of(sv_dtype_t dt) { return dt == SV_DTYPE_F32 ? 4 : 8; }
inline size_t esize_of(sv_dtype_t dt) { return dt == SV_DTYPE_F32 ? 4 : 2; }

// The caller's dtype field as an integer (any int may be stored there by a C caller).
template <class Shape>
int32_t dtype_of(const Shape* sh)
{
    static_assert(sizeof(sh->dtype) == sizeof(int32_t), "sv_dtype_t is an int-sized enum");
    int32_t v;
    memcpy(&v, &sh->dtype, sizeof v);
    return v;
}

// A launch counts its threads in 32 bits.
inline bool launchable(double workgroups, int threads) { return workgroups * threads <= (double)UINT32_MAX; }

// Whether the places of N dimensions of `size` with these strides, `width` bytes each, are all distinct: every stride
// clears the extent of the dimensions inside it.  *bytes: the extent of all of them.
template <int N>
bool distinct_places(const std::array<int64_t, N>& size, const std::array<int64_t, N>& stride, int64_t width,
                     int64_t* bytes)
{
    int64_t& extent = *bytes;
    extent = width;
    bool done[N] = {};
    for (int k = 0; k < N; ++k) {
        int at = -1;  // the smallest stride left, of the dimensions that have more than one place
        for (int i = 0; i < N; ++i)
            if (!done[i] && size[i] > 1 && (at < 0 || stride[i] < stride[at])) at = i;
        if (at < 0) return true;
        done[at] = true;
        if (stride[at] < extent || stride[at] > (INT64_MAX - extent) / (size[at] - 1)) return false;
        extent += stride[at] * (size[at] - 1);
    }
    return true;
}

// Calls fn with std::integral_constant<int, DT> for the element type
// (the shape check has already rejected any other value).
template <class F>
sv_status_t by_dtype(sv_dtype_t dt, F&& fn)
{
    switch (dt) {
        case SV_DTYPE_F32: return fn(std::integral_constant<int, sv::DT_F32>{});
        case SV_DTYPE_BF16: return fn(std::integral_constant<int, sv::DT_BF16>{});
        case SV_DTYPE_F16: return fn(std::integral_constant<int, sv::DT_F16>{});
    }
    return SV_ERR_INVALID_ARGUMENT;
}

// Chunks per row of the streaming passes: a row with start misalignment up
// to VEC-1 elements touches at most ceil((V + VEC - 1) / VEC) blocks.
inline int32_t chunks_for(int32_t vocab, int vec, int loads)
{
    const int64_t nblk = ((int64_t)vocab + 2 * vec - 2) / vec;
    const int64_t per = (int64_t)sv::kThreads * loads;
    return (int32_t)((nblk + per - 1) / per);
}

// Launch a streaming-pass kernel, one tile per workgroup.  With `prof`
// (the benchmark entry points), the launch itself records the caller's
// events right before and after the kernel on the call's stream.
template <class K, class... Args>
void launch_stream_nt(const sv_profile_events_t* prof, K kernel, uint32_t ntiles, uint32_t nt, hipStream_t s,
                      Args... args)
{
    if (prof != nullptr) {
        hipExtLaunchKernelGGL(kernel, dim3(ntiles), dim3(nt), 0, s, prof->start, prof->stop, 0, args...);
    } else {
        hipLaunchKernelGGL(kernel, dim3(ntiles), dim3(nt), 0, s, args...);
    }
}

template <class K, class... Args>
void launch_stream(const sv_profile_events_t* prof, K kernel, uint32_t ntiles, hipStream_t s, Args... args)
{
    launch_stream_nt(prof, kernel, ntiles, sv::kThreads, s, args...);
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

template <class T>
T* ws_at(void* ws, size_t off)
{
    return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

inline sv_status_t launch_status()
{
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? SV_OK : SV_ERR_HIP;
}

// Limits of the attention calls.
constexpr int32_t kMaxPosStride = 1 << 25;  // bytes: 64 positions stay within a 31-bit offset
constexpr int32_t kMaxPositions = 1 << 30;

// A cache's pointer and strides (elements of 2 bytes): 16-byte places.
inline bool cache_ok(const sv_cache_t* c)
{
    if (c == nullptr || c->data == nullptr || !aligned(c->data, 16)) return false;
    return c->batch_stride >= 0 && c->head_stride >= 0 && c->position_stride >= 0 && c->batch_stride % 8 == 0 &&
           c->head_stride % 8 == 0 && c->position_stride % 8 == 0;
}

// Whether `count` places this far apart (elements) stay within what 64 bits count, in bytes of any element type.
inline bool stride_ok(int64_t stride, int64_t count) { return stride <= INT64_MAX / 16 / count; }

// The limits of a cache of 2-byte elements: `outer` groups, sequences or pages of `heads` heads.
inline bool cache_fits(const sv_cache_t* c, int64_t outer, int64_t heads)
{
    return c->position_stride <= kMaxPosStride / 2 && stride_ok(c->batch_stride, outer) &&
           stride_ok(c->head_stride, heads);
}

// Whether rows of `width` elements at two strides lie apart.
inline bool distinct_rows(int64_t s0, int64_t n0, int64_t s1, int64_t n1, int64_t width)
{
    if (n0 < 2) s0 = 0;
    if (n1 < 2) s1 = 0;
    const bool first = n1 < 2 || (n0 > 1 && s0 < s1);  // the inner of the two
    const int64_t si = first ? s0 : s1, ni = first ? n0 : n1, so = first ? s1 : s0, no = first ? n1 : n0;
    if (ni > 1 && si < width) return false;
    return no < 2 || (ni < 2 ? so >= width : so >= width && (so - width) / si >= ni - 1);
}

// c = fl32(log2(e) / T): the softmax's exp(l / T) is computed as exp2(l * c).
inline float scale_of(float temperature) { return (float)(1.4426950408889634 / (double)temperature); }

}  // namespace
