// Host-side helpers shared by the entry points: alignment, element types,
// workspace offsets and kernel launches.
#pragma once

#include "specverify.h"
#include "specverify_profile.h"

#include <hip/hip_ext.h>

#include <stdint.h>

#include <type_traits>

#include "sv_common.hpp"

namespace {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int vec_of(sv_dtype_t dt) { return dt == SV_DTYPE_F32 ? 4 : 8; }
inline size_t esize_of(sv_dtype_t dt) { return dt == SV_DTYPE_F32 ? 4 : 2; }

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

// c = fl32(log2(e) / T): the softmax's exp(l / T) is computed as exp2(l * c).
inline float scale_of(float temperature) { return (float)(1.4426950408889634 / (double)temperature); }

}  // namespace
