// rk_serve_device.hpp -- device helpers of the serving operators.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include "rk_device.hpp"
#include "rk_serve.hpp"

namespace rk {

// WORDS 32-bit words at any element's address, in one load or store: gfx950
// takes global accesses of any alignment.  Lines of an odd length start
// anywhere, so no alignment beyond the element's own is asked of them.
template <int WORDS> struct Words {
    typedef uint32_t T __attribute__((ext_vector_type(WORDS)));
    typedef uint32_t Any __attribute__((ext_vector_type(WORDS), aligned(2)));
    __device__ __forceinline__ static T load(const void *p) { return *static_cast<const Any *>(p); }
    template <bool STREAM>
    __device__ __forceinline__ static void store(void *p, T v)
    {
        if constexpr (STREAM)                              // past the caches
            __builtin_nontemporal_store(v, static_cast<Any *>(p));
        else
            *static_cast<Any *>(p) = v;
    }
};

// A small array's bits as N words.
template <int N, class T, size_t M>
__device__ __forceinline__ typename Words<N>::T words_of(const T (&v)[M])
{
    static_assert(sizeof v == 4 * N, "size mismatch");
    typename Words<N>::T w;
    __builtin_memcpy(&w, v, sizeof v);
    return w;
}

__device__ __forceinline__ u32x4 load16(const void *p) { return Words<4>::load(p); }

__device__ __forceinline__ uint32_t divide(uint32_t x, const Divider &d)
{
    return d.shift ? uint32_t((uint64_t(x) * d.m) >> d.shift) : x;
}

// Inclusive scan over the 64 lanes (all active).
template <class T>
__device__ __forceinline__ T wave_prefix(T v)
{
    const int lane = lane_id();
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const T o = __shfl_up(v, d);
        if (lane >= d)
            v += o;
    }
    return v;
}

// Exclusive scan over a block of whole waves; `total` is the block's sum.
// `part` is LDS of BLOCK / 64 values; callers separate two uses by a barrier.
template <int BLOCK, class T>
__device__ __forceinline__ T block_prefix(T v, T *part, T *total)
{
    constexpr int NW = BLOCK / 64;
    const T incl = wave_prefix(v);
    const int w = int(threadIdx.x >> 6);
    if (lane_id() == 63)
        part[w] = incl;
    __syncthreads();
    T before = T(0), sum = T(0);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const T s = part[i];
        if (i < w)
            before += s;
        sum += s;
    }
    *total = sum;
    return before + (incl - v);
}

template <class... KArgs, class... Args>
void launch_timed(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t lds, void *stream, void *ev_begin,
                  void *ev_end, Args... args)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (ev_begin && ev_end)
        hipExtLaunchKernelGGL(kernel, grid, block, lds, st, static_cast<hipEvent_t>(ev_begin),
                              static_cast<hipEvent_t>(ev_end), 0, args...);
    else
        hipLaunchKernelGGL(kernel, grid, block, lds, st, args...);
}

}  // namespace rk
