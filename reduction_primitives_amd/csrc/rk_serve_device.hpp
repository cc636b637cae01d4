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
    template <bool STREAM = false>
    __device__ __forceinline__ static T load(const void *p)
    {
        if constexpr (STREAM)                              // what is read once
            return __builtin_nontemporal_load(static_cast<const Any *>(p));
        else
            return *static_cast<const Any *>(p);
    }
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

struct Plus {
    template <class T> __device__ __forceinline__ static T apply(T a, T b) { return a + b; }
};

// Inclusive scan over the 64 lanes (all active) by DPP moves: shifts within
// rows of 16, then the last lane of a row to the next row, of the lower half
// to the upper.  Lanes without a source get 0, which Op must take as neutral.
template <int CTRL, int ROWS, class T>
__device__ __forceinline__ T dpp_or_0(T v)
{
    return move_words(v, [](uint32_t w) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w, CTRL, ROWS, 0xf, false);
    });
}

template <class Op = Plus, class T>
__device__ __forceinline__ T wave_prefix(T v)
{
    v = Op::apply(v, dpp_or_0<0x111, 0xf>(v));    // row_shr:1
    v = Op::apply(v, dpp_or_0<0x112, 0xf>(v));
    v = Op::apply(v, dpp_or_0<0x114, 0xf>(v));
    v = Op::apply(v, dpp_or_0<0x118, 0xf>(v));
    v = Op::apply(v, dpp_or_0<0x142, 0xa>(v));    // row_bcast:15 into rows 1 and 3
    v = Op::apply(v, dpp_or_0<0x143, 0xc>(v));    // row_bcast:31 into rows 2 and 3
    return v;
}

// Exclusive scan over a block of whole waves; `total` is the block's sum.
// `part` is LDS of BLOCK / 64 values; callers separate two uses by a barrier.
template <int BLOCK, class Op = Plus, class T>
__device__ __forceinline__ T block_prefix(T v, T *part, T *total)
{
    constexpr int NW = BLOCK / 64;
    const T incl = wave_prefix<Op>(v);
    const int w = int(threadIdx.x >> 6);
    if (lane_id() == 63)
        part[w] = incl;
    const T excl = dpp_or_0<0x138, 0xf>(incl);    // wave_shr:1
    __syncthreads();
    T before = T(0), sum = T(0);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const T s = part[i];
        if (i < w)
            before = Op::apply(before, s);
        sum = Op::apply(sum, s);
    }
    *total = sum;
    return Op::apply(before, excl);
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
