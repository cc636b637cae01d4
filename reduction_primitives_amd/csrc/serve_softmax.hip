// serve_softmax.hip -- softmax of contiguous lines with a temperature each.
//
//   p_i = exp((x_i - m) / t) / s,   m = max_j x_j,   s = sum_j exp((x_j - m) / t)
//
// A line is cut into chunks, a block each.  The first launch leaves every
// chunk's largest entry m_c and s_c = sum exp((x_j - m_c) / t); the second
// folds them, s = sum_c s_c exp((m_c - m) / t), and writes the line.  Sums and
// statistics are float32; the one rounding to the output's type is the
// store's.  An entry of -inf counts as masked (0 whatever the temperature is);
// a line of nothing else gives zeros.  NaN, or +inf at t > 0, makes the line
// NaN.  t <= 0 puts 1 on the first largest entry.
#define RK_UNIT unit_serve_softmax
#include "rk_serve_device.hpp"

namespace rk {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kMaxFloat = 3.40282346638528859812e38f;

// 1 / t as a factor of base-2 exponents, kept finite: 0 * factor stays 0.
__device__ __forceinline__ float scale_of(float t)
{
    const float c = kLog2e / t;
    return c > kMaxFloat ? kMaxFloat : c;
}

// exp((x - m) / t), 0 for a masked entry.  v_exp_f32 is good to 1 ulp and the
// argument is rounded twice, an error of |argument| 2^-23 in the result.
__device__ __forceinline__ float soft_term(float x, float m, float c)
{
    const float e = __builtin_amdgcn_exp2f((x - m) * c);
    return x == -std::numeric_limits<float>::infinity() ? 0.0f : e;
}

template <class Out> struct OutTraits;
template <> struct OutTraits<float> {
    using S = float;
    __device__ static S one(float v) { return v; }
};
template <> struct OutTraits<bf16_in> {
    using S = uint16_t;
    __device__ static S one(float v) { return f32_to_bf16_rne(v); }
};
template <> struct OutTraits<f16_in> {
    using S = uint16_t;
    __device__ static S one(float v) { return bitcast<uint16_t>((_Float16)v); }
};

// V results (V = elements of a 16-byte input vector) to consecutive places.
template <class Out, int V>
__device__ __forceinline__ void store_vec(typename OutTraits<Out>::S *p, const float *v)
{
    using S = typename OutTraits<Out>::S;
    constexpr int per = 16 / sizeof(S);
    if constexpr (V < per) {                  // f32 in, 16-bit out: 8 bytes
        typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = uint32_t(OutTraits<Out>::one(v[2 * i])) | uint32_t(OutTraits<Out>::one(v[2 * i + 1])) << 16;
        u32x2_any o;
        o[0] = w[0];
        o[1] = w[1];
        *reinterpret_cast<u32x2_any *>(p) = o;
    } else {
#pragma unroll
        for (int k = 0; k < V; k += per) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(S) == 4)
                    o[i] = bitcast<uint32_t>(OutTraits<Out>::one(v[k + i]));
                else
                    o[i] = uint32_t(OutTraits<Out>::one(v[k + 2 * i])) |
                           uint32_t(OutTraits<Out>::one(v[k + 2 * i + 1])) << 16;
            }
            store16(p + k, o);
        }
    }
}

// Whole-block reduction whose result every thread gets.
template <class Op, int BLOCK, class T>
__device__ __forceinline__ T block_all(T v, T *part)
{
    constexpr int NW = BLOCK / 64;
    v = wave_reduce<Op>(v);
    if constexpr (NW > 1) {
        __syncthreads();
        if (lane_id() == 0)
            part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int i = 1; i < NW; ++i)
            v = Op::apply(v, part[i]);
    }
    return v;
}

constexpr int kNone = 0x7fffffff;

// First launch: the statistics of one chunk.
template <class In>
__global__ __launch_bounds__(tune::kSoftBlock) void k_soft_stats(SoftmaxArgs a)
{
    using S = typename InTraits<In>::S;
    constexpr int V = InTraits<In>::vec, B = tune::kSoftBlock;
    constexpr int U = tune::kSoftChunk / (B * V);
    __shared__ float part[B / 64];
    __shared__ int parti[B / 64];
    const int64_t line = blockIdx.x / uint32_t(a.chunks);
    const int c = int(blockIdx.x % uint32_t(a.chunks));
    const S *x = static_cast<const S *>(a.x) + line * a.xs + int64_t(c) * a.chunk;
    const int n = int(a.n - int64_t(c) * a.chunk < a.chunk ? a.n - int64_t(c) * a.chunk : a.chunk);
    const float t = a.t ? a.t[line] : 1.0f;
    float v[U * V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = (u * B + int(threadIdx.x)) * V;
        if (i + V <= n) {
            InTraits<In>::decode(load16(x + i), v + u * V);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[u * V + k] = i + k < n ? InTraits<In>::template one<float>(x[i + k])
                                         : -std::numeric_limits<float>::infinity();
        }
    }
    float m = OpMax::identity<float>();
#pragma unroll
    for (int k = 0; k < U * V; ++k)
        m = OpMax::apply(m, v[k]);
    m = block_all<OpMax, B>(m, part);
    float s = 0.0f;
    int first = kNone;
    if (t <= 0.0f) {
#pragma unroll
        for (int u = U - 1; u >= 0; --u)
#pragma unroll
            for (int k = V - 1; k >= 0; --k)
                if (v[u * V + k] == m)
                    first = (u * B + int(threadIdx.x)) * V + k;
        first = block_all<OpMin, B>(first, parti);
    } else {
        const float f = scale_of(t);
#pragma unroll
        for (int k = 0; k < U * V; ++k)
            s += soft_term(v[k], m, f);
        s = block_all<OpSum, B>(s, part);
    }
    if (threadIdx.x == 0) {
        a.stats[2 * int64_t(blockIdx.x)] = m;
        a.stats[2 * int64_t(blockIdx.x) + 1] = s;
        a.first[blockIdx.x] = first;
    }
}

// Second launch: fold the line's statistics and write one chunk of it.
template <class In, class Out>
__global__ __launch_bounds__(tune::kSoftBlock) void k_soft_write(SoftmaxArgs a)
{
    using S = typename InTraits<In>::S;
    using O = typename OutTraits<Out>::S;
    constexpr int V = InTraits<In>::vec, B = tune::kSoftBlock;
    constexpr int U = tune::kSoftChunk / (B * V);
    const int64_t line = blockIdx.x / uint32_t(a.chunks);
    const int c = int(blockIdx.x % uint32_t(a.chunks));
    const int64_t base = int64_t(c) * a.chunk;
    const S *x = static_cast<const S *>(a.x) + line * a.xs + base;
    O *out = static_cast<O *>(a.out) + line * a.os + base;
    const int n = int(a.n - base < a.chunk ? a.n - base : a.chunk);
    const float t = a.t ? a.t[line] : 1.0f;
    const float f = scale_of(t);
    const float *st = a.stats + 2 * line * a.chunks;
    float m = OpMax::identity<float>();
    for (int i = lane_id(); i < a.chunks; i += 64)
        m = OpMax::apply(m, st[2 * i]);
    m = wave_reduce<OpMax>(m);
    float s = 0.0f;
    int64_t at = -1;                          // t <= 0: place of the 1
    if (t <= 0.0f) {
        int first = kNone;                    // the first chunk that holds the largest entry
        for (int i = lane_id(); i < a.chunks; i += 64)
            if (st[2 * i] == m && i < first)
                first = i;
        first = wave_reduce<OpMin>(first);
        if (first != kNone && m > -std::numeric_limits<float>::infinity())
            at = int64_t(first) * a.chunk + a.first[line * a.chunks + first] - base;
        s = m == m ? 1.0f : m;
    } else {
        for (int i = lane_id(); i < a.chunks; i += 64)
            s += st[2 * i + 1] * soft_term(st[2 * i], m, f);
        s = wave_reduce<OpSum>(s);
    }
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
    const bool greedy = t <= 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = (u * B + int(threadIdx.x)) * V;
        float v[V];
        if (i + V <= n) {
            InTraits<In>::decode(load16(x + i), v);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[k] = i + k < n ? InTraits<In>::template one<float>(x[i + k]) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < V; ++k)
            v[k] = greedy ? (i + k == at ? inv : 0.0f * inv) : soft_term(v[k], m, f) * inv;
        if (i + V <= n) {
            store_vec<Out, V>(out + i, v);
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (i + k < n)
                    out[i + k] = OutTraits<Out>::one(v[k]);
        }
    }
}

template <class In, class Out>
int run_softmax(const SoftmaxLaunch &L)
{
    const dim3 grid(uint32_t(L.plan.grid)), block(L.plan.block);
    launch_timed(k_soft_stats<In>, grid, block, 0, L.stream, L.ev_begin, L.ev_end, L.a);
    launch_timed(k_soft_write<In, Out>, grid, block, 0, L.stream, nullptr, nullptr, L.a);
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

template <class In>
int run_softmax_in(const SoftmaxLaunch &L)
{
    switch (L.out) {
    case F32: return run_softmax<In, float>(L);
    case BF16: return run_softmax<In, bf16_in>(L);
    case F16: return run_softmax<In, f16_in>(L);
    }
    return ST_UNSUPPORTED;
}

}  // namespace

int launch_softmax(const SoftmaxLaunch &L)
{
    switch (L.in) {
    case F32: return run_softmax_in<float>(L);
    case BF16: return run_softmax_in<bf16_in>(L);
    case F16: return run_softmax_in<f16_in>(L);
    }
    return ST_UNSUPPORTED;
}

}  // namespace rk
