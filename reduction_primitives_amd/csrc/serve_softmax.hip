// serve_softmax.hip -- softmax of contiguous lines with a temperature each.
//
//   p_i = exp((x_i - m) / t) / s,   m = max_j x_j,   s = sum_j exp((x_j - m) / t)
//
// Two forms.  A line of up to 32 entries a thread of one block (a quarter of a
// wave for the shortest, 1024 threads for the longest) is read once, kept in registers, and
// written: one launch, each byte moved once.  Of a longer one the first launch
// leaves every tile's largest entry m_c and s_c = sum exp((x_j - m_c) / t), a
// tile a wave, with no barrier between the waves; the second folds them,
// s = sum_c s_c exp((m_c - m) / t), reads the line again and writes it (lines
// of over a million entries are folded by a launch between).
//
// Sums and statistics are float32; the one rounding to the output's type is
// the store's.  An entry of -inf counts as masked (0 whatever the temperature
// is); a line of nothing else gives zeros.  NaN, a NaN temperature, or +inf at
// t > 0, makes the line NaN.  t <= 0 puts 1 on the first largest entry.
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

// exp((x - m) / t).  v_exp_f32 is good to 1 ulp and its argument is rounded
// three times with the factor's own, an error of 3 |argument| 2^-24 in the
// result.  With m finite and a factor above 0 a masked entry gives 0 by
// itself, as -inf's power of two; GUARD sets it to 0 where that fails, and
// halves the two before it subtracts them: x - m passes the largest float
// where m is beyond half its last place, which a large t makes up for.
template <bool GUARD>
__device__ __forceinline__ float soft_term(float x, float m, float c)
{
    if constexpr (GUARD) {
        const float e = __builtin_amdgcn_exp2f((x * 0.5f - m * 0.5f) * c * 2.0f);
        return x == -std::numeric_limits<float>::infinity() ? 0.0f : e;
    } else {
        return __builtin_amdgcn_exp2f((x - m) * c);
    }
}

constexpr float kHalfLastPlace = 0x1p103f;    // of the largest float

__device__ __forceinline__ bool needs_guard(float m, float c)
{
    return !(m > -std::numeric_limits<float>::infinity() && m < kHalfLastPlace && c > 0.0f);
}

// Outputs: rounded to nearest even by gfx950's own conversions.
template <class Out> struct OutTraits;
template <> struct OutTraits<float> {
    using S = float;
    __device__ __forceinline__ static S one(float v) { return v; }
};
template <> struct OutTraits<bf16_in> {
    using S = uint16_t;
    __device__ __forceinline__ static S one(float v) { return bitcast<uint16_t>((__bf16)v); }
};
template <> struct OutTraits<f16_in> {
    using S = uint16_t;
    __device__ __forceinline__ static S one(float v) { return bitcast<uint16_t>((_Float16)v); }
};

// -inf in every entry of a 32-bit word.
template <class In> constexpr uint32_t kMaskedWord = 0xff800000u;
template <> constexpr uint32_t kMaskedWord<bf16_in> = 0xff80ff80u;
template <> constexpr uint32_t kMaskedWord<f16_in> = 0xfc00fc00u;

// Entries of a vector: 16 bytes of the wider of input and output.  Loads then
// take 8 bytes a lane where the output is twice as wide, and every store of a
// wave covers one run of whole lines; with 16-byte loads there, a lane's two
// stores leave gaps (320 x 131072 bf16 to f32: 68.8 us, 64.5 us without gaps,
// and streaming stores, 50.9 us, took 114 us with them).
template <class In, class Out>
constexpr int vec_of()
{
    constexpr int a = InTraits<In>::vec, b = InTraits<Out>::vec;
    return a < b ? a : b;
}

// Reduction over each group of N neighbouring lanes (N a power of two); every
// lane gets its group's result.
template <int N, class Op, class T>
__device__ __forceinline__ T wave_reduce_rows(T v)
{
    if constexpr (N > 1) v = Op::apply(v, lane_xor<1>(v));
    if constexpr (N > 2) v = Op::apply(v, lane_xor<2>(v));
    if constexpr (N > 4) v = Op::apply(v, lane_xor<4>(v));
    if constexpr (N > 8) v = Op::apply(v, lane_xor<8>(v));
    return v;
}

// Reduction over the LANES threads that share a line: a quarter of a wave, a
// wave, or a block whose waves meet in LDS (`part`, one value a wave, a buffer of its own per use).
template <class Op, int LANES, class T>
__device__ __forceinline__ T line_all(T v, T *part)
{
    constexpr int NW = LANES / 64;
    if constexpr (LANES == 16) {              // a DPP row: no lane of another line takes part
        v = Op::apply(v, dpp_move<kDppQuadXor1>(v));
        v = Op::apply(v, dpp_move<kDppQuadXor2>(v));
        v = Op::apply(v, dpp_move<kDppRowHalfMirror>(v));
        v = Op::apply(v, dpp_move<kDppRowMirror>(v));
    } else {
        v = wave_reduce<Op>(v);
    }
    if constexpr (NW > 1) {
        if (lane_id() == 0)
            part[threadIdx.x >> 6] = v;
        __syncthreads();
        v = wave_reduce_rows<NW, Op>(part[lane_id() % NW]);
    }
    return v;
}

constexpr int kNone = 0x7fffffff;

// U vectors of V entries of a piece of n entries, interleaved over LANES
// threads, and one entry more: vector u of thread tid holds entries place(u)
// .. place(u) + V - 1, or -inf where they are not all there; the n % V entries
// behind the last whole vector are the `rest` of the first threads.
// FULL: the piece has every entry it has room for.
template <class In, int V, int LANES, int U, bool FULL>
struct Piece {
    using S = typename InTraits<In>::S;
    static constexpr int kWords = V * int(sizeof(S)) / 4;
    using W = Words<kWords>;
    typename W::T w[U];
    float rest;
    int n, tid;

    __device__ __forceinline__ int place(int u) const { return (u * LANES + tid) * V; }
    __device__ __forceinline__ bool any(int u) const { return FULL || u * LANES * V < n; }     // uniform
    __device__ __forceinline__ bool has(int u) const { return FULL || place(u) + V <= n; }
    __device__ __forceinline__ int rest_place() const { return n - n % V + tid; }
    __device__ __forceinline__ bool has_rest() const { return !FULL && rest_place() < n; }

    __device__ __forceinline__ void load(const S *x, int count, int thread)
    {
        n = count;
        tid = thread;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[u][i] = kMaskedWord<In>;
            if (any(u) && has(u))
                w[u] = W::load(x + place(u));
        }
        rest = -std::numeric_limits<float>::infinity();
        if (has_rest())
            rest = InTraits<In>::template one<float>(x[rest_place()]);
    }

    __device__ __forceinline__ void get(int u, float *v) const
    {
        if constexpr (sizeof(S) == 4) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[k] = bitcast<float>(w[u][k]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                v[2 * i] = InTraits<In>::template one<float>(uint16_t(w[u][i] & 0xffffu));
                v[2 * i + 1] = InTraits<In>::template one<float>(uint16_t(w[u][i] >> 16));
            }
        }
    }

    // results of vector u to the same places of out
    template <class Out, bool STREAM>
    __device__ __forceinline__ void put(typename OutTraits<Out>::S *out, int u, const float *v) const
    {
        using OW = Words<V * int(sizeof(typename OutTraits<Out>::S)) / 4>;
        typename OW::T o;
        if constexpr (sizeof(typename OutTraits<Out>::S) == 4) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                o[k] = bitcast<uint32_t>(v[k]);
        } else {
#pragma unroll
            for (int k = 0; k < V; k += 2)
                o[k / 2] = uint32_t(OutTraits<Out>::one(v[k])) | uint32_t(OutTraits<Out>::one(v[k + 1])) << 16;
        }
        if (has(u))
            OW::template store<STREAM>(out + place(u), o);
    }

    __device__ __forceinline__ float largest() const
    {
        float m = rest;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!any(u))
                continue;
            float v[V];
            get(u, v);
#pragma unroll
            for (int k = 0; k < V; ++k)
                m = OpMax::apply(m, v[k]);
        }
        return m;
    }

    template <bool GUARD>
    __device__ __forceinline__ float sum(float m, float c) const
    {
        float s = soft_term<true>(rest, m, c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!any(u))
                continue;
            float v[V];
            get(u, v);
#pragma unroll
            for (int k = 0; k < V; ++k)
                s += soft_term<GUARD>(v[k], m, c);
        }
        return s;
    }

    // place of the first entry equal to m, kNone where there is none
    __device__ __forceinline__ int first(float m) const
    {
        int f = has_rest() && rest == m ? rest_place() : kNone;
#pragma unroll
        for (int u = U - 1; u >= 0; --u) {
            if (!any(u))
                continue;
            float v[V];
            get(u, v);
#pragma unroll
            for (int k = V - 1; k >= 0; --k)
                if (v[k] == m && has(u))
                    f = place(u) + k;
        }
        return f;
    }

    // exp((x - m) / t) / s to out
    template <class Out, bool STREAM, bool GUARD>
    __device__ __forceinline__ void write(typename OutTraits<Out>::S *out, float m, float c, float inv) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!any(u))
                continue;
            float v[V];
            get(u, v);
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[k] = soft_term<GUARD>(v[k], m, c) * inv;
            put<Out, STREAM>(out, u, v);
        }
        if (has_rest())
            out[rest_place()] = OutTraits<Out>::one(soft_term<true>(rest, m, c) * inv);
    }

    // 1 at entry f, `others` elsewhere
    template <class Out, bool STREAM>
    __device__ __forceinline__ void write_one(typename OutTraits<Out>::S *out, int64_t f, float others) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!any(u))
                continue;
            float v[V];
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[k] = place(u) + k == f ? 1.0f : others;
            put<Out, STREAM>(out, u, v);
        }
        if (has_rest())
            out[rest_place()] = OutTraits<Out>::one(rest_place() == f ? 1.0f : others);
    }
};

// t <= 0, m the line's largest entry: what the entries but the first largest
// one get (NaN where there is a NaN), and whether there is a largest one.
__device__ __forceinline__ float others_of(float m) { return m == m ? 0.0f : m; }
__device__ __forceinline__ bool some(float m) { return m > -std::numeric_limits<float>::infinity(); }

// The factor 1 / s; s = 0 where all entries are masked: they get 0, or, at a
// NaN temperature (c, its factor, is NaN then), 0 * inf.
__device__ __forceinline__ float inverse(float s, float c) { return s == 0.0f && c == c ? 0.0f : 1.0f / s; }

// A line in the registers of LANES threads, BLOCK / LANES lines a block.  One
// block works on a line whose exponentials take a CU's VALUs longer than its
// bytes take to come, so each is computed once and kept, as float32.
template <class In, class Out, int LANES, int BLOCK>
__global__ __launch_bounds__(BLOCK) void k_soft_line(SoftmaxArgs a)
{
    constexpr int V = vec_of<In, Out>(), U = tune::kSoftPer / V;
    using P = Piece<In, V, LANES, U, false>;
    using O = typename OutTraits<Out>::S;
    constexpr int NW = LANES > 64 ? LANES / 64 : 1;
    __shared__ float part[2][NW];
    __shared__ int parti[NW];
    const int in_block = int(threadIdx.x / LANES);
    const int64_t line = int64_t(blockIdx.x) * (BLOCK / LANES) +
                         (LANES < 64 ? in_block : __builtin_amdgcn_readfirstlane(in_block));
    if (line >= a.lines)
        return;                               // (all of a line's lanes, and only where LANES <= 64: no barrier is missed)
    const float t = a.t ? a.t[line] : 1.0f;
    P p;
    p.load(static_cast<const typename P::S *>(a.x) + line * a.xs, int(a.n), int(threadIdx.x % LANES));
    O *out = static_cast<O *>(a.out) + line * a.os;
    const float m = line_all<OpMax, LANES>(p.largest(), part[0]);
    if (t <= 0.0f) {
        const int f = line_all<OpMin, LANES>(p.first(m), parti);
        p.template write_one<Out, false>(out, some(m) ? f : -1, others_of(m));
        return;
    }
    const float c = scale_of(t);
    float v[U][V], r;
    auto exponentials = [&](auto guard) {
        float s = r = soft_term<true>(p.rest, m, c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!p.any(u))
                continue;
            p.get(u, v[u]);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                v[u][k] = soft_term<decltype(guard)::value>(v[u][k], m, c);
                s += v[u][k];
            }
        }
        return s;
    };
    const float s = needs_guard(m, c) ? exponentials(std::true_type()) : exponentials(std::false_type());
    const float inv = inverse(line_all<OpSum, LANES>(s, part[1]), c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!p.any(u))
            continue;
#pragma unroll
        for (int k = 0; k < V; ++k)
            v[u][k] *= inv;
        p.template put<Out, false>(out, u, v[u]);
    }
    if (p.has_rest())
        out[p.rest_place()] = OutTraits<Out>::one(r * inv);
}

// Split lines: a tile is a wave's, the tiles of a block are of one line.
template <class In, int V, bool FULL>
using TilePiece = Piece<In, V, 64, tune::kSoftTile / (64 * V), FULL>;

struct Tile {
    int64_t line, base;       // its line, and its first entry there
    int64_t at;               // its place in the statistics
    int n;                    // its entries (<= 0: none)
};

// All of it is uniform over the wave, and kept in scalar registers.  BACK: the
// tiles from the last to the first, each on the XCD (block number modulo 8)
// that has it without.  The second launch goes back, so it begins with what
// the first has read last, which its L2 and the Infinity Cache still hold:
// 320 x 131072 bf16 to f32 50.1 us forwards, 48.2 us backwards.
template <bool BACK>
__device__ __forceinline__ Tile tile_of(const SoftmaxArgs &a)
{
    Tile t;
    uint32_t bid = blockIdx.x;
    const uint32_t eights = gridDim.x & ~(kXcds - 1);
    if (BACK && bid < eights)
        bid = eights - kXcds - (bid & ~(kXcds - 1)) + (bid & (kXcds - 1));
    const uint32_t line = divide(bid, a.per_line);
    const uint32_t tile = (bid - line * a.per_line.d) * (tune::kSoftBlock / 64) +
                          uint32_t(__builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)));
    t.line = line;
    t.base = int64_t(tile) * tune::kSoftTile;
    t.at = t.line * a.chunks + tile;
    const int64_t left = a.n - t.base;
    t.n = left < tune::kSoftTile ? int(left > 0 ? left : 0) : tune::kSoftTile;
    return t;
}

// The statistics of a tile.
template <class In, bool FULL>
__device__ __forceinline__ void tile_stats(const SoftmaxArgs &a, const Tile &tile)
{
    using P = TilePiece<In, InTraits<In>::vec, FULL>;
    P p;
    p.load(static_cast<const typename P::S *>(a.x) + tile.line * a.xs + tile.base, tile.n, lane_id());
    const float t = a.t ? a.t[tile.line] : 1.0f;
    const float m = wave_reduce<OpMax>(p.largest());
    const float c = scale_of(t);
    float s = 0.0f;
    int f = kNone;
    if (t <= 0.0f)
        f = wave_reduce<OpMin>(p.first(m));
    else
        s = wave_reduce<OpSum>(needs_guard(m, c) ? p.template sum<true>(m, c) : p.template sum<false>(m, c));
    if (lane_id() == 0) {
        a.stats[2 * tile.at] = m;
        a.stats[2 * tile.at + 1] = s;
        a.first[tile.at] = f;
    }
}

// First launch.
template <class In>
__global__ __launch_bounds__(tune::kSoftBlock) void k_soft_stats(SoftmaxArgs a)
{
    const Tile tile = tile_of<false>(a);
    if (tile.n == tune::kSoftTile)
        tile_stats<In, true>(a, tile);
    else if (tile.n > 0)
        tile_stats<In, false>(a, tile);
}

// A line's statistics.
struct Folded {
    float m, s;               // largest entry, sum (t > 0)
    int tile;                 // the first tile that holds the largest entry (t <= 0)
};

// Folded by `threads` threads, `reduce` giving all of them the reduction of
// their values.
template <class Reduce>
__device__ __forceinline__ Folded fold_line(const SoftmaxArgs &a, int64_t line, int thread, int threads, float t, float c,
                                            Reduce &&reduce)
{
    const float *st = a.stats + 2 * line * a.chunks;
    Folded l{OpMax::identity<float>(), 0.0f, kNone};
    for (int i = thread; i < a.chunks; i += threads)
        l.m = OpMax::apply(l.m, st[2 * i]);
    l.m = reduce(OpMax(), l.m);
    if (t <= 0.0f) {
        for (int i = thread; i < a.chunks; i += threads)
            if (st[2 * i] == l.m && i < l.tile)
                l.tile = i;
        l.tile = reduce(OpMin(), l.tile);
    } else {
        for (int i = thread; i < a.chunks; i += threads)
            l.s += st[2 * i + 1] * soft_term<true>(st[2 * i], l.m, c);
        l.s = reduce(OpSum(), l.s);
    }
    return l;
}

// The launch between, for lines of many tiles: one block a line.
__global__ __launch_bounds__(tune::kSoftBlock) void k_soft_fold(SoftmaxArgs a)
{
    constexpr int B = tune::kSoftBlock;
    __shared__ float part[2][B / 64];
    __shared__ int parti[B / 64];
    const int64_t line = blockIdx.x;
    const float t = a.t ? a.t[line] : 1.0f;
    int use = 0;
    const Folded l = fold_line(a, line, int(threadIdx.x), B, t, scale_of(t), [&](auto op, auto v) {
        if constexpr (std::is_same_v<decltype(v), int>)
            return line_all<decltype(op), B>(v, parti);
        else
            return line_all<decltype(op), B>(v, part[use++]);
    });
    if (threadIdx.x == 0) {
        a.stats[2 * (a.lines * a.chunks + line)] = l.m;
        a.stats[2 * (a.lines * a.chunks + line) + 1] = l.s;
        a.first[a.lines * a.chunks + line] = l.tile;
    }
}

__device__ __forceinline__ Folded folded(const SoftmaxArgs &a, int64_t line)
{
    const int64_t at = a.lines * a.chunks + line;
    return Folded{a.stats[2 * at], a.stats[2 * at + 1], a.first[at]};
}

// Write a tile of the line.
template <class In, class Out, bool STREAM, bool FULL>
__device__ __forceinline__ void tile_write(const SoftmaxArgs &a, const Tile &tile)
{
    using P = TilePiece<In, vec_of<In, Out>(), FULL>;
    P p;
    p.load(static_cast<const typename P::S *>(a.x) + tile.line * a.xs + tile.base, tile.n, lane_id());
    const float t = a.t ? a.t[tile.line] : 1.0f;
    const float c = scale_of(t);
    const Folded l = a.fold ? folded(a, tile.line) : fold_line(a, tile.line, lane_id(), 64, t, c, [](auto op, auto v) {
        return wave_reduce<decltype(op)>(v);
    });
    auto *out = static_cast<typename OutTraits<Out>::S *>(a.out) + tile.line * a.os + tile.base;
    if (t <= 0.0f) {
        int64_t at = -1;
        if (l.tile != kNone && some(l.m))
            at = int64_t(l.tile) * tune::kSoftTile + a.first[tile.line * a.chunks + l.tile] - tile.base;
        p.template write_one<Out, STREAM>(out, at, others_of(l.m));
        return;
    }
    const float inv = inverse(l.s, c);
    if (needs_guard(l.m, c))
        p.template write<Out, STREAM, true>(out, l.m, c, inv);
    else
        p.template write<Out, STREAM, false>(out, l.m, c, inv);
}

// Second launch.
template <class In, class Out, bool STREAM>
__global__ __launch_bounds__(tune::kSoftBlock) void k_soft_write(SoftmaxArgs a)
{
    const Tile tile = tile_of<true>(a);
    if (tile.n == tune::kSoftTile)
        tile_write<In, Out, STREAM, true>(a, tile);
    else if (tile.n > 0)
        tile_write<In, Out, STREAM, false>(a, tile);
}

template <class In, class Out, int LANES, int BLOCK>
void launch_line(const SoftmaxLaunch &L)
{
    launch_timed(k_soft_line<In, Out, LANES, BLOCK>, dim3(uint32_t(L.plan.grid)), dim3(BLOCK), 0, L.stream, L.ev_begin,
                 L.ev_end, L.a);
}

template <class In, class Out>
int run_softmax(const SoftmaxLaunch &L)
{
    if (L.plan.kernel == VK_SOFT_LINE) {
        switch (L.plan.lanes) {
        case 16: launch_line<In, Out, 16, 256>(L); break;
        case 64: launch_line<In, Out, 64, 256>(L); break;
        case 256: launch_line<In, Out, 256, 256>(L); break;
        case 512: launch_line<In, Out, 512, 512>(L); break;
        case 1024: launch_line<In, Out, 1024, 1024>(L); break;
        default: return ST_UNSUPPORTED;
        }
    } else {
        const dim3 grid(uint32_t(L.plan.grid)), block(L.plan.block);
        launch_timed(k_soft_stats<In>, grid, block, 0, L.stream, L.ev_begin, L.ev_end, L.a);
        if (L.plan.fold)
            launch_timed(k_soft_fold, dim3(uint32_t(L.a.lines)), block, 0, L.stream, nullptr, nullptr, L.a);
        if (L.plan.stream_out)
            launch_timed(k_soft_write<In, Out, true>, grid, block, 0, L.stream, nullptr, nullptr, L.a);
        else
            launch_timed(k_soft_write<In, Out, false>, grid, block, 0, L.stream, nullptr, nullptr, L.a);
    }
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
