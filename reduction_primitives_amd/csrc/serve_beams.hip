// serve_beams.hip -- beam search's selection: the `count` best continuations of a
// request's beams.
//
// Candidate (line j, token v) of a request scores
//     s = (x_jv - m_j) + (score_j - log sum_w exp(x_jw - m_j)),   m_j the line's largest logit
// in float64, from float32 exponentials: two lines' candidates may be as near as
// their logarithms.  Within a line s falls with x, so a line's best are its
// largest logits, and one pass over the logits finds both them and the sum.
//
// First launch: a wave takes consecutive tiles of a line, every lane keeping its
// own running maximum and sum.  The wave's best so far are a list across its
// lanes, sorted, and an entry is looked at again only if it passes the list's
// last one: after the first tile, one comparison of a lane's largest entry for 32.
// There the bar is the count-th largest of the lanes' maxima, found bit by bit
// with ballots.  Entries are inserted in the order of their tokens, so of equal
// ones the first stays first.
//
// Second launch: a block a request folds its lines' sums and merges their lists
// the same way, in float64.
#define RK_UNIT unit_serve_beams
#include "rk_serve_device.hpp"

namespace rk {
namespace {

constexpr int kB = tune::kBeamBlock;
constexpr int kTile = tune::kBeamTile;
constexpr int kWaves = kB / 64;
constexpr float kLog2e = 1.44269504f;
constexpr float kNone = -std::numeric_limits<float>::infinity();
constexpr double kNone64 = -std::numeric_limits<double>::infinity();

// Floats as integers of the same order (no NaN; -0 below 0).
__device__ __forceinline__ int32_t ordered(float v)
{
    const int32_t i = bitcast<int32_t>(v);
    return i ^ ((i >> 31) & 0x7fffffff);
}

__device__ __forceinline__ float from_ordered(int32_t i) { return bitcast<float>(i ^ ((i >> 31) & 0x7fffffff)); }

// The largest b so that n lanes hold a value of at least b (n <= 64 lanes, no NaN).
__device__ __forceinline__ int32_t nth_largest(int32_t v, int n)
{
    const uint32_t u = uint32_t(v) ^ 0x80000000u;
    uint32_t b = 0;
#pragma unroll
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t with = b | (1u << bit);
        b = __popcll(__ballot(u >= with)) >= n ? with : b;
    }
    return int32_t(b ^ 0x80000000u);
}

template <class T>
__device__ __forceinline__ T lane_before(T v)
{
    return move_words(v, [](uint32_t w) {
        return (uint32_t)__builtin_amdgcn_update_dpp((int)w, (int)w, 0x138, 0xf, 0xf, false);   // wave_shr:1
    });
}

// A wave's best entries, the i-th in lane i.
struct Best {
    float x;
    int32_t at;
    float bar;                // at least the n-th largest's value, or what is below it: only larger ones come in
    int n;

    __device__ explicit Best(int count) : x(kNone), at(-1), bar(kNone), n(count) {}

    // (wave-uniform v and i, in the order of i)
    __device__ __forceinline__ void insert(float v, int32_t i)
    {
        const int p = __popcll(__ballot(x >= v)), lane = lane_id();
        const float px = lane_before(x);
        const int32_t pa = lane_before(at);
        x = lane < p ? x : lane == p ? v : px;
        at = lane < p ? at : lane == p ? i : pa;
        bar = __builtin_fmaxf(bar, read_lane(x, n - 1));
    }
};

// A lane's entries of a tile, V of each of U vectors.
template <class In>
struct Tile {
    using S = typename InTraits<In>::S;
    static constexpr int V = InTraits<In>::vec, U = kTile / (64 * V);
    float v[U][V];

    __device__ __forceinline__ static int place(int u) { return (u * 64 + lane_id()) * V; }

    __device__ __forceinline__ void load(const S *x, int left)
    {
        if (left >= kTile) {
            u32x4 w[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                w[u] = Words<4>::load<true>(x + place(u));
            issue_barrier();
#pragma unroll
            for (int u = 0; u < U; ++u)
                InTraits<In>::decode(w[u], v[u]);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    v[u][k] = place(u) + k < left ? InTraits<In>::template one<float>(x[place(u) + k]) : kNone;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[u][k] += 0.0f;              // -0 is 0
    }

    __device__ __forceinline__ float largest(int u) const
    {
        float m = v[u][0];
#pragma unroll
        for (int k = 1; k < V; ++k)
            m = OpMax::apply(m, v[u][k]);
        return m;
    }

    __device__ __forceinline__ void select(Best &best, int32_t base) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float m = largest(u);
            for (uint64_t hit = __ballot(m > best.bar); hit;) {
                const int l = __builtin_ctzll(hit);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float x = read_lane(v[u][k], l);
                    if (x > best.bar)
                        best.insert(x, base + (u * 64 + l) * V + k);
                }
                hit = l == 63 ? 0 : __ballot(m > best.bar) & (~uint64_t(0) << (l + 1));
            }
        }
    }
};

__device__ __forceinline__ bool proposes(float score, bool ended) { return score > kNone && !ended; }

template <class In>
__global__ __launch_bounds__(kB) void k_beam_lines(BeamArgs a)
{
    using S = typename InTraits<In>::S;
    using T = Tile<In>;
    const int64_t item = int64_t(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    if (item >= a.items)
        return;
    const int64_t line = item / a.chunks;
    const int chunk = int(item - line * a.chunks);
    if (!proposes(a.scores[line], a.ended && a.ended[line]))
        return;                                // (nothing of this line is read by the second launch)
    const S *x = static_cast<const S *>(a.x) + line * a.stride;
    const int64_t from = int64_t(chunk) * a.per_wave, to = from + a.per_wave < a.n ? from + a.per_wave : a.n;
    Best best(a.count);
    float m = kNone;
    double s = 0.0;
    for (int64_t base = from; base < to; base += kTile) {
        T t;
        t.load(x + base, int(to - base < kTile ? to - base : kTile));
        float top = t.largest(0);
#pragma unroll
        for (int u = 1; u < T::U; ++u)
            top = OpMax::apply(top, t.largest(u));
        const float now = OpMax::apply(m, top), ref = now > kNone ? now : 0.0f;
        float part = 0.0f;
#pragma unroll
        for (int u = 0; u < T::U; ++u)
#pragma unroll
            for (int k = 0; k < T::V; ++k)
                part += __builtin_amdgcn_exp2f((t.v[u][k] - ref) * kLog2e);
        s = s * double(__builtin_amdgcn_exp2f((m - ref) * kLog2e)) + double(part);
        m = now;
        const uint64_t over = __ballot(top > best.bar);
        if (over) {
            // many lanes at once: of their largest entries the count-th best bars the rest
            if (__popcll(over) > a.count) {
                const int32_t k = nth_largest(ordered(top == top ? top : kNone), a.count);
                best.bar = __builtin_fmaxf(best.bar, from_ordered(k == 0 ? -2 : k - 1));   // (-1: -0, which is 0)
            }
            t.select(best, int32_t(base));
        }
    }
    // (a NaN in a lane makes the maximum one)
    const float all = wave_reduce<OpMax>(m);
    const float ref = all > kNone ? all : 0.0f;
    const double sum = wave_reduce<OpSum>(s * double(__builtin_amdgcn_exp2f((m - ref) * kLog2e)));
    const int lane = lane_id();
    if (lane == 0) {
        a.tops[item] = all;
        a.sums[item] = sum;
    }
    if (lane < a.count) {
        a.best_x[item * a.count + lane] = best.x;
        a.best_at[item * a.count + lane] = best.at;
    }
}

// A candidate of the second launch, and the order of two.
struct Candidate {
    double s;
    float x;
    int32_t line, at;         // line of the request
    __device__ __forceinline__ bool before(const Candidate &o) const
    {
        if (s != o.s)
            return s > o.s;
        if (line != o.line)
            return line < o.line;
        return x != o.x ? x > o.x : at < o.at;
    }
};

__device__ __forceinline__ Candidate read_candidate(const Candidate &c, int l)
{
    return Candidate{read_lane(c.s, l), read_lane(c.x, l), read_lane(c.line, l), read_lane(c.at, l)};
}

struct Merge {
    Candidate c;              // the i-th best in lane i
    double bar;
    int n;

    __device__ explicit Merge(int count) : c{kNone64, kNone, 0x7fffffff, 0x7fffffff}, bar(kNone64), n(count) {}

    __device__ __forceinline__ void insert(const Candidate &v)
    {
        const int p = __popcll(__ballot(c.before(v))), lane = lane_id();
        const Candidate q{lane_before(c.s), lane_before(c.x), lane_before(c.line), lane_before(c.at)};
        if (lane == p)
            c = v;
        else if (lane > p)
            c = q;
        bar = read_lane(c.s, n - 1);
    }

    // 64 candidates, those of -inf left out
    __device__ __forceinline__ void offer(const Candidate &v)
    {
        uint64_t over = __ballot(v.s > kNone64 && v.s >= bar);
        if (__popcll(over) > n) {
            // rounded to float32 (monotone), the n-th best bars what is below it
            const float f = from_ordered(nth_largest(ordered(float(v.s) + 0.0f), n));
            over &= __ballot(float(v.s) >= f);
        }
        for (uint64_t hit = over; hit; hit &= hit - 1) {
            const int l = __builtin_ctzll(hit);
            if (read_lane(v.s, l) >= bar)
                insert(read_candidate(v, l));
        }
    }
};

template <class Tok>
__global__ __launch_bounds__(kB) void k_beam_merge(BeamArgs a)
{
    extern __shared__ double s_base[];        // of every line: score - log sum, -inf: no candidate
    float *s_top = reinterpret_cast<float *>(s_base + a.beams);   // and what is taken from its logits first
    __shared__ Candidate s_list[kWaves][64];
    __shared__ int s_odd[kWaves];
    const int64_t req = blockIdx.x, line0 = req * a.beams;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    bool odd = false;                          // NaN or +inf where there is something to choose
    for (int j = wave; j < a.beams; j += kWaves) {
        const float score = a.scores[line0 + j];
        const bool ended = a.ended && a.ended[line0 + j];
        double base = kNone64;
        float m = 0.0f;
        odd |= !(score < std::numeric_limits<float>::infinity());
        if (proposes(score, ended)) {
            const int64_t i0 = (line0 + j) * a.chunks;
            m = kNone;
            for (int c = lane; c < a.chunks; c += 64)
                m = OpMax::apply(m, a.tops[i0 + c]);
            m = wave_reduce<OpMax>(m);
            odd |= !(m < std::numeric_limits<float>::infinity());
            if (m > kNone && m < std::numeric_limits<float>::infinity()) {
                double s = 0.0;
                for (int c = lane; c < a.chunks; c += 64)
                    s += a.sums[i0 + c] * exp(double(a.tops[i0 + c]) - double(m));
                s = wave_reduce<OpSum>(s);
                base = double(score) - log(s);
            }
        } else if (ended) {
            base = double(score);
        }
        if (lane == 0) {
            s_base[j] = base;
            s_top[j] = m;
        }
    }
    if (lane == 0)
        s_odd[wave] = odd;
    __syncthreads();
    Merge best(a.count);
    const int64_t per_line = int64_t(a.chunks) * a.count, all = per_line * a.beams;
    for (int64_t i0 = int64_t(wave) * 64; i0 < all; i0 += kB) {
        const int64_t i = i0 + lane;
        Candidate v{kNone64, kNone, 0, 0};
        if (i < all) {
            const int j = int(i / per_line);
            const int64_t k = i - int64_t(j) * per_line;
            v.line = j;
            if (a.ended && a.ended[line0 + j]) {
                if (k == 0) {
                    v.s = s_base[j];
                    v.x = 0.0f;
                    v.at = int32_t(a.end_token);
                }
            } else if (s_base[j] > kNone64) {
                const int64_t e = line0 * per_line + i;
                v.x = a.best_x[e];
                v.at = a.best_at[e];
                if (v.x > kNone)
                    v.s = (double(v.x) - double(s_top[j])) + s_base[j];
            }
        }
        best.offer(v);
    }
    if (wave > 0)
        s_list[wave][lane] = best.c;
    __syncthreads();
    if (wave != 0)
        return;
    for (int w = 1; w < kWaves; ++w) {
        Candidate v = s_list[w][lane];
        if (lane >= a.count)
            v.s = kNone64;
        best.offer(v);
    }
    bool bad = false;
    for (int w = 0; w < kWaves; ++w)
        bad |= s_odd[w] != 0;
    if (lane < a.count) {
        const bool some = !bad && best.c.s > kNone64;
        const int64_t o = req * a.count + lane;
        a.best[o] = bad ? std::numeric_limits<float>::quiet_NaN() : float(best.c.s);
        static_cast<Tok *>(a.tokens)[o] = some ? Tok(best.c.at) : Tok(-1);
        a.parents[o] = some ? int32_t(line0 + best.c.line) : -1;
    }
}

template <class In>
void launch_lines(const BeamLaunch &L)
{
    launch_timed(k_beam_lines<In>, dim3(uint32_t(L.plan.grid)), dim3(kB), 0, L.stream, L.ev_begin, L.ev_end, L.a);
}

}  // namespace

int launch_beams(const BeamLaunch &L)
{
    switch (L.dtype) {
    case F32: launch_lines<float>(L); break;
    case BF16: launch_lines<bf16_in>(L); break;
    default: launch_lines<f16_in>(L); break;
    }
    if (hipGetLastError() != hipSuccess)
        return ST_HIP;
    const size_t lds = size_t(L.a.beams) * 12;
    const auto kernel = L.token_dtype == I32 ? k_beam_merge<int32_t> : k_beam_merge<int64_t>;
    hipLaunchKernelGGL(kernel, dim3(uint32_t(L.a.req)), dim3(kB), lds, static_cast<hipStream_t>(L.stream), L.a);
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

}  // namespace rk
