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
// own running maximum and sum.  What passes the wave's bar goes to a list in LDS, in
// any order, and when that holds more than 64 the count-th largest is found bit by
// bit with ballots, the rest dropped, and the bar raised to it; a tile none of whose
// lanes' largest entries passes costs one comparison.  In the first tile the bar is
// the count-th largest of the lanes' maxima, later also what other waves of the block
// have for the same line.  (A sorted list across the lanes, each entry put in its
// place: 50 instructions an entry, more than the exponentials, and 41 us where this
// takes 33, at 512 lines of 131072 bf16.)  Equal entries without end, as in a line of
// one value, are put into such a list all the same, one after the other.
//
// Second launch: a block a request folds its lines' sums, finds a bar the same way,
// and ranks what is left, all against all, in float64.
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

// The n-th largest of the values of the lanes, two a lane (no NaN), found bit by bit,
// as an unsigned integer of the same order, for values whose LOW lowest bits do not
// matter (all 0 or all 1).  n values are at least it.
template <int LOW>
__device__ __forceinline__ uint32_t nth_of(uint32_t u, uint32_t w, int n)
{
    uint32_t b = 0;
#pragma unroll
    for (int bit = 31; bit >= LOW; --bit) {
        const uint32_t with = b | (1u << bit);
        b = __popcll(__ballot(u >= with)) + __popcll(__ballot(w >= with)) >= n ? with : b;
    }
    return b;
}

__device__ __forceinline__ uint32_t rising(float v) { return uint32_t(ordered(v)) ^ 0x80000000u; }

// One value a lane.
template <int LOW>
__device__ __forceinline__ float nth_largest(float v, int n)
{
    const uint32_t u = rising(v);
    uint32_t b = 0;
#pragma unroll
    for (int bit = 31; bit >= LOW; --bit) {
        const uint32_t with = b | (1u << bit);
        b = __popcll(__ballot(u >= with)) >= n ? with : b;
    }
    return from_ordered(int32_t((b >> 31 ? b : b | ((1u << LOW) - 1)) ^ 0x80000000u));
}

// The next smaller float (of 0 and -0 what is below both).
__device__ __forceinline__ float below(float v)
{
    const int32_t i = ordered(v);
    return from_ordered(i == 0 ? -2 : i - 1);
}

template <class T>
__device__ __forceinline__ T lane_before(T v)
{
    return move_words(v, [](uint32_t w) {
        return (uint32_t)__builtin_amdgcn_update_dpp((int)w, (int)w, 0x138, 0xf, 0xf, false);   // wave_shr:1
    });
}

// A wave's best entries in order, the i-th in lane i.
struct Best {
    float x;
    int32_t at;
    float bar;                // at least the n-th largest's value, or what is below it: only larger ones come in
    int n;

    __device__ explicit Best(int count) : x(kNone), at(-1), bar(kNone), n(count) {}

    // (wave-uniform v and i)
    __device__ __forceinline__ void insert(float v, int32_t i)
    {
        const int p = __popcll(__ballot(x > v || (x == v && at < i))), lane = lane_id();
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
    static constexpr int LOW = std::is_same_v<In, bf16_in> ? 16 : std::is_same_v<In, f16_in> ? 13 : 0;   // bits that are all alike
    float v[U][V];

    // A whole tile as it comes from memory.
    struct Raw {
        u32x4 w[U];
        __device__ __forceinline__ void load(const S *x)
        {
#pragma unroll
            for (int u = 0; u < U; ++u)
                w[u] = Words<4>::load<true>(x + place(u));
        }
    };

    __device__ __forceinline__ static int place(int u) { return (u * 64 + lane_id()) * V; }

    __device__ __forceinline__ void decode(const Raw &r)
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
            InTraits<In>::decode(r.w[u], v[u]);
    }

    // the line's end: `left` entries, fewer than a tile's
    __device__ __forceinline__ void load_rest(const S *x, int left)
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[u][k] = place(u) + k < left ? InTraits<In>::template one<float>(x[place(u) + k]) : kNone;
    }

    __device__ __forceinline__ float largest(int u) const
    {
        float m = v[u][0];
#pragma unroll
        for (int k = 1; k < V; ++k)
            m = OpMax::apply(m, v[u][k]);
        return m;
    }

    // f(u, k, which lanes' entries pass)
    template <class F>
    __device__ __forceinline__ void passing(const float (&tops)[U], float bar, F &&f) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (__ballot(tops[u] > bar))
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const uint64_t m = __ballot(v[u][k] > bar);
                    if (m)
                        f(u, k, m);
                }
    }

    // one after the other, in the order of their tokens
    __device__ __forceinline__ void select(Best &best, int32_t base) const
    {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float m = largest(u);
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

constexpr int kList = 128;

// A wave's entries that may be among its line's best, in LDS.
template <class In>
struct List {
    using T = Tile<In>;
    float *x;
    int32_t *at;
    int n, count;
    float bar;                // at least `count` entries of the line are larger or, of lower tokens, as large

    __device__ __forceinline__ static void in_order()
    {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }

    __device__ __forceinline__ void take(const T &t, const float (&tops)[T::U], int32_t base)
    {
        const int before = n, lane = lane_id();
        t.passing(tops, bar, [&](int u, int k, uint64_t m) {
            const int p = n + int(__builtin_amdgcn_mbcnt_hi(uint32_t(m >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(m), 0)));
            if ((m >> lane & 1) && p < kList) {
                x[p] = t.v[u][k];
                at[p] = base + (u * 64 + lane) * T::V + k;
            }
            n += __popcll(m);
        });
        in_order();
        if (n > kList) {
            n = before;
            in_turn(t, base);
        } else if (n > 64) {
            drop();
        }
    }

    // The `count` best, of equal ones those of the lowest tokens.
    __device__ __forceinline__ void drop()
    {
        if (n <= count)
            return;
        const int lane = lane_id();
        const bool some[2] = {lane < n, lane + 64 < n};
        float v[2];
        int32_t i[2];
        uint32_t u[2];
        uint64_t keep[2], equal[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v[h] = x[lane + 64 * h];
            i[h] = at[lane + 64 * h];
            u[h] = some[h] ? rising(v[h] + 0.0f) : 0;      // (0 is no number's)
        }
        const uint32_t b = nth_of<T::LOW>(u[0], u[1], count);
        int over = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            keep[h] = __ballot(some[h] && u[h] >> T::LOW >= b >> T::LOW);
            equal[h] = __ballot(some[h] && u[h] >> T::LOW == b >> T::LOW);
            over += __popcll(keep[h]);
        }
        for (; over > count; --over) {
            const int32_t a0 = equal[0] >> lane & 1 ? i[0] : -1, a1 = equal[1] >> lane & 1 ? i[1] : -1;
            const int32_t last = wave_reduce<OpMax>(a0 > a1 ? a0 : a1);
            const uint64_t out[2] = {__ballot(a0 == last), __ballot(a1 == last)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                equal[h] &= ~out[h];
                keep[h] &= ~out[h];
            }
        }
        in_order();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (keep[h] >> lane & 1) {
                const int p = (h ? __popcll(keep[0]) : 0) + __popcll(keep[h] & ((uint64_t(1) << lane) - 1));
                x[p] = v[h];
                at[p] = i[h];
            }
        n = count;
        in_order();
        bar = __builtin_fmaxf(bar, from_ordered(int32_t((b >> 31 ? b : b | ((1u << T::LOW) - 1)) ^ 0x80000000u)));
    }

    __device__ __forceinline__ void in_turn(const T &t, int32_t base)
    {
        Best best(count);
        const int lane = lane_id();
        for (int i = 0; i < n; ++i)
            best.insert(x[i], at[i]);
        best.bar = __builtin_fmaxf(best.bar, bar);
        t.select(best, base);
        in_order();
        if (lane < count) {
            x[lane] = best.x;
            at[lane] = best.at;
        }
        n = __popcll(__ballot(lane < count && best.x > kNone));
        bar = best.bar;
        in_order();
    }
};

__device__ __forceinline__ bool proposes(float score, bool ended) { return score > kNone && !ended; }

template <class In>
__global__ __launch_bounds__(kB) void k_beam_lines(BeamArgs a)
{
    using S = typename InTraits<In>::S;
    using T = Tile<In>;
    // the waves' bars: of those that go through the same line, the highest holds for all
    __shared__ float s_bar[kWaves], s_x[kWaves][kList];
    __shared__ int32_t s_at[kWaves][kList];
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    if (threadIdx.x < kWaves)
        s_bar[threadIdx.x] = kNone;
    __syncthreads();
    const int64_t item = int64_t(blockIdx.x) * kWaves + wave;
    if (item >= a.items)
        return;
    const int64_t line = uint32_t(item) / uint32_t(a.chunks);
    const int chunk = int(item - line * a.chunks);
    if (!proposes(a.scores[line], a.ended && a.ended[line]))
        return;                                // (nothing of this line is read by the second launch)
    const S *x = static_cast<const S *>(a.x) + line * a.stride;
    const int64_t from = int64_t(chunk) * a.per_wave, to = from + a.per_wave < a.n ? from + a.per_wave : a.n;
    List<In> best{s_x[wave], s_at[wave], 0, a.count, kNone};
    float m = kNone;
    double s = 0.0;
    typename T::Raw raw;                       // the next tile is on its way while one is gone through
    if (from + kTile <= to)
        raw.load(x + from);
    for (int64_t base = from; base < to; base += kTile) {
        T t;
        if (base + kTile <= to)
            t.decode(raw);
        else
            t.load_rest(x + base, int(to - base));
        if (base + 2 * kTile <= to)
            raw.load(x + base + kTile);
        issue_barrier();
        float tops[T::U], top = tops[0] = t.largest(0);
#pragma unroll
        for (int u = 1; u < T::U; ++u)
            top = OpMax::apply(top, tops[u] = t.largest(u));
        top += 0.0f;                           // (-0 is 0, where they are ordered as integers)
        const float now = OpMax::apply(m, top), ref = now > kNone ? now : 0.0f;
        float part = 0.0f;
#pragma unroll
        for (int u = 0; u < T::U; ++u)
#pragma unroll
            for (int k = 0; k < T::V; ++k)
                part += __builtin_amdgcn_exp2f((t.v[u][k] - ref) * kLog2e);
        s = s * double(__builtin_amdgcn_exp2f((m - ref) * kLog2e)) + double(part);
        m = now;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            if (w >= wave - chunk && w < wave - chunk + a.chunks) {   // (`count` entries reach it: one that does not is out)
                const float b = __hip_atomic_load(s_bar + w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
                best.bar = b > kNone && w != wave ? __builtin_fmaxf(best.bar, below(b)) : best.bar;
            }
        const uint64_t over = __ballot(top > best.bar);
        if (over) {
            // many lanes at once: of their largest entries the count-th best bars the rest
            if (__popcll(over) > a.count)
                best.bar = __builtin_fmaxf(best.bar, below(nth_largest<T::LOW>(top == top ? top : kNone, a.count)));
            best.take(t, tops, int32_t(base));
            if (lane_id() == 0)
                __hip_atomic_store(s_bar + wave, best.bar, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
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
    best.drop();
    if (lane < a.count) {
        a.best_x[item * a.count + lane] = lane < best.n ? best.x[lane] : kNone;
        a.best_at[item * a.count + lane] = best.at[lane];
    }
}

// A candidate of the second launch, and the order of two.
struct Candidate {
    double s;
    float x;
    int32_t line, at;         // line of the request
    __device__ __forceinline__ bool before(const Candidate &o) const
    {
        // (no branches: all four are there already)
        const bool by_at = (x > o.x) | ((x == o.x) & (at < o.at));
        const bool by_line = (line < o.line) | ((line == o.line) & by_at);
        return (s > o.s) | ((s == o.s) & by_line);
    }
};

__device__ __forceinline__ Candidate read_candidate(const Candidate &c, int l)
{
    return Candidate{read_lane(c.s, l), read_lane(c.x, l), read_lane(c.line, l), read_lane(c.at, l)};
}

// The best candidates of a wave, the i-th in lane i.
struct Merge {
    Candidate c;
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
        for (uint64_t hit = __ballot(v.s > kNone64 && v.s >= bar); hit; hit &= hit - 1) {
            const int l = __builtin_ctzll(hit);
            if (read_lane(v.s, l) >= bar)
                insert(read_candidate(v, l));
        }
    }
};

// What is kept of a request's lines for its second launch.
struct Lines {
    const BeamArgs &a;
    int64_t line0;
    const double *base;       // score - log sum; -inf: no candidate
    const float *top;         // what is taken from the logits first

    // Entry i of the request's lists (a line's that has none may hold anything).
    struct Entry {
        float x;
        int32_t at;
    };
    __device__ __forceinline__ Entry entry(uint32_t i) const
    {
        const int64_t e = line0 * int64_t(a.per_line.d) + i;
        return Entry{a.best_x[e], a.best_at[e]};
    }
    // the candidate it is (of s = -inf: none)
    __device__ __forceinline__ Candidate candidate(uint32_t i, const Entry &e) const
    {
        const uint32_t j = divide(i, a.per_line);
        Candidate v{kNone64, e.x, int32_t(j), e.at};
        const float t = top[j];
        if (t == kEnded) {
            if (i == j * a.per_line.d) {
                v.s = base[j];
                v.x = 0.0f;
                v.at = int32_t(a.end_token);
            }
        } else if (base[j] > kNone64 && e.x > kNone) {
            v.s = (double(e.x) - double(t)) + base[j];
        }
        return v;
    }
    __device__ __forceinline__ Candidate candidate(uint32_t i) const { return candidate(i, entry(i)); }
    static constexpr float kEnded = kNone;    // a top that no line with candidates has
};

// Sum or largest value over each group of `lanes` neighbouring lanes.
template <class Op, class T>
__device__ __forceinline__ T group_reduce(T v, int lanes)
{
    for (int d = 1; d < lanes; d *= 2) {
        const int from = lane_id() ^ d;
        v = Op::apply(v, move_words(v, [from](uint32_t w) { return bpermute32(w, from); }));
    }
    return v;
}

constexpr int kNear = 512;                     // candidates that are ranked against each other

template <class Tok>
__global__ __launch_bounds__(kB) void k_beam_merge(BeamArgs a)
{
    extern __shared__ double s_base[];        // of every line, then their tops
    float *s_top = reinterpret_cast<float *>(s_base + a.beams);
    __shared__ Candidate s_near[kNear];
    __shared__ int s_odd, s_count;
    __shared__ float s_bar[kWaves];
    const int64_t req = blockIdx.x, line0 = req * a.beams;
    const int tid = int(threadIdx.x), lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (tid == 0) {
        s_odd = 0;
        s_count = 0;
    }
    __syncthreads();
    const Lines lines{a, line0, s_base, s_top};
    const uint32_t all = a.per_line.d * uint32_t(a.beams);
    // a thread's first entries, on their way while the lines' sums are
    constexpr int kMine = 4;
    Lines::Entry mine[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        mine[k] = lines.entry(uint32_t(tid + k * kB) < all ? tid + k * kB : 0);
    bool odd = false;                          // NaN or +inf where there is something to choose
    const int group = a.lanes;                 // lanes that share a line's chunks
    for (int j0 = 0; j0 < a.beams; j0 += kB / group) {
        const int j = j0 + tid / group;
        const bool there = j < a.beams;
        const int64_t i0 = (line0 + (there ? j : 0)) * a.chunks, first = i0 + (tid % group < a.chunks ? tid % group : 0);
        const float score = there ? a.scores[line0 + j] : kNone, top0 = a.tops[first];
        const double sum0 = a.sums[first];
        const bool ended = there && a.ended && a.ended[line0 + j], live = there && proposes(score, ended);
        float m = live && tid % group < a.chunks ? top0 : kNone;
        double s = 0.0;
        if (live)
            for (int64_t c = tid % group + group; c < a.chunks; c += group)
                m = OpMax::apply(m, a.tops[i0 + c]);
        m = group_reduce<OpMax>(m, group);
        const bool fine = live && m > kNone && m < std::numeric_limits<float>::infinity();
        if (fine) {
            if (tid % group < a.chunks)
                s = sum0 * exp(double(top0) - double(m));
            for (int64_t c = tid % group + group; c < a.chunks; c += group)
                s += a.sums[i0 + c] * exp(double(a.tops[i0 + c]) - double(m));
        }
        s = group_reduce<OpSum>(s, group);
        odd |= there && !(score < std::numeric_limits<float>::infinity());
        odd |= live && !(m < std::numeric_limits<float>::infinity());
        if (there && tid % group == 0) {
            s_base[j] = fine ? double(score) - log(s) : ended ? double(score) : kNone64;
            s_top[j] = fine ? m : Lines::kEnded;
        }
    }
    if (odd)
        s_odd = 1;
    __syncthreads();

    // A bar below which nothing is kept: the count-th largest of the lanes' best, rounded to float32 (which keeps
    // their order), of the wave where that is highest.
    float low = kNone;
    Candidate first[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        first[k] = lines.candidate(uint32_t(tid + k * kB) < all ? tid + k * kB : 0, mine[k]);
        if (uint32_t(tid + k * kB) >= all)
            first[k].s = kNone64;
        low = __builtin_fmaxf(low, float(first[k].s) + 0.0f);
    }
    for (uint32_t i = tid + kMine * kB; i < all; i += kB)
        low = __builtin_fmaxf(low, float(lines.candidate(i).s) + 0.0f);
    const float bar = nth_largest<0>(low, a.count);
    if (lane == 0)
        s_bar[wave] = bar;
    __syncthreads();
    low = s_bar[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
        low = __builtin_fmaxf(low, s_bar[w]);
    // What is left is ranked, all against all.
    const auto keep = [&](const Candidate &v) {
        if (v.s > kNone64 && float(v.s) >= low) {
            const int at = atomicAdd(&s_count, 1);
            if (at < kNear)
                s_near[at] = v;
        }
    };
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        keep(first[k]);
    for (uint32_t i = tid + kMine * kB; i < all; i += kB)
        keep(lines.candidate(i));
    __syncthreads();
    const int near = s_count;
    const bool bad = s_odd != 0;
    const auto write = [&](int64_t o, const Candidate &c, bool some) {
        a.best[o] = bad ? std::numeric_limits<float>::quiet_NaN() : some ? float(c.s) : kNone;
        static_cast<Tok *>(a.tokens)[o] = some && !bad ? Tok(c.at) : Tok(-1);
        a.parents[o] = some && !bad ? int32_t(line0 + c.line) : -1;
    };
    if (near <= kNear) {
        // `share` lanes a candidate, each against every share-th; four reads on their way at once.  (One lane a
        // candidate and one read after the other took 10 us of 19 at 64 requests of 8 lines.)
        int share = 1;
        while (share < 16 && near * share * 2 <= kB)
            share *= 2;
        for (int i0 = 0; i0 < near; i0 += kB / share) {
            const int i = i0 + tid / share, mod = tid % share;
            const Candidate v = s_near[i < near ? i : 0];
            int rank = 0;
            for (int k = mod; k < near; k += 4 * share) {
                Candidate o[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    o[u] = s_near[k + u * share < near ? k + u * share : k];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    rank += int(o[u].before(v)) & int(k + u * share < near);
            }
            rank = group_reduce<OpSum>(rank, share);
            if (mod == 0 && i < near && rank < a.count)
                write(req * a.count + rank, v, true);
        }
        for (int i = near + tid; i < a.count; i += kB)
            write(req * a.count + i, Candidate{}, false);
        return;
    }
    // Too many alike: one after the other, a quarter of them a wave.
    Merge best(a.count);
    for (uint32_t i0 = uint32_t(wave) * 64; i0 < all; i0 += kB) {
        Candidate v{kNone64, kNone, 0, 0};
        if (i0 + lane < all)
            v = lines.candidate(i0 + lane);
        best.offer(v);
    }
    __syncthreads();
    s_near[wave * 64 + lane] = best.c;
    __syncthreads();
    if (wave != 0)
        return;
    for (int w = 1; w < kWaves; ++w) {
        Candidate v = s_near[w * 64 + lane];
        if (lane >= a.count)
            v.s = kNone64;
        best.offer(v);
    }
    if (lane < a.count)
        write(req * a.count + lane, best.c, best.c.s > kNone64);
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
