// serve_verify.hip -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Request b keeps its drafted tokens x_0, x_1, ... while
//     u_i q_i(x_i) < p_i(x_i)
// (the product of two float32 values is exact in float64, so the comparison
// is).  At the first one turned down, i, the next token is drawn from
//     w_j = max(p_i(j) - q_i(j), 0),
// after the last one from w = p: the first j whose running sum passes
// r sum(w).  Running sums are float64: a border between two tokens then moves
// by 2^-52 of the whole sum with the order of the additions, not by the 2^-23
// that would change drawn tokens.
//
// Only one target line per request, and one draft line where a token is
// turned down, is read.  Every block of a request finds the kept tokens by
// itself (a few dependent loads, all drafts at once) and sums its tiles of the
// line, a tile a wave.  Then one block finds the tile in which the running sum
// passes and goes through that tile alone: the request's last to arrive, or a
// second launch's where blocks or requests are many and in a captured call.
#define RK_UNIT unit_serve_verify
#include "rk_serve_device.hpp"

namespace rk {
namespace {

constexpr int kB = tune::kVerifyBlock;
constexpr int kTile = tune::kVerifyTile;

// Probabilities that are not positive finite numbers weigh nothing.
__device__ __forceinline__ double weight(double w)
{
    return w > 0.0 && w < __builtin_inf() ? w : 0.0;
}

template <class Tok>
__device__ __forceinline__ int64_t token_at(const void *p, int64_t i)
{
    return static_cast<const Tok *>(p)[i];
}

template <class T>
__device__ __forceinline__ T wave_uniform(T v)
{
    return move_words(v, [](uint32_t w) { return uint32_t(__builtin_amdgcn_readfirstlane(int(w))); });
}

template <class In, class Tok>
__device__ __forceinline__ VerifyDrawn accept(const VerifyArgs &a, int64_t b)
{
    using S = typename InTraits<In>::S;
    VerifyDrawn d;
    int64_t lo = b * a.max_draft, hi = lo + a.max_draft;
    if (a.starts) {
        lo = a.starts[b];
        hi = a.starts[b + 1];
        lo = lo < 0 ? 0 : lo > a.drafts ? a.drafts : lo;
        hi = hi < lo ? lo : hi > a.drafts ? a.drafts : hi;
        hi = hi - lo > a.max_draft ? lo + a.max_draft : hi;
    }
    // uniform, and kept in scalar registers: addresses that follow from it take none of the vector ones
    lo = wave_uniform(lo);
    d.lo = lo;
    d.count = wave_uniform(int(hi - lo));
    d.kept = d.count;
    d.x = -1;
    for (int base = 0; base < d.count; base += 64) {
        const int i = base + lane_id();
        bool turned = false;
        int64_t x = -1;
        if (i < d.count) {
            x = token_at<Tok>(a.drafted, lo + i);
            turned = true;
            if (x >= 0 && x < a.n) {
                const double p = weight(InTraits<In>::template one<double>(
                    static_cast<const S *>(a.p)[(lo + i + b) * a.ps + x]));
                const double q = a.q ? InTraits<In>::template one<double>(static_cast<const S *>(a.q)[(lo + i) * a.qs + x])
                                     : 1.0;
                turned = !(double(a.u[lo + i]) * q < p);
            }
        }
        const uint64_t m = __ballot(turned);
        if (m) {
            const int at = __builtin_ctzll(m);
            d.kept = base + at;
            d.x = wave_uniform(read_lane(x, at));
            break;
        }
    }
    d.kept = wave_uniform(d.kept);
    return d;
}

// The lines of the request's next token: target line p, draft line q (NULL:
// nothing to subtract), and the one token whose weight loses 1 (-1: none).
template <class S> struct Lines {
    const S *p, *q;
    int64_t x;
};

template <class S>
__device__ __forceinline__ Lines<S> lines_of(const VerifyArgs &a, int64_t b, const VerifyDrawn &d)
{
    Lines<S> l;
    l.p = static_cast<const S *>(a.p) + (d.lo + d.kept + b) * a.ps;
    const bool turned = d.kept < d.count;
    l.q = turned && a.q ? static_cast<const S *>(a.q) + (d.lo + d.kept) * a.qs : nullptr;
    l.x = turned && !a.q ? d.x : -1;
    return l;
}

// Weights of V consecutive entries, one vector load a line: entries i .. i +
// V - 1 after entry `base` of the line (base uniform, i a lane's).  Entries from n
// on weigh nothing: a vector that would pass the line's end is read from n - V
// instead and its first entries, which belong to others, dropped.
// FAST: the vectors do not pass the line's end, l.x is not among them, and
// infinities (which weigh nothing) come out as infinities.  These are the
// lines' bulk, read once and past the caches (256 x 7 x 131072 f32, captured:
// 36.7 us without that, 32.9 with).
template <class In, bool FAST, class S>
struct Loaded {
    static constexpr int V = InTraits<In>::vec;
    u32x4 p, q;

    // the vector's first entry, after base
    __device__ __forceinline__ static int at(int i, int64_t left) { return FAST || i + V <= left ? i : int(left) - V; }

    // left: entries of the line after base
    __device__ __forceinline__ void load(const S *lp, const S *lq, int i, int64_t left)
    {
        p = Words<4>::load<FAST>(lp + at(i, left));
        if (lq)
            q = Words<4>::load<FAST>(lq + at(i, left));
    }

    // x: l.x after base
    __device__ __forceinline__ void weights(const S *lq, int i, int64_t left, int64_t x, double *w) const
    {
        InTraits<In>::decode(p, w);
        if (lq) {
            double f[V];
            InTraits<In>::decode(q, f);
#pragma unroll
            for (int k = 0; k < V; ++k)
                w[k] -= f[k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (FAST) {
                w[k] = __builtin_fmax(w[k], 0.0);          // (NaN: 0)
            } else {
                w[k] = weight(at(i, left) + k == x ? w[k] - 1.0 : w[k]);
                w[k] = at(i, left) + k < i ? 0.0 : w[k];
            }
        }
    }
};

// Lines shorter than a vector.
template <class In, class S>
__device__ __forceinline__ double weight_at(const Lines<S> &l, int64_t i)
{
    double w = InTraits<In>::template one<double>(l.p[i]);
    if (l.q)
        w -= InTraits<In>::template one<double>(l.q[i]);
    return weight(i == l.x ? w - 1.0 : w);
}

// A lane's part of the sum of the tile at `base`, G vectors of a line in flight.
template <class In, bool FAST, int G, class S>
__device__ __forceinline__ double sum_of(const Lines<S> &l, int64_t n, int64_t base)
{
    constexpr int V = InTraits<In>::vec, U = kTile / (64 * V);
    static_assert(U % G == 0, "whole rounds");
    const S *lp = l.p + base, *lq = l.q ? l.q + base : nullptr;
    const int64_t left = n - base, x = l.x - base;
    double s = 0.0;
#pragma unroll 1
    for (int g = 0; g < U; g += G) {
        Loaded<In, FAST, S> v[G];
#pragma unroll
        for (int u = 0; u < G; ++u)
            v[u].load(lp, lq, ((g + u) * 64 + lane_id()) * V, left);
#pragma unroll
        for (int u = 0; u < G; ++u) {
            double w[V];
            v[u].weights(lq, ((g + u) * 64 + lane_id()) * V, left, x, w);
#pragma unroll
            for (int k = 0; k < V; ++k)
                s += w[k];
            issue_barrier();                  // one vector's float64 weights at a time: registers bound the waves
        }
    }
    return s;
}

// Sum of one tile's weights, in every lane of the wave.
template <class In, class S>
__device__ __forceinline__ double tile_sum(const Lines<S> &l, int64_t n, int64_t tile, bool fast)
{
    constexpr int U = kTile / (64 * InTraits<In>::vec);
    const int64_t base = tile * kTile;
    if (n < InTraits<In>::vec)
        return wave_reduce<OpSum>(lane_id() < n ? weight_at<In>(l, lane_id()) : 0.0);
    if (fast && base + kTile <= n && !(l.x >= base && l.x < base + kTile)) {
        const double s = wave_reduce<OpSum>(sum_of<In, true, U>(l, n, base));
        if (s < __builtin_inf())
            return s;
    }
    return wave_reduce<OpSum>(sum_of<In, false, U / 2>(l, n, base));
}

// The place that the first of a block's threads to have one names in `at`, and
// the last in `last` (kNowhere: none has).  A lane is picked by ballot and the
// waves meet in LDS (against LDS atomics of 64 lanes on one word, captured:
// 1 x 4 x 32768 f32 12.4 -> 8.3 us, 64 x 4 x 131072 20.7 -> 13.9).
struct Found {
    int at, last;
};
constexpr int kNowhere = -1;

struct FoundLds {
    int at[kB / 64], last[kB / 64];
};

__device__ __forceinline__ Found first_of(FoundLds &lds, int at, int last)
{
    const uint64_t ma = __ballot(at != kNowhere), ml = __ballot(last != kNowhere);
    if (lane_id() == 0) {
        lds.at[threadIdx.x >> 6] = ma ? read_lane(at, __builtin_ctzll(ma)) : kNowhere;
        lds.last[threadIdx.x >> 6] = ml ? read_lane(last, 63 - __builtin_clzll(ml)) : kNowhere;
    }
    __syncthreads();
    Found f{kNowhere, kNowhere};
#pragma unroll
    for (int i = 0; i < kB / 64; ++i) {
        f.at = f.at == kNowhere ? lds.at[i] : f.at;
        f.last = lds.last[i] != kNowhere ? lds.last[i] : f.last;
    }
    return f;
}

// The first index whose running sum passes r * (whole sum), -1 where nothing
// weighs anything.  Called by the whole block, with the tiles' sums in `sums`.
template <class In, class S>
__device__ __forceinline__ int64_t find(const Lines<S> &l, int64_t n, const double *sums, int64_t tiles, double r)
{
    constexpr int V = InTraits<In>::vec, per = kTile / kB;
    static_assert(per % V == 0, "whole vectors a thread");
    __shared__ double part[kB / 64];
    __shared__ FoundLds lds;
    // The whole sum, in the order of the running one, and the tile in which the
    // running sum passes: every wave for itself, four sums a lane, no barrier.
    constexpr int K = 4;
    double v[K], before = 0.0, whole = 0.0;
    const auto round = [&](int64_t base, double upto) {        // returns the running sum after it
        double mine = 0.0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t i = base + lane_id() * K + k;
            v[k] = i < tiles ? load_partial(sums + i) : 0.0;
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            mine += v[k];
        const double incl = wave_prefix(mine);
        before = upto + dpp_or_0<0x138, 0xf>(incl);            // wave_shr:1
        return upto + read_lane(incl, 63);
    };
    for (int64_t base = 0; base < tiles; base += 64 * K)
        whole = round(base, whole);
    if (!(whole > 0.0))
        return -1;
    const double bar = r * whole;
    int t = kNowhere, last = kNowhere;
    double start = -__builtin_inf(), upto = 0.0;
    for (int64_t base = 0; base < tiles && t == kNowhere; base += 64 * K) {
        if (tiles > 64 * K)                   // (otherwise the one round above has left v and before)
            upto = round(base, upto);
        int at = kNowhere, pos = kNowhere;
        double run = before, begin = 0.0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = int(base) + lane_id() * K + k;
            const double next = run + v[k];
            pos = v[k] > 0.0 ? i : pos;
            if (at == kNowhere && v[k] > 0.0 && next > bar) {
                at = i;
                begin = run;
            }
            run = next;
        }
        const uint64_t passes = __ballot(at != kNowhere), some = __ballot(pos != kNowhere);
        if (passes) {
            t = read_lane(at, __builtin_ctzll(passes));
            start = read_lane(begin, __builtin_ctzll(passes));
        }
        if (some)
            last = read_lane(pos, 63 - __builtin_clzll(some));
    }
    // none (r so near 1 that r * whole rounds to whole): the last entry that weighs something
    if (t == kNowhere)
        t = last;
    __syncthreads();                          // a second call's uses of LDS come after the first's
    // the entry
    const int64_t base = int64_t(wave_uniform(t)) * kTile, left = n - base;
    const int first = int(threadIdx.x) * per;
    double w[per], mine = 0.0;
    int off[per / V];                         // place of each vector's first entry in the tile
    if (n < V) {
#pragma unroll
        for (int k = 0; k < per; ++k)
            w[k] = first + k < n ? weight_at<In>(l, first + k) : 0.0;
#pragma unroll
        for (int u = 0; u < per / V; ++u)
            off[u] = first + u * V;
    } else {
        using L = Loaded<In, false, S>;
        const S *lp = l.p + base, *lq = l.q ? l.q + base : nullptr;
        L x[per / V];
#pragma unroll
        for (int u = 0; u < per / V; ++u)
            x[u].load(lp, lq, first + u * V, left);
#pragma unroll
        for (int u = 0; u < per / V; ++u) {
            x[u].weights(lq, first + u * V, left, l.x - base, w + u * V);
            off[u] = L::at(first + u * V, left);
        }
    }
#pragma unroll
    for (int k = 0; k < per; ++k)
        mine += w[k];
    double sum, run = start + block_prefix<kB>(mine, part, &sum);
    int at = kNowhere, pos = kNowhere;
#pragma unroll
    for (int k = 0; k < per; ++k) {
        run += w[k];
        const int place = off[k / V] + k % V;
        pos = w[k] > 0.0 ? place : pos;
        at = at == kNowhere && w[k] > 0.0 && run > bar ? place : at;
    }
    const Found entry = first_of(lds, at, pos);
    return int64_t(t) * kTile + (entry.at != kNowhere ? entry.at : entry.last);
}

template <class In, bool FAST, class S>
__device__ __forceinline__ void sum_tiles(const VerifyArgs &a, int64_t b, const Lines<S> &l, int64_t from, int64_t step)
{
    for (int64_t tile = from + wave_uniform(int(threadIdx.x >> 6)); tile < a.tiles; tile += step) {
        const double s = tile_sum<In>(l, a.n, tile, FAST);
        if (lane_id() == 0)
            store_partial(a.sums + b * a.tiles + tile, s);
    }
    wait_stores();
    __syncthreads();
}

// Draws the request's next token.
template <class In, class Tok>
__device__ __forceinline__ void finish(const VerifyArgs &a, int64_t b, const VerifyDrawn &d)
{
    using S = typename InTraits<In>::S;
    Lines<S> l = lines_of<S>(a, b, d);
    double r = double(a.r[b]);
    r = r > 0.0 ? (r < 1.0 ? r : 1.0) : 0.0;  // (NaN draws the first)
    const double *sums = a.sums + b * a.tiles;
    int64_t token = find<In>(l, a.n, sums, a.tiles, r);
    if (token < 0 && (l.q || l.x >= 0)) {     // the draft leaves nothing of the target: draw from the target
        // All waves have read the same sums, so all are here or none.  Each has read them for itself,
        // and none may still be doing so when they are written anew.
        __syncthreads();
        l.q = nullptr;
        l.x = -1;
        sum_tiles<In, false>(a, b, l, 0, kB / 64);
        token = find<In>(l, a.n, sums, a.tiles, r);
    }
    if (threadIdx.x == 0)
        static_cast<Tok *>(a.tokens)[b * (int64_t(a.max_draft) + 1) + d.kept] = Tok(token);
}

// What is known before the next token is: the kept tokens, how many they are,
// and -1 behind the next one.
template <class Tok>
__device__ __forceinline__ void write_kept(const VerifyArgs &a, int64_t b, const VerifyDrawn &d)
{
    Tok *out = static_cast<Tok *>(a.tokens) + b * (int64_t(a.max_draft) + 1);
    for (int i = int(threadIdx.x); i <= a.max_draft; i += kB)
        if (i != d.kept)
            out[i] = i < d.kept ? static_cast<const Tok *>(a.drafted)[d.lo + i] : Tok(-1);
    if (threadIdx.x == 0)
        a.accepted[b] = d.kept;
}

template <class In, class Tok>
__global__ __launch_bounds__(kB) void k_verify(VerifyArgs a)
{
    using S = typename InTraits<In>::S;
    const int64_t b = blockIdx.x / uint32_t(a.chunks);
    const int c = int(blockIdx.x % uint32_t(a.chunks));
    const VerifyDrawn d = accept<In, Tok>(a, b);
    const Lines<S> l = lines_of<S>(a, b, d);
    if (c == 0) {
        write_kept<Tok>(a, b, d);
        if (a.chunks > 1 && a.slot < 0 && threadIdx.x == 0)
            a.drawn[b] = d;                   // for the second launch
    }
    sum_tiles<In, true>(a, b, l, int64_t(c) * (kB / 64), int64_t(a.chunks) * (kB / 64));
    if (a.chunks > 1) {
        if (a.slot < 0)
            return;                           // the second launch finishes
        __shared__ bool last;
        if (threadIdx.x == 0)
            last = arrive_last(a.slot, b, uint32_t(c), uint32_t(a.chunks));
        __syncthreads();
        if (!last)
            return;
    }
    finish<In, Tok>(a, b, d);
}

template <class In, class Tok>
__global__ __launch_bounds__(kB) void k_verify_finish(VerifyArgs a)
{
    const int64_t b = blockIdx.x;
    finish<In, Tok>(a, b, a.drawn[b]);
}

template <class In, class Tok>
int run_verify(const VerifyLaunch &L)
{
    launch_timed(k_verify<In, Tok>, dim3(uint32_t(L.plan.grid)), dim3(kB), 0, L.stream, L.ev_begin, L.ev_end, L.a);
    if (L.a.chunks > 1 && L.a.slot < 0)
        launch_timed(k_verify_finish<In, Tok>, dim3(uint32_t(L.a.req)), dim3(kB), 0, L.stream, nullptr, nullptr, L.a);
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

template <class In>
int run_verify_in(const VerifyLaunch &L)
{
    return L.token_dtype == I64 ? run_verify<In, int64_t>(L) : run_verify<In, int32_t>(L);
}

}  // namespace

int launch_verify(const VerifyLaunch &L)
{
    switch (L.dtype) {
    case F32: return run_verify_in<float>(L);
    case BF16: return run_verify_in<bf16_in>(L);
    case F16: return run_verify_in<f16_in>(L);
    }
    return ST_UNSUPPORTED;
}

}  // namespace rk
