// rk_recur_kernels.hpp -- the gated linear recurrence and its backward pass.
//
// Forward, per channel:  h_t = a_t h_(t-1) + w_t x_t,  a the gate, w = 1 or
// 1 - a.  Backward:      g_t = d_t + u_(t+1),  u_t = a_t g_t  (d the gradient
// of the output, u what a token hands to the one before it).  Both are scans of
// affine maps s -> A s + H, the backward one from the last token to the first;
// "step" below is a token's number in the scan's order.  Two maps in a row are
// (A2 A1, A2 H1 + H2).
//
// Tiles of a strip of channels x consecutive steps, all of it in registers: a
// lane holds kRecurVec channels of R steps, neighbouring lanes the strip's
// channels (a row of a tile is whole 128-byte lines), the block's lane groups
// consecutive runs of steps.  A lane folds its steps, groups are folded by lane
// moves and through LDS, and the state that enters the tile comes from the
// tiles before it by decoupled look-back (Merrill and Garland, 2016), so every
// input is read once and every output written once.  The state goes on from
// the nearest tile whose outgoing state is known through the maps of the tiles
// between, in order: however far a tile has to look, it computes the same
// products and sums, so equal inputs give equal bits.
//
// A sequence's first step in the scan's order resets the state to the
// sequence's own; nothing of the maps before a reset is used, so neither an
// infinity nor a NaN passes from one sequence to the next, and a tile that holds
// a reset hands on its state without waiting.
//
// States, products of gates and sums are float32; outputs are rounded once.
#pragma once

#include "rk_host.hpp"
#include "rk_recur.hpp"
#include "rk_serve_device.hpp"

namespace rk {
namespace {

constexpr int kB = tune::kRecurBlock;
constexpr int kWaves = kB / 64;
constexpr int kStrip = tune::kRecurStrip;

// V elements of a row.
template <class T, int V> struct Pack {
    using S = typename InTraits<T>::S;
    static constexpr int NW = (V * int(sizeof(S)) + 3) / 4;
    using Raw = std::conditional_t<V == 1, S, typename Words<NW>::T>;

    __device__ __forceinline__ static Raw load(const S *p)
    {
        if constexpr (V == 1)
            return *p;
        else
            return Words<NW>::load(p);
    }
    __device__ __forceinline__ static void get(Raw r, float (&f)[V])
    {
        S s[V];
        __builtin_memcpy(s, &r, sizeof s);
#pragma unroll
        for (int i = 0; i < V; ++i)
            f[i] = InTraits<T>::template one<float>(s[i]);
    }
    __device__ __forceinline__ static S one(float v)
    {
        if constexpr (sizeof(S) == 4)
            return v;
        else if constexpr (std::is_same_v<T, bf16_in>)
            return bitcast<uint16_t>((__bf16)v);
        else
            return bitcast<uint16_t>((_Float16)v);
    }
    // the elements from `drop` on (the ones before belong to another lane)
    __device__ __forceinline__ static void store(S *p, const float (&f)[V], int drop)
    {
        S s[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            s[i] = one(f[i]);
        if constexpr (V == 1) {
            if (drop == 0)
                *p = s[0];
        } else if (drop == 0) {
            Words<NW>::template store<false>(p, words_of<NW>(s));
        } else {
#pragma unroll
            for (int i = 1; i < V; ++i)
                if (i >= drop)
                    p[i] = s[i];
        }
    }
};

// exp(t) to about an ulp: t log2(e) as a sum of two floats, the smaller one's
// power of two to first order.  (One float alone is off by |t| 2^-24.)
__device__ __forceinline__ float exp_of(float t)
{
    const float p = t * 1.44269502f;
    const float q = __builtin_fmaf(t, 1.44269502f, -p) + t * 1.92596303e-8f;   // log2(e) = 1.44269502f + 1.92596303e-8
    const float e = __builtin_amdgcn_exp2f(p);
    // (far out p is infinite and q a NaN, where e is 0 or inf already)
    return __builtin_fabsf(t) < 88.0f ? __builtin_fmaf(e, q * 0.693147182f, e) : e;
}

// a and 1 - a of a gate, the difference without cancellation where the gate is
// given by its logarithm or logit.
template <int KIND, bool WANT_W>
__device__ __forceinline__ void gate_of(float g, float &a, float &w)
{
    if constexpr (KIND == RECUR_SIGMOID) {
        const float e = exp_of(-__builtin_fabsf(g)), r = __builtin_amdgcn_rcpf(1.0f + e), f = e * r;
        const bool up = g >= 0.0f;
        a = up ? r : f;
        w = up ? f : r;
    } else if constexpr (KIND == RECUR_LOG) {
        a = exp_of(g);
        w = 1.0f - a;
        if constexpr (WANT_W) {
            // exp(g) - 1 = g (1 + g/2 (1 + g/3 (1 + ...))): to 2^-25 of it below 1/4 with eight terms
            float s = 1.0f + g * 0.125f;
            s = 1.0f + g * (1.0f / 7.0f) * s;
            s = 1.0f + g * (1.0f / 6.0f) * s;
            s = 1.0f + g * 0.2f * s;
            s = 1.0f + g * 0.25f * s;
            s = 1.0f + g * (1.0f / 3.0f) * s;
            s = 1.0f + g * 0.5f * s;
            w = __builtin_fabsf(g) < 0.25f ? -g * s : w;
        }
    } else {
        a = g;
        w = 1.0f - g;
    }
}

// A s + H; from a state of 0 it is H, whatever became of A (a product of gates
// may pass float32's range where every state is finite).
__device__ __forceinline__ float apply(float A, float s, float H) { return s == 0.0f ? H : __builtin_fmaf(A, s, H); }

constexpr uint32_t kIn = 1, kReset = 2, kEnd = 4;   // of a step: in a sequence, its first, its last in the scan's order

// The sequence of a row (-1: none) and the row's flags.
template <bool BWD>
__device__ __forceinline__ int32_t sequence_of(const RecurArgs &a, int64_t seg, int64_t row, uint32_t *flag)
{
    int64_t b, lo, hi;
    if (a.starts) {
        b = last_start([&](int i) { return int64_t(a.starts[i]); }, 0, int(a.n_seq), row);
        lo = a.starts[b];
        hi = a.starts[b + 1];
        lo = lo < 0 ? 0 : lo;
        hi = hi > a.rows ? a.rows : hi;
        if (row < lo || row >= hi) {
            *flag = 0;
            return -1;
        }
    } else {
        const int64_t i = divide(uint32_t(row), a.period);
        lo = i * a.period.d;
        hi = lo + a.period.d;
        b = a.segs > 1 ? seg : i;
    }
    const bool first = row == lo, last = row == hi - 1;
    *flag = kIn | ((BWD ? last : first) ? kReset : 0) | ((BWD ? first : last) ? kEnd : 0);
    return int32_t(b);
}

// The state a sequence starts from, channels c .. c + V - 1.
template <int V>
__device__ __forceinline__ void first_state(const RecurArgs &a, int64_t b, int64_t c, float (&s)[V])
{
    const int64_t i = a.sources ? a.sources[b] : b;
    const bool there = a.state && i >= 0 && i < a.n_states;
#pragma unroll
    for (int k = 0; k < V; ++k)
        s[k] = there ? a.state[i * a.channels + c + k] : 0.0f;
}

template <int V>
__device__ __forceinline__ void last_gradient(const RecurArgs &a, int64_t b, int64_t c, float (&s)[V])
{
#pragma unroll
    for (int k = 0; k < V; ++k)
        s[k] = a.dlast ? a.dlast[b * a.channels + c + k] : 0.0f;
}

struct RecurRecord {
    char *at;
    __device__ RecurRecord(const RecurArgs &a, int64_t col, int64_t tile)
        : at(reinterpret_cast<char *>(a.ws) + kRecurHeaderBytes + (col * a.tiles + tile) * kRecurRecBytes) {}
    __device__ uint32_t *flag() const { return reinterpret_cast<uint32_t *>(at); }
    __device__ float *factor(int c) const { return reinterpret_cast<float *>(at + 128) + c; }
    __device__ float *addend(int c) const { return reinterpret_cast<float *>(at + 128) + kStrip + c; }
    __device__ float *after(int c) const { return reinterpret_cast<float *>(at + 128) + 2 * kStrip + c; }
};
constexpr uint32_t kMapKnown = 1, kStateKnown = 2;

__device__ __forceinline__ void publish(const RecurRecord &r, uint32_t flag)
{
    wait_stores();                            // the wave's values first
    if (lane_id() == 0)
        __hip_atomic_store(r.flag(), flag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that enters tile `tile`, channel c = this lane's, run by one whole
// wave.  Every tile with a smaller number has started (tiles are numbered in
// the order blocks start) and makes its map known without waiting; the first
// one that has no state yet has a tile with one right before it, so a window
// of 64 tiles always comes to hold a state with maps only behind it and the
// wait ends.  It is bounded all the same: past the bound it is counted and the
// wave goes on.
__device__ __forceinline__ float look_back(const RecurArgs &a, int64_t col, int64_t tile, int c)
{
    const int lane = lane_id();
    const int64_t j = tile - 1 - lane;
    uint64_t known;
    for (uint32_t spin = 0;; ++spin) {
        const uint32_t f = j >= 0 ? __hip_atomic_load(RecurRecord(a, col, j).flag(), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                                  : 0u;
        known = __ballot(f == kStateKnown);
        const uint64_t nothing = __ballot(f == 0);
        if (known && (nothing & ((known & (0 - known)) - 1)) == 0 && !a.force_wait)
            break;
        if (spin >= a.spin_limit) {
            if (lane == 0)
                record_timeout(-1);
            return 0.0f;
        }
        __builtin_amdgcn_s_sleep(1);
    }
    const int first = __builtin_ctzll(known);
    float s = load_partial(RecurRecord(a, col, tile - 1 - first).after(c));
    for (int i = first - 1; i >= 0; i -= 8) {
        float A[8], H[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const RecurRecord r(a, col, tile - 1 - (i - k > 0 ? i - k : 0));
            A[k] = load_partial(r.factor(c));
            H[k] = load_partial(r.addend(c));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s = i - k >= 0 ? apply(A[k], s, H[k]) : s;
    }
    return s;
}

// The last states (backward: the first states' gradients) of sequences
// without tokens, dealt to the grid's blocks.
template <bool BWD>
__device__ __forceinline__ void empty_sequences(const RecurArgs &a)
{
    if (!a.state_out)
        return;
    for (int64_t b = blockIdx.x; b < a.n_seq; b += gridDim.x) {
        if (a.starts) {
            const int64_t lo = a.starts[b] < 0 ? 0 : a.starts[b], hi = a.starts[b + 1];
            if (lo < (hi > a.rows ? a.rows : hi))
                continue;
        }
        for (int64_t c = threadIdx.x; c < a.channels; c += kB) {
            float s[1];
            if constexpr (BWD)
                last_gradient(a, b, c, s);
            else
                first_state(a, b, c, s);
            a.state_out[b * a.channels + c] = s[0];
        }
    }
}

template <bool BWD>
__global__ __launch_bounds__(kB) void k_recur_empty(RecurArgs a)
{
    empty_sequences<BWD>(a);
}

// Zero the tile counter and the flags.
__global__ __launch_bounds__(kB) void k_recur_clear(RecurArgs a, int64_t recs)
{
    const int64_t i = int64_t(blockIdx.x) * kB + threadIdx.x;
    if (i == 0)
        a.ws[0] = 0;
    if (i < recs)
        *RecurRecord(a, 0, i).flag() = 0;
}

template <class T>
__device__ __forceinline__ const typename InTraits<T>::S *row_at(const RecurTensor &t, int64_t seg, int64_t row, int64_t c)
{
    return static_cast<const typename InTraits<T>::S *>(t.p) + seg * t.bs + row * t.ts + c;
}

template <class X, class G, int V, int R, bool BWD>
__global__ __launch_bounds__(kB, 2) void k_recur(RecurArgs a)
{
    using PX = Pack<X, V>;
    using PG = Pack<G, V>;
    using XS = typename PX::S;
    using GS = typename PG::S;
    __shared__ uint32_t s_id;
    __shared__ __attribute__((aligned(16))) uint8_t s_flag[kB * R];
    __shared__ int32_t s_seq[kB * R];
    __shared__ float s_A[kWaves][kStrip], s_H[kWaves][kStrip], s_in[kStrip];
    __shared__ int s_reset[kWaves];

    const int tid = int(threadIdx.x), lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int LC = 1 << a.lanes_log2;
    uint32_t id = blockIdx.x;
    if (a.linked) {
        if (tid == 0)
            s_id = __hip_atomic_fetch_add(a.ws, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        id = __builtin_amdgcn_readfirstlane(s_id);
        if (id >= gridDim.x)                   // never: the counter starts at zero
            return;
    }
    const uint32_t cols = uint32_t(a.strips) * uint32_t(a.segs);
    const int64_t tile = id / cols;
    const uint32_t col = id % cols;
    const int64_t seg = col / uint32_t(a.strips);
    const int64_t cl = int64_t(col % uint32_t(a.strips)) * (LC * V) + (tid & (LC - 1)) * V;
    // a lane that would pass the last channel takes the last V ones and drops those that are not its own
    const int64_t c0 = cl + V <= a.channels ? cl : a.channels - V;
    const int drop = cl - c0 < V ? int(cl - c0) : V;
    const int64_t tile0 = tile * a.tile_rows, tile_end = tile0 + a.tile_rows < a.rows ? tile0 + a.tile_rows : a.rows;
    const int r0 = (tid >> a.lanes_log2) * R;

    // rows of this lane's steps, kept inside the tile
    auto row_of = [&](int r) {
        int64_t s = tile0 + r0 + r;
        s = s < tile_end ? s : tile_end - 1;
        return BWD ? a.rows - 1 - s : s;
    };
    typename PG::Raw gate[R];
    typename PX::Raw x[R], d[BWD ? R : 1], h[BWD ? R : 1];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = row_of(r);
        gate[r] = PG::load(row_at<G>(a.gate, seg, row, c0));
        if constexpr (BWD) {
            d[r] = PX::load(row_at<X>(a.dout, seg, row, c0));
            h[r] = PX::load(row_at<X>(a.h, seg, row > 0 ? row - 1 : 0, c0));
            if (a.blend)
                x[r] = PX::load(row_at<X>(a.x, seg, row, c0));
            else
                x[r] = typename PX::Raw{};
        } else {
            x[r] = PX::load(row_at<X>(a.x, seg, row, c0));
        }
    }
    issue_barrier();
    for (int i = tid; i < (kB >> a.lanes_log2) * R; i += kB) {
        const int64_t s = tile0 + i;
        uint32_t f = 0;
        int32_t b = -1;
        if (s < tile_end)
            b = sequence_of<BWD>(a, seg, BWD ? a.rows - 1 - s : s, &f);
        s_flag[i] = uint8_t(f);
        s_seq[i] = b;
    }
    __syncthreads();
    uint8_t flag[R];
    __builtin_memcpy(flag, __builtin_assume_aligned(s_flag + r0, R), R);

    float A[V], H[V], start[V];
    bool reset = false;
    int last_reset = -1;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        A[k] = 1.0f;
        H[k] = 0.0f;
        start[k] = 0.0f;
    }
    auto reset_value = [&](int r, float (&s)[V]) {
        if constexpr (BWD)
            last_gradient(a, s_seq[r0 + r], c0, s);
        else
            first_state(a, s_seq[r0 + r], c0, s);
    };
    // the lane's map, from state 0; `start`: the state of its last reset, not read again where the
    // sequence's last state may take its place
    auto fold = [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = flag[r] & kIn;
            float g[V], v[V];
            PG::get(gate[r], g);
            if constexpr (BWD)
                PX::get(d[r], v);
            else
                PX::get(x[r], v);
            if (flag[r] & kReset) {
                reset = true;
                last_reset = r;
                reset_value(r, start);
#pragma unroll
                for (int k = 0; k < V; ++k)
                    H[k] = start[k];
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float ak, wk;
                gate_of<KIND, !BWD>(g[k], ak, wk);
                if constexpr (BWD)
                    H[k] = in ? ak * (v[k] + H[k]) : H[k];
                else
                    H[k] = in ? __builtin_fmaf(ak, H[k], a.blend ? wk * v[k] : v[k]) : H[k];
                A[k] = in ? A[k] * ak : A[k];
            }
        }
    };
    if (a.kind == RECUR_SIGMOID)
        fold(std::integral_constant<int, RECUR_SIGMOID>{});
    else if (a.kind == RECUR_LOG)
        fold(std::integral_constant<int, RECUR_LOG>{});
    else
        fold(std::integral_constant<int, RECUR_VALUE>{});

    // maps of the groups up to this one in the wave, then of those before it
    for (int dist = LC; dist < 64; dist <<= 1) {
        const int from = lane >= dist ? lane - dist : lane;
        const bool pr = bpermute32(reset, from);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float pA = bitcast<float>(bpermute32(bitcast<uint32_t>(A[k]), from));
            const float pH = bitcast<float>(bpermute32(bitcast<uint32_t>(H[k]), from));
            const bool use = lane >= dist && !reset;
            H[k] = use ? apply(A[k], pH, H[k]) : H[k];
            A[k] = use ? A[k] * pA : A[k];
        }
        reset = reset || (lane >= dist && pr);
    }
    if (lane >= 64 - LC) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            s_A[wave][(tid & (LC - 1)) * V + k] = A[k];
            s_H[wave][(tid & (LC - 1)) * V + k] = H[k];
        }
        if (lane == 63)
            s_reset[wave] = reset;
    }
    bool before_reset = bpermute32(reset, lane >= LC ? lane - LC : lane);
    before_reset = lane >= LC && before_reset;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int from = lane >= LC ? lane - LC : lane;
        const float pA = bitcast<float>(bpermute32(bitcast<uint32_t>(A[k]), from));
        const float pH = bitcast<float>(bpermute32(bitcast<uint32_t>(H[k]), from));
        A[k] = lane >= LC ? pA : 1.0f;
        H[k] = lane >= LC ? pH : 0.0f;
    }
    __syncthreads();
    if (a.linked) {
        if (wave == 0) {
            const int c = lane < LC * V ? lane : LC * V - 1;
            float tA = s_A[0][c], tH = s_H[0][c];
            bool tr = s_reset[0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) {
                const bool r = s_reset[w];
                tH = r ? s_H[w][c] : apply(s_A[w][c], tH, s_H[w][c]);
                tA *= s_A[w][c];
                tr = tr || r;
            }
            const RecurRecord rec(a, col, tile);
            const bool known = tr || tile == 0, behind = tile + 1 < a.tiles;
            if (behind) {
                if (known) {
                    store_partial(rec.after(c), tH);
                } else {
                    store_partial(rec.factor(c), tA);
                    store_partial(rec.addend(c), tH);
                }
                publish(rec, known ? kStateKnown : kMapKnown);
            }
            float s = 0.0f;
            if (tile > 0 && !(s_flag[0] & kReset)) {
                s = look_back(a, col, tile, c);
                if (behind && !known) {
                    store_partial(rec.after(c), apply(tA, s, tH));
                    publish(rec, kStateKnown);
                }
            }
            if (lane < LC * V)
                s_in[c] = s;
        }
        __syncthreads();
    }
    // the state that enters this lane's steps
    float s[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = (tid & (LC - 1)) * V + k;
        s[k] = a.linked ? s_in[c] : 0.0f;
        for (int w = 0; w < wave; ++w)
            s[k] = s_reset[w] ? s_H[w][c] : apply(s_A[w][c], s[k], s_H[w][c]);
        s[k] = before_reset ? H[k] : apply(A[k], s[k], H[k]);
    }

    auto finish = [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float g[V], v[V];
            PG::get(gate[r], g);
            if (flag[r] & kReset) {
                if (r == last_reset) {
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        s[k] = start[k];
                } else {
                    reset_value(r, s);
                }
            }
            const int64_t row = row_of(r);
            if constexpr (BWD) {
                float dv[V], hv[V], dx[V], dg[V];
                PX::get(d[r], dv);
                PX::get(h[r], hv);
                PX::get(x[r], v);
                if (flag[r] & kEnd)
                    first_state(a, s_seq[r0 + r], c0, hv);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float ak, wk;
                    gate_of<KIND, true>(g[k], ak, wk);
                    const float gr = dv[k] + s[k];
                    dx[k] = a.blend ? wk * gr : gr;
                    const float da = a.blend ? gr * (hv[k] - v[k]) : gr * hv[k];
                    dg[k] = KIND == RECUR_SIGMOID ? da * (ak * wk) : KIND == RECUR_LOG ? da * ak : da;
                    s[k] = (flag[r] & kIn) ? ak * gr : s[k];
                }
                if (flag[r] & kIn) {
                    PX::store(const_cast<XS *>(row_at<X>(a.out, seg, row, c0)), dx, drop);
                    PG::store(const_cast<GS *>(row_at<G>(a.dgate, seg, row, c0)), dg, drop);
                }
            } else {
                PX::get(x[r], v);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float ak, wk;
                    gate_of<KIND, true>(g[k], ak, wk);
                    const float n = __builtin_fmaf(ak, s[k], a.blend ? wk * v[k] : v[k]);
                    s[k] = (flag[r] & kIn) ? n : s[k];
                }
                if (flag[r] & kIn)
                    PX::store(const_cast<XS *>(row_at<X>(a.out, seg, row, c0)), s, drop);
            }
            if ((flag[r] & kEnd) && a.state_out) {
                float *p = a.state_out + int64_t(s_seq[r0 + r]) * a.channels + c0;
                Pack<float, V>::store(p, s, drop);
            }
        }
    };
    if (a.kind == RECUR_SIGMOID)
        finish(std::integral_constant<int, RECUR_SIGMOID>{});
    else if (a.kind == RECUR_LOG)
        finish(std::integral_constant<int, RECUR_LOG>{});
    else
        finish(std::integral_constant<int, RECUR_VALUE>{});
    if (a.starts)
        empty_sequences<BWD>(a);
}

template <class X, class G, int V, int R, bool BWD>
int launch_one(const RecurLaunch &L)
{
    launch_timed(k_recur<X, G, V, R, BWD>, dim3(uint32_t(L.plan.grid)), dim3(kB), 0, L.stream,
                 L.ev_begin, L.ev_end, L.a);
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

template <class X, class G, bool BWD>
int launch_recur(const RecurLaunch &L)
{
    const RecurPlan &p = L.plan;
    if (p.tiles == 0) {                        // sequences without tokens only
        const int64_t most = 1024;
        launch_timed(k_recur_empty<BWD>, dim3(uint32_t(L.a.n_seq < most ? L.a.n_seq : most)), dim3(kB), 0, L.stream,
                     L.ev_begin, L.ev_end, L.a);
        return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
    }
    if (p.linked) {
        const int64_t recs = p.grid;
        hipLaunchKernelGGL(k_recur_clear, dim3(uint32_t((recs + kB - 1) / kB)), dim3(kB), 0,
                           static_cast<hipStream_t>(L.stream), L.a, recs);
        if (hipGetLastError() != hipSuccess)
            return ST_HIP;
    }
    if (p.vec == 1)
        return p.per_lane == 1 ? launch_one<X, G, 1, 1, BWD>(L) : launch_one<X, G, 1, 4, BWD>(L);
    constexpr int R = recur_rows(sizeof(typename InTraits<X>::S), sizeof(typename InTraits<G>::S), BWD);
    static_assert(R == (BWD && std::is_same_v<G, float> ? 8 : 16), "the plan's tokens of a lane");
    switch (p.per_lane) {
    case 1: return launch_one<X, G, 4, 1, BWD>(L);
    case 4: return launch_one<X, G, 4, 4, BWD>(L);
    default: return launch_one<X, G, 4, R, BWD>(L);
    }
}

template <class X>
int launch_recur_x(const RecurLaunch &L)
{
    if (L.gate_dtype == F32)
        return L.backward ? launch_recur<X, float, true>(L) : launch_recur<X, float, false>(L);
    if constexpr (!std::is_same_v<X, float>)
        return L.backward ? launch_recur<X, X, true>(L) : launch_recur<X, X, false>(L);
    return ST_UNSUPPORTED;
}

inline int take_recur_timeouts(uint64_t *count)
{
    uint32_t n = 0;
    const uint32_t zero = 0;
    const size_t at = size_t(kArriveSlots) * 4;
    if (hipMemcpyFromSymbol(&n, HIP_SYMBOL(g_timeouts), 4, at, hipMemcpyDeviceToHost) != hipSuccess)
        return ST_HIP;
    if (n && hipMemcpyToSymbol(HIP_SYMBOL(g_timeouts), &zero, 4, at, hipMemcpyHostToDevice) != hipSuccess)
        return ST_HIP;
    *count += n;
    return ST_OK;
}

}  // namespace
}  // namespace rk
