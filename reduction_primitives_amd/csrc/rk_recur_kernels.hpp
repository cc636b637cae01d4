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
// Nothing depends on the order in which blocks start: one that would wait for a
// tile that no block has begun computes that tile's map itself.
//
// States, products of gates and sums are float32; outputs are rounded once.
//
// Measured, us a call, 2048 channels of bf16 unless said: 512 x 128 tokens, where no tile
// waits, 167 forward (805 MB, 4.8 TB/s) and 512 x 64 backward 173 (as many bytes); 16 x
// 4096 forward 207, 4 x 16384 204, 1 x 65536 247 (3.3 TB/s), 8 x 4096 109, 1 x 4096 21, 37
// sequences packed in 20011 tokens 87; 8 x 4096 backward 197, 20011 x 1001 float32 packed
// 138.  What the tiles wait for each other is what is left, and 5 to 7 us of clearing the
// records: four blocks a CU hide a load's latency but not that as well, and a fifth has no
// registers (40 spilled).  (Blocks that go from tile to tile with the next one's inputs loaded
// ahead took 337 us for 1 x 65536: three blocks a CU then, and loads that come back in
// order behind the look-back's.  The other three waves loading the 12 records before the
// nearest four while the first polls: 258 us, for the traffic.)
#pragma once

#include "rk_recur.hpp"
#include "rk_serve_device.hpp"

namespace rk {
namespace {

constexpr int kB = tune::kRecurBlock;
constexpr int kWaves = kB / 64;
constexpr int kStrip = tune::kRecurStrip;

// What is decoded from `raw` before and after this is not the same to the
// compiler, which would otherwise keep the decoded values, two or four times as
// many registers, in place of the raw ones.
template <class T>
__device__ __forceinline__ void decode_anew(T &raw)
{
    if constexpr (sizeof(T) >= 4) {
        asm volatile("" : "+v"(raw));
    } else {
        uint32_t w = raw;
        asm volatile("" : "+v"(w));
        raw = T(w);
    }
}

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

constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596303e-8f;   // log2(e) as a sum of two floats

// exp(t) from its power of two.  A product t log2(e) of one float is off by
// |t| 2^-24: enough for gates of 16 bits (FINE false), where t itself stands for
// all within half of its last place; else the rest of the product is made good to
// first order.
template <bool FINE>
__device__ __forceinline__ float mend_exp(float e, float t, float p)
{
    if constexpr (!FINE)
        return e;
    const float q = __builtin_fmaf(t, kLog2e, -p) + t * kLog2eRest;
    return __builtin_fabsf(t) < 88.0f ? __builtin_fmaf(e, q * 0.693147182f, e) : e;   // (farther out q may be a NaN)
}

// a and 1 - a of a gate, the difference without cancellation where the gate is
// given by its logarithm or logit.
template <int KIND, bool FINE, bool WANT_W>
__device__ __forceinline__ void gate_of(float g, float &a, float &w)
{
    if constexpr (KIND == RECUR_SIGMOID) {
        // a = 1 / (1 + e), 1 - a = e a with e = exp(-g), kept finite (a NaN stays one)
        const float p = -g * kLog2e;
        const float e = mend_exp<FINE>(__builtin_amdgcn_exp2f(__builtin_elementwise_minimum(p, 126.0f)), -g, p);
        a = __builtin_amdgcn_rcpf(1.0f + e);
        w = e * a;
    } else if constexpr (KIND == RECUR_LOG) {
        const float p = g * kLog2e;
        a = mend_exp<FINE>(__builtin_amdgcn_exp2f(p), g, p);
        w = 1.0f - a;
        if constexpr (WANT_W) {
            // 1 - exp(g) = -g (1 + g/2 (1 + g/3 (1 + ...))): to 2^-25 of it below 1/4 with eight terms
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

// A tile's record: per channel two words of a float and a tag that says what it
// is.  The tag travels with its value, so nobody waits for a store to arrive
// before a flag.  Word 0: the map's addend, then the state behind the tile; word
// 1: the map's factor.
constexpr uint32_t kMapKnown = 1, kStateKnown = 2;

struct RecurRecord {
    uint64_t *at;
    __device__ RecurRecord(const RecurArgs &a, int64_t col, int64_t tile)
        : at(reinterpret_cast<uint64_t *>(a.ws) + (col * a.tiles + tile) * (2 * kStrip)) {}
    __device__ __forceinline__ void put(int word, int c, float v, uint32_t tag) const
    {
        __hip_atomic_store(at + word * kStrip + c, uint64_t(tag) << 32 | bitcast<uint32_t>(v), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    }
    // where nothing is known yet: what the tile's own block puts later is the same, or its state
    __device__ __forceinline__ void offer(int word, int c, float v, uint32_t tag) const
    {
        uint64_t nothing = 0;
        __hip_atomic_compare_exchange_strong(at + word * kStrip + c, &nothing, uint64_t(tag) << 32 | bitcast<uint32_t>(v),
                                             __ATOMIC_RELAXED, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ uint64_t get(int word, int c) const
    {
        return __hip_atomic_load(at + word * kStrip + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
};

__device__ __forceinline__ uint32_t tag_of(uint64_t w) { return uint32_t(w >> 32); }
__device__ __forceinline__ float value_of(uint64_t w) { return bitcast<float>(uint32_t(w)); }

// kRecurBatch consecutive records' words of a channel, the first of them `i` tiles
// before the one whose state is wanted.  (Records of a column lie one after the
// other, so a batch takes one address; it may reach that tile's own and the next
// ones, whose words are not looked at.)
struct RecordBatch {
    static constexpr int N = kRecurBatch;
    uint64_t A[N], H[N];

    __device__ __forceinline__ void load(const RecurRecord &r, int c)
    {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            H[k] = r.get(2 * k, c);
            A[k] = r.get(2 * k + 1, c);
        }
    }
    // whether every lane has all words of the records `from` to i - 1, and of number `state` the state (a tile's words
    // of different channels lie in different lines, and the state of one may be seen while another's is on its way)
    __device__ __forceinline__ bool there(int i, int from = 0, int state = -1) const
    {
        bool t = true;
#pragma unroll
        for (int k = 0; k < N; ++k)
            t = t && (k >= i || k < from || tag_of(H[k]) == kStateKnown ||
                      (k != state && tag_of(H[k]) == kMapKnown && tag_of(A[k]) == kMapKnown));
        return __ballot(!t) == 0;
    }
    // the state behind them (where a tile's state has taken its addend's place, the same state)
    __device__ __forceinline__ float go_on(float s, int i) const
    {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < i)
                s = tag_of(H[k]) == kStateKnown ? value_of(H[k]) : apply(value_of(A[k]), s, value_of(H[k]));
        return s;
    }
};

// The state that enters tile `tile`, channel c = this lane's, run by one whole
// wave: from the nearest tile whose state is known through the maps of those
// behind it, in order.  Every tile makes its map known without waiting, and a
// column's first tile its state, so this comes to an end once the blocks of the
// tiles between have started.  They start in the order of their numbers as far as
// the device goes by these, which nothing depends on: where a map is missing after
// a.patience polls, *missing is its tile, whose map the waiting block computes
// itself (else -1); one that has done so before (helped) waits for the next one no
// longer than a tile under way takes.  a.force_help: every block asks for it once (a
// test's).  *back: 0, or how far the state is where that is more than a batch, which
// is the whole block's to gather.
__device__ __forceinline__ float look_back(const RecurArgs &a, int64_t col, int64_t tile, int c, bool helped,
                                           int64_t *missing, int64_t *back)
{
    constexpr int N = RecordBatch::N;
    const int near = tile < N ? int(tile) : N;
    RecordBatch b;
    const bool force = a.force_help && !helped;
    uint32_t polls = helped ? a.patience - tune::kRecurPatienceAgain : 0;
    *missing = -1;
    *back = 0;
    for (int64_t first = tile - 1;;) {         // 64 tiles from `first` down: what channel 0 knows of them
        const int64_t j = first - lane_id();
        const uint32_t f = j >= 0 ? tag_of(RecurRecord(a, col, j).get(0, 0)) : kMapKnown;
        b.load(RecurRecord(a, col, tile - near), c);   // and all words of the nearest ones
        const uint64_t known = __ballot(f == kStateKnown), nothing = __ballot(f == 0);
        if (force || (nothing && polls >= a.patience)) {
            *missing = force ? tile - 1 : first - __builtin_ctzll(nothing);
            return 0.0f;
        }
        if (known && (nothing & ((known & (0 - known)) - 1)) == 0) {
            const int64_t i = tile - first + __builtin_ctzll(known);
            if (i > near) {
                *back = i;
                return 0.0f;
            }
            if (b.there(near, near - int(i), near - int(i)))
                return b.go_on(0.0f, near);    // (what comes before the known state falls to it)
        } else if (!nothing) {
            first -= 64;                       // maps only: the tiles before them
            continue;
        }
        ++polls;
        __builtin_amdgcn_s_sleep(1);
    }
}

// The maps of `count` <= kAhead records from tile `from` on, a few from every
// wave, to LDS: addend and factor, the factor kTaken for a state.  first: the first
// one's state.
constexpr int kAhead = 2 * kRecurBatch * kWaves;
constexpr uint32_t kTaken = 0x7fc0dead;        // (a NaN that a product of gates is not without its addend being one)

__device__ __forceinline__ void gather_maps(const RecurArgs &a, int64_t col, int64_t from, int count, bool first, int wave, int c,
                                            float2 (*maps)[kStrip])
{
    constexpr int N = RecordBatch::N;
#pragma unroll 1
    for (int i = wave * N; i < count; i += kWaves * N) {
        const int n = count - i < N ? count - i : N;
        RecordBatch b;
        while (b.load(RecurRecord(a, col, from + i), c), !b.there(n, 0, first && i == 0 ? 0 : -1))
            __builtin_amdgcn_s_sleep(1);       // (words of channels beside the first are on their way)
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < n)
                maps[i + k][c] = make_float2(value_of(b.H[k]), tag_of(b.H[k]) == kStateKnown ? bitcast<float>(kTaken) : value_of(b.A[k]));
    }
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

// Zero the records, and copy n first states to where the tiles read them.
__global__ __launch_bounds__(kB) void k_recur_clear(RecurArgs a, int64_t vectors, const float *state, float *kept, int64_t n)
{
    for (int64_t i = int64_t(blockIdx.x) * kB + threadIdx.x; i < vectors; i += int64_t(gridDim.x) * kB)
        reinterpret_cast<u32x4 *>(a.ws)[i] = u32x4{0, 0, 0, 0};
    for (int64_t i = int64_t(blockIdx.x) * kB + threadIdx.x; i < n; i += int64_t(gridDim.x) * kB)
        kept[i] = state[i];
}

// Where a lane stands in a tile.
template <int V, int R, bool BWD>
struct Place {
    int64_t seg, c0, tile0, tile_end, row0;
    int drop, more;
    bool whole;

    __device__ __forceinline__ Place(const RecurArgs &a, int64_t tile, uint32_t col, int tid)
    {
        const int LC = 1 << a.lanes_log2, rows = (kB >> a.lanes_log2) * R;
        seg = col / uint32_t(a.strips);
        const int64_t cl = int64_t(col % uint32_t(a.strips)) * (LC * V) + (tid & (LC - 1)) * V;
        // a lane that would pass the last channel takes the last V ones and drops those that are not its own
        c0 = cl + V <= a.channels ? cl : a.channels - V;
        drop = cl - c0 < V ? int(cl - c0) : V;
        tile0 = tile * a.tile_rows;
        tile_end = tile0 + a.tile_rows < a.rows ? tile0 + a.tile_rows : a.rows;
        // The lane's first row, and how many follow it in the tile (in the scan's direction); lanes behind the
        // tile's end stay on its last row.
        const int r0 = (tid >> a.lanes_log2) * R;
        const int64_t step = tile0 + r0 < tile_end ? tile0 + r0 : tile_end - 1;
        row0 = BWD ? a.rows - 1 - step : step;
        more = tile_end - 1 - step < R - 1 ? int(tile_end - 1 - step) : R - 1;
        // (backward: the last tile reaches row 0, which has no row before it)
        whole = tile0 + rows <= tile_end && (!BWD || tile_end < a.rows);
    }
    // the lane's first element of a tensor
    template <class T>
    __device__ __forceinline__ typename InTraits<T>::S *at(const RecurTensor &t) const
    {
        return static_cast<typename InTraits<T>::S *>(const_cast<void *>(t.p)) + seg * t.bs + row0 * t.ts + c0;
    }
};

// A lane's place in a tensor, a row further with each step.  (The stride is opaque:
// its multiples, held for every row and tensor, are more scalars than there are, and
// those that do not fit went to and from vector registers, 200 instructions a tile.)
template <class T, bool BWD>
struct Rows {
    using S = typename InTraits<T>::S;
    S *p;
    int64_t by;
    __device__ __forceinline__ Rows(S *first, int64_t ts) : p(first), by(BWD ? -ts : ts) { asm volatile("" : "+s"(by)); }
    __device__ __forceinline__ void next() { p += by; }
    __device__ __forceinline__ void next_if(bool more) { p += more ? by : 0; }
};

// A lane's inputs as they come from memory.
template <class X, class G, bool BLEND, int V, int R, bool BWD>
struct Inputs {
    using PX = Pack<X, V>;
    using PG = Pack<G, V>;
    static constexpr bool HAS_X = !BWD || BLEND;
    typename PG::Raw gate[R];
    typename PX::Raw x[HAS_X ? R : 1], d[BWD ? R : 1], h[BWD ? R : 1];

    template <bool CLAMP>
    __device__ __forceinline__ void load_rows(const RecurArgs &a, const Place<V, R, BWD> &p)
    {
        Rows<G, BWD> gate_p(p.template at<G>(a.gate), a.gate.ts);
        Rows<X, BWD> x_p(p.template at<X>(a.x), a.x.ts), d_p(p.template at<X>(a.dout), a.dout.ts), h_p(p.template at<X>(a.h), a.h.ts);
        if constexpr (BWD)
            h_p.next_if(!CLAMP || p.row0 > 0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            gate[r] = PG::load(gate_p.p);
            if constexpr (HAS_X)
                x[r] = PX::load(x_p.p);
            if constexpr (BWD) {
                d[r] = PX::load(d_p.p);
                h[r] = PX::load(h_p.p);
            }
            if (r + 1 < R) {
                const bool more = !CLAMP || r < p.more;
                gate_p.next_if(more);
                if constexpr (HAS_X)
                    x_p.next_if(more);
                if constexpr (BWD) {
                    d_p.next_if(more);
                    h_p.next_if(!CLAMP || (more && r + 2 <= p.row0));
                }
            }
        }
    }
    __device__ __forceinline__ void load(const RecurArgs &a, const Place<V, R, BWD> &p)
    {
        if (p.whole)
            load_rows<false>(a, p);
        else
            load_rows<true>(a, p);
    }
};

// The kernel's arguments, read again: held from one end of it to the other they are more
// scalars than there are, and go to vector registers and back.
__device__ __forceinline__ const RecurArgs &args_again()
{
    using At = const __attribute__((address_space(4))) RecurArgs *;
    At p = (At)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const RecurArgs *)p;
}

template <class X, class G, int KIND, bool BLEND, int V, int R, bool BWD>
__global__ __launch_bounds__(kB, kRecurWaves)
void k_recur(RecurArgs given)
{
    using PX = Pack<X, V>;
    using PG = Pack<G, V>;
    constexpr bool FINE = sizeof(typename PG::S) == 4;
    __shared__ __attribute__((aligned(16))) uint8_t s_flag[kB * R];
    __shared__ int32_t s_seq[kB * R];
    __shared__ float s_A[kWaves][kStrip], s_H[kWaves][kStrip], s_in[kStrip];
    __shared__ int s_reset[kWaves], s_next, s_back;
    __shared__ float2 s_maps[kAhead][kStrip];

    const int LC = 1 << given.lanes_log2, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const uint32_t cols = uint32_t(given.strips) * uint32_t(given.segs), col = blockIdx.x % cols;
    const int64_t tile = blockIdx.x / cols;
    constexpr int kWords = (R + 3) / 4;
    Inputs<X, G, BLEND, V, R, BWD> in;
    uint32_t flags[kWords];
    float ga[BWD ? 1 : R][V], gb[BWD ? 1 : R][V], A[V], H[V];
    bool plain, before_reset;
    float tile_A = 1.0f, tile_H = 0.0f;       // the tile's own map, in the first wave
    bool tile_known = true;
    const auto flag = [&](int r) { return flags[r / 4] >> (r % 4 * 8) & 0xffu; };

    // The tile's map, and the state that enters it.  (More than one turn only where a tile before it has not been
    // started: this block then computes that one's map, and its own again.)
    bool helped = false;
#pragma unroll 1
    for (int64_t target = tile;;) {
    // (what follows from the thread's number is not kept from turn to turn: there is hardly ever a second)
    int tid = int(threadIdx.x);
    asm volatile("" : "+v"(tid));
    const RecurArgs &a = args_again();
    const int lane = tid & 63, r0 = (tid >> a.lanes_log2) * R;
    const Place<V, R, BWD> at(a, target, col, tid);
    in.load(a, at);
    issue_barrier();
    for (int i = tid; i < (kB >> a.lanes_log2) * R; i += kB) {
        const int64_t s = at.tile0 + i;
        uint32_t f = 0;
        int32_t b = -1;
        if (s < at.tile_end)
            b = sequence_of<BWD>(a, at.seg, BWD ? a.rows - 1 - s : s, &f);
        s_flag[i] = uint8_t(f);
        s_seq[i] = b;
    }
    __syncthreads();
    // steps in the middle of sequences are all alike; others are looked at one by one
    bool inside = true;
    if constexpr (R < 4) {
        flags[0] = s_flag[r0];
        inside = flags[0] == kIn;
    } else {
        static_assert(R % 4 == 0, "whole words");
        __builtin_memcpy(flags, __builtin_assume_aligned(s_flag + r0, R % 8 == 0 ? 8 : 4), R);
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            inside = inside && flags[i] == kIn * 0x01010101u;
    }
    plain = __ballot(!inside) == 0;

    // The lane's map, from state 0.  A forward lane keeps, for each step, what the state is multiplied with and
    // what is added; a sequence's first state goes into its first step's.  (Tiles that pass states on may be computed
    // late, or again: where the last states take the first ones' place they read a copy, made before any of them
    // was begun; other tiles' sequences are all their own, and read before the block's barriers.)  A backward lane keeps its inputs as they came and computes the gates
    // twice: four inputs a step, of 16 bits, take fewer registers than what they come to.
    bool reset = false;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        A[k] = 1.0f;
        H[k] = 0.0f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float g[V], v[V], ak[V], wk[V];
        PG::get(in.gate[r], g);
        if constexpr (BWD)
            PX::get(in.d[r], v);
        else
            PX::get(in.x[r], v);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            gate_of<KIND, FINE, BLEND && !BWD>(g[k], ak[k], wk[k]);
            if constexpr (BLEND && !BWD)
                v[k] *= wk[k];
        }
        if (!plain && flag(r) != kIn) {
            if (flag(r) & kReset) {
                reset = true;
                float start[V];
                if constexpr (BWD)
                    last_gradient(a, s_seq[r0 + r], at.c0, start);
                else
                    first_state(a, s_seq[r0 + r], at.c0, start);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if constexpr (BWD) {
                        H[k] = start[k];
                    } else {
                        v[k] = __builtin_fmaf(ak[k], start[k], v[k]);
                        ak[k] = 0.0f;
                        H[k] = 0.0f;
                    }
                }
            } else if (!(flag(r) & kIn)) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    ak[k] = 1.0f;          // a token of no sequence passes the state on
                    v[k] = 0.0f;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (BWD) {
                H[k] = ak[k] * (v[k] + H[k]);
            } else {
                H[k] = __builtin_fmaf(ak[k], H[k], v[k]);
                ga[r][k] = ak[k];
                gb[r][k] = v[k];
            }
            A[k] *= ak[k];
        }
        issue_barrier();                   // a row at a time: registers bound the tokens on their way
    }
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
    before_reset = bpermute32(reset, lane >= LC ? lane - LC : lane);
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
    if (!a.linked)
        break;
    if (wave == 0) {
        const RecurArgs &a = args_again();
        const int c = lane < LC * V ? lane : LC * V - 1;   // a lane a channel of the strip
        float tA = 1.0f, tH = 0.0f, s = 0.0f;
        bool known = target == 0;
        for (int w = 0; w < kWaves; ++w) {
            const bool r = s_reset[w];
            tH = r ? s_H[w][c] : apply(s_A[w][c], tH, s_H[w][c]);
            tA *= s_A[w][c];
            known = known || r;
        }
        const RecurRecord rec(a, col, target);
        int64_t next = -1, back = 0;
        if (target != tile) {
            rec.offer(1, c, tA, kMapKnown);
            rec.offer(0, c, tH, known ? kStateKnown : kMapKnown);
            next = tile;
        } else {
            const bool behind = tile + 1 < a.tiles;
            if (behind) {
                rec.put(0, c, tH, known ? kStateKnown : kMapKnown);
                if (!known)
                    rec.put(1, c, tA, kMapKnown);
            }
            if (tile > 0 && !(s_flag[0] & kReset)) {
                s = look_back(a, col, tile, c, helped, &next, &back);
                if (next < 0 && back == 0 && behind && !known)
                    rec.put(0, c, apply(tA, s, tH), kStateKnown);
            } else {
                // (outputs may take the inputs' place: a block that computes this tile's map too must not read
                // them and find no record; a look-back's loads have come back behind the record's store)
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
        }
        if (lane < LC * V)
            s_in[c] = s;
        if (lane == 0) {
            s_next = int(next);
            s_back = int(back);
        }
        tile_A = tA;
        tile_H = tH;
        tile_known = known;
    }
    helped = true;
    __syncthreads();
    const int next = __builtin_amdgcn_readfirstlane(s_next);
    if (next < 0)
        break;
    target = next;
    }
    const RecurArgs &a = args_again();
    if (a.linked) {
        const int lane = lane_id(), c = lane < LC * V ? lane : LC * V - 1;
        int back = __builtin_amdgcn_readfirstlane(s_back);
        if (back > 0) {
            float s = 0.0f;
            bool first = true;
            for (; back > 0; back -= kAhead, first = false) {
                const int count = back < kAhead ? back : kAhead;
                gather_maps(a, col, tile - back, count, first, wave, c, s_maps);
                __syncthreads();
                if (wave == 0)
                    for (int i = 0; i < count; ++i) {
                        const float2 m = s_maps[i][c];
                        s = bitcast<uint32_t>(m.y) == kTaken ? m.x : apply(m.y, s, m.x);
                    }
                if (back > kAhead)
                    __syncthreads();
            }
            if (wave == 0) {
                if (tile + 1 < a.tiles && !tile_known)
                    RecurRecord(a, col, tile).put(0, c, apply(tile_A, s, tile_H), kStateKnown);
                if (lane < LC * V)
                    s_in[c] = s;
            }
            __syncthreads();
        }
    }
    const int tid = int(threadIdx.x), r0 = (tid >> a.lanes_log2) * R;
    const Place<V, R, BWD> at(a, tile, col, tid);
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
    Rows<X, BWD> out_p(at.template at<X>(a.out), a.out.ts);
    Rows<G, BWD> dgate_p(at.template at<G>(a.dgate), a.dgate.ts);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool special = !plain && flag(r) != kIn, there = !special || (flag(r) & kIn) != 0;
        if (special && (flag(r) & kReset)) {
            if constexpr (BWD) {
                last_gradient(a, s_seq[r0 + r], at.c0, s);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    s[k] = 0.0f;               // (nothing of what was before, were it a NaN)
            }
        }
        if constexpr (BWD) {
            float g[V], v[V], dv[V], hv[V], dx[V], dg[V];
            decode_anew(in.gate[r]);
            decode_anew(in.d[r]);
            PG::get(in.gate[r], g);
            PX::get(in.d[r], dv);
            PX::get(in.h[r], hv);
            if constexpr (BLEND)
                PX::get(in.x[r], v);
            if (special && (flag(r) & kEnd))
                first_state(a, s_seq[r0 + r], at.c0, hv);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float ak, wk;
                gate_of<KIND, FINE, BLEND || KIND == RECUR_SIGMOID>(g[k], ak, wk);
                const float gr = dv[k] + s[k], da = BLEND ? gr * (hv[k] - v[k]) : gr * hv[k];
                dx[k] = BLEND ? wk * gr : gr;
                dg[k] = KIND == RECUR_VALUE ? da : da * (KIND == RECUR_LOG ? ak : ak * wk);
                s[k] = there ? ak * gr : s[k];
            }
            if (there) {
                PX::store(out_p.p, dx, at.drop);
                PG::store(dgate_p.p, dg, at.drop);
            }
            dgate_p.next();
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                s[k] = __builtin_fmaf(ga[r][k], s[k], gb[r][k]);
            if (there)
                PX::store(out_p.p, s, at.drop);
        }
        out_p.next();
        if (special && (flag(r) & kEnd) && a.state_out)
            Pack<float, V>::store(a.state_out + int64_t(s_seq[r0 + r]) * a.channels + at.c0, s, at.drop);
        issue_barrier();
    }
    if (a.starts)
        empty_sequences<BWD>(a);
}

// One token a sequence: no scan, a lane four channels of a row.  (64 x 2048 bf16: 3.2 us, as
// tiles of the kernel above 6.1.)
template <class X, class G, int KIND, bool BLEND, int V>
__device__ __forceinline__ void one_token(const RecurArgs &a, int64_t row, int64_t c)
{
    using PX = Pack<X, V>;
    using PG = Pack<G, V>;
    constexpr bool FINE = sizeof(typename PG::S) == 4;
    const auto at = [&](const RecurTensor &t, auto *type) {
        return static_cast<std::remove_pointer_t<decltype(type)> *>(const_cast<void *>(t.p)) + row * t.ts + c;
    };
    const typename PG::Raw gate = PG::load(at(a.gate, static_cast<typename PG::S *>(nullptr)));
    const typename PX::Raw in = PX::load(at(a.x, static_cast<typename PX::S *>(nullptr)));
    float g[V], v[V], s[V];
    first_state(a, row, c, s);
    PG::get(gate, g);
    PX::get(in, v);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        float ak, wk;
        gate_of<KIND, FINE, BLEND>(g[k], ak, wk);
        s[k] = __builtin_fmaf(ak, s[k], BLEND ? v[k] * wk : v[k]);
    }
    PX::store(at(a.out, static_cast<typename PX::S *>(nullptr)), s, 0);
    Pack<float, V>::store(a.state_out + row * a.channels + c, s, 0);
}

template <class X, class G, int KIND, bool BLEND>
__global__ __launch_bounds__(kB) void k_recur_step(RecurArgs a)
{
    const int tid = int(threadIdx.x), lanes = 1 << a.lanes_log2;
    const int64_t row = int64_t(blockIdx.x / uint32_t(a.strips)) * (kB >> a.lanes_log2) + (tid >> a.lanes_log2);
    int64_t c = (int64_t(blockIdx.x % uint32_t(a.strips)) * lanes + (tid & (lanes - 1))) * tune::kRecurVec;
    if (row >= a.rows)
        return;
    if (c + tune::kRecurVec <= a.channels)
        one_token<X, G, KIND, BLEND, tune::kRecurVec>(a, row, c);
    else
        for (; c < a.channels; ++c)            // (only its own: outputs may take the inputs' place)
            one_token<X, G, KIND, BLEND, 1>(a, row, c);
}

template <class X, class G>
int launch_step(const RecurLaunch &L)
{
    const auto go = [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
        const auto kernel = L.a.blend ? k_recur_step<X, G, KIND, true> : k_recur_step<X, G, KIND, false>;
        launch_timed(kernel, dim3(uint32_t(L.plan.grid)), dim3(kB), 0, L.stream, L.ev_begin, L.ev_end, L.a);
    };
    switch (L.a.kind) {
    case RECUR_SIGMOID: go(std::integral_constant<int, RECUR_SIGMOID>{}); break;
    case RECUR_LOG: go(std::integral_constant<int, RECUR_LOG>{}); break;
    default: go(std::integral_constant<int, RECUR_VALUE>{}); break;
    }
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

template <class X, class G, int V, int R, bool BWD>
int launch_one(const RecurLaunch &L)
{
    const auto go = [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
        const auto kernel = L.a.blend ? k_recur<X, G, KIND, true, V, R, BWD> : k_recur<X, G, KIND, false, V, R, BWD>;
        launch_timed(kernel, dim3(uint32_t(L.plan.grid)), dim3(kB), 0, L.stream, L.ev_begin, L.ev_end, L.a);
    };
    switch (L.a.kind) {
    case RECUR_SIGMOID: go(std::integral_constant<int, RECUR_SIGMOID>{}); break;
    case RECUR_LOG: go(std::integral_constant<int, RECUR_LOG>{}); break;
    default: go(std::integral_constant<int, RECUR_VALUE>{}); break;
    }
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
    if constexpr (!BWD)
        if (p.step)
            return launch_step<X, G>(L);
    if (p.linked) {
        const int64_t vectors = p.tiles * p.strips * L.a.segs * kRecurRecBytes / 16;
        const int64_t states = L.kept ? L.a.n_seq * L.a.channels : 0, items = vectors > states ? vectors : states;
        const int64_t blocks = (items + kB * 2 - 1) / (kB * 2), most = 4096;
        hipLaunchKernelGGL(k_recur_clear, dim3(uint32_t(blocks < most ? blocks : most)), dim3(kB), 0,
                           static_cast<hipStream_t>(L.stream), L.a, vectors, L.state, L.kept, states);
        if (hipGetLastError() != hipSuccess)
            return ST_HIP;
    }
    constexpr int R = recur_rows(sizeof(typename InTraits<X>::S), sizeof(typename InTraits<G>::S), BWD);
    if (p.vec == 1)
        return launch_one<X, G, 1, 4, BWD>(L);
    return p.per_lane == 1 ? launch_one<X, G, 4, 1, BWD>(L) : launch_one<X, G, 4, R, BWD>(L);
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

}  // namespace
}  // namespace rk
