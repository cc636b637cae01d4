// serve_blocks.hip -- block tables and slot maps from request lengths.
//
// block_tables.  Request b needs need_b = ceil(len_b / block) blocks and holds
// held_b.  With give_b = max(held_b - need_b, 0), take_b = max(need_b - held_b, 0)
// and their exclusive sums over the requests G_b, T_b, block number i of those
// b gives back goes to place tail + G_b + i of the ring of free blocks, and
// block number i of those it takes comes from place head + T_b + i.  A place
// at or behind the old tail holds a block given back in this very call: it
// is read from the giver's table row, never from the ring, so no block waits
// for another's store.
//
// slot_map.  starts_b, the exclusive sum of the new tokens, is scanned by
// every block for itself (a few thousand counts cost less than a launch);
// token t then finds its request by bisection in LDS.
#define RK_UNIT unit_serve_blocks
#include "rk_serve_device.hpp"

namespace rk {
namespace {

__device__ __forceinline__ int blocks_of(int len, const Divider &d)
{
    return len > 0 ? int(divide(uint32_t(len - 1), d)) + 1 : 0;
}

// v modulo size (1 <= size < 2^31), not negative.  A 64-bit remainder takes
// over a hundred instructions, so counters that fit 32 bits do without.
__device__ __forceinline__ int64_t ring_place(int64_t v, int64_t size)
{
    if (v >= 0 && v < (int64_t(1) << 32))
        return uint32_t(v) % uint32_t(size);
    const int64_t m = v % size;
    return m < 0 ? m + size : m;
}

// A place of the ring, 0 <= at < 2 * size.
__device__ __forceinline__ int64_t wrap(int64_t at, int64_t size) { return at >= size ? at - size : at; }

// What one request asks for.
struct Ask {
    int held, need, over;     // blocks it holds and gets to hold; blocks beyond the table's width
    __device__ __forceinline__ int give() const { return held > need ? held - need : 0; }
    __device__ __forceinline__ int take() const { return need > held ? need - held : 0; }
    __device__ __forceinline__ int after(int64_t left) const   // blocks held when `left` blocks are left for it
    {
        const int kept = need < held ? need : held;
        return kept + (left < 0 ? 0 : left < take() ? int(left) : take());
    }
};

// Four requests from b on (those from req on ask for nothing).
struct Asks {
    Ask q[4];
    __device__ __forceinline__ void load(const TablesArgs &a, int64_t b)
    {
        int len[4] = {0, 0, 0, 0}, held[4] = {0, 0, 0, 0};
        if (b + 4 <= a.req) {
            const u32x4 l = load16(a.lens + b), h = load16(a.held + b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                len[i] = int(l[i]);
                held[i] = int(h[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (b + i < a.req) {
                    len[i] = a.lens[b + i];
                    held[i] = a.held[b + i];
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int want = blocks_of(len[i], a.block);
            q[i].need = want < a.max_blocks ? want : a.max_blocks;
            q[i].over = want - q[i].need;
            q[i].held = held[i] < 0 ? 0 : held[i] > a.max_blocks ? a.max_blocks : held[i];
        }
    }
};

// The ring before and after the call.
struct Ring {
    int64_t there, head;      // blocks that were free, and the place of the first
    int64_t given, taken;     // blocks that come and go

    __device__ __forceinline__ Ring(int64_t head_, int64_t tail, int64_t size, int64_t gives, int64_t takes)
    {
        head = ring_place(head_, size);
        there = tail - head_;
        there = there < 0 ? 0 : there > size ? size : there;
        given = gives < size - there ? gives : size - there;
        taken = takes < there + given ? takes : there + given;
    }
};

__device__ __forceinline__ void write_state(const TablesArgs &a, const Ring &r, int64_t head, int64_t tail, int64_t gives,
                                            int64_t takes, int64_t over)
{
    a.state_out[0] = head + r.taken;
    a.state_out[1] = tail + r.given;
    a.state_out[2] = takes - r.taken + over;
    a.state_out[3] = gives - r.given;
}

// A wave's share `part` of `parts` of one request's moves, kMoveEach ids a
// lane at a time.  p: the request's plan; given_id(g): the id of give number g.
template <class GivenId>
__device__ __forceinline__ void move(const TablesArgs &a, int64_t b, const TablesPlan &p, const Ring &r, uint32_t part,
                                     uint32_t parts, GivenId &&given_id)
{
    constexpr int E = tune::kMoveEach;
    int32_t *line = a.table + b * a.ts;
    const bool gives = p.held > p.need;
    const int64_t from = gives ? p.give0 : p.take0;
    const int64_t limit = (gives ? r.given : r.taken) - from;
    int64_t count = gives ? p.held - p.need : p.need - p.held;
    count = count < limit ? count : limit;
    const int first = gives ? p.need : p.held;
    for (int64_t k = int64_t(part) * (64 * E) + lane_id(); k < count; k += int64_t(parts) * (64 * E)) {
        int32_t id[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t i = k + 64 * e;
            if (i < count) {
                if (gives)
                    id[e] = line[first + i];
                else if (from + i < r.there)
                    id[e] = a.ring[wrap(r.head + from + i, a.ring_size)];
                else
                    id[e] = given_id(from + i - r.there);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t i = k + 64 * e;
            if (i < count) {
                if (gives)                    // (head + there + given <= head + size < 2 * size)
                    a.ring[wrap(r.head + r.there + from + i, a.ring_size)] = id[e];
                else
                    line[first + i] = id[e];
            }
        }
    }
}

// The last request of [lo, hi) whose offset is <= i: off[lo] <= i.
__device__ __forceinline__ int owner(const uint32_t *off, int lo, int hi, uint32_t i)
{
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The same for one i of the whole wave among up to 4096 requests: 64 probes at
// a time, two rounds.
__device__ __forceinline__ int wave_owner(const uint32_t *off, int req, uint32_t i)
{
    static_assert(tune::kMoveLdsRequests <= 64 * 64, "two rounds");
    const int step = (req + 63) / 64;
    int at = lane_id() * step;
    const int lo = (__popcll(__ballot(at < req && off[at < req ? at : 0] <= i)) - 1) * step;
    at = lo + lane_id();
    const bool in = lane_id() < step && at < req;
    return lo + __popcll(__ballot(in && off[in ? at : 0] <= i)) - 1;
}

// One launch: every block scans the requests for itself (more work in all, but
// one launch and no round trip through memory between scan and moves) and keeps
// their offsets in LDS; the ids that move are then dealt to the waves in equal
// shares, whatever requests they belong to.  A wave finds the requests at its
// ends together, its lanes theirs by bisection between these (bisection among
// all 2048 took 4 us more).  Only for outputs apart from the inputs: other
// blocks may still read these.
__global__ __launch_bounds__(tune::kMoveBlock) void k_tables(TablesArgs a)
{
    constexpr int B = tune::kMoveBlock;
    __shared__ uint64_t part[2][B / 64], part_over[B / 64];
    extern __shared__ uint32_t give0[];
    const int req = int(a.req);
    uint32_t *take0 = give0 + req + 1;
    int *first = reinterpret_cast<int *>(take0 + req + 1);     // the first of its table line's entries that move
    const int64_t head = a.state[0], tail = a.state[1];
    uint64_t sum = 0;                         // gives, takes in its halves
    uint64_t over = 0;
    int turn = 0;
    for (int base = 0; base < req; base += 4 * B, turn ^= 1) {
        const int b = base + 4 * int(threadIdx.x);
        Asks asks;
        asks.load(a, b);
        uint64_t mine = 0, all;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mine += uint64_t(asks.q[i].give()) << 32 | uint32_t(asks.q[i].take());
        uint64_t at = sum + block_prefix<B>(mine, part[turn], &all);
        sum += all;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Ask &q = asks.q[i];
            over += q.over;
            if (b + i < req) {
                give0[b + i] = uint32_t(at >> 32);
                take0[b + i] = uint32_t(at);
                first[b + i] = q.need < q.held ? q.need : q.held;
            }
            at += uint64_t(q.give()) << 32 | uint32_t(q.take());
        }
    }
    const int64_t gives = int64_t(sum >> 32), takes = int64_t(uint32_t(sum));
    if (threadIdx.x == 0) {
        give0[req] = uint32_t(gives);
        take0[req] = uint32_t(takes);
    }
    __syncthreads();
    const Ring r(head, tail, a.ring_size, gives, takes);
    if (blockIdx.x == 0) {
        uint64_t beyond;
        block_prefix<B>(over, part_over, &beyond);
        if (threadIdx.x == 0)
            write_state(a, r, head, tail, gives, takes, int64_t(beyond));
    }
    const uint32_t threads = gridDim.x * B, id0 = blockIdx.x * B + threadIdx.x;
    for (int b = int(id0); b < req; b += int(threads)) {
        const int64_t left = r.taken - take0[b], take = take0[b + 1] - take0[b];
        a.held_out[b] = first[b] + int(left < 0 ? 0 : left < take ? left : take);
    }
    const auto given_id = [&](uint32_t g, int lo, int hi) {
        const int b = owner(give0, lo, hi, g);
        return a.table[b * a.ts + first[b] + (g - give0[b])];
    };
    const int64_t moves = r.taken + r.given;
    const auto deal = [&](auto each) {
        constexpr int E = decltype(each)::value;
        const int64_t wave = blockIdx.x * (B / 64) + __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
        for (int64_t base = wave * (64 * E); base < moves; base += int64_t(threads) * E) {
            // the requests that the wave's ids can belong to: takes first, then gives
            const int64_t end = base + 64 * E < moves ? base + 64 * E : moves;
            int t_lo = 0, t_hi = 0, g_lo = 0, g_hi = 0;
            if (base < r.taken) {
                t_lo = wave_owner(take0, req, uint32_t(base));
                t_hi = wave_owner(take0, req, uint32_t((end < r.taken ? end : r.taken) - 1)) + 1;
            }
            if (end > r.taken) {
                g_lo = wave_owner(give0, req, uint32_t((base > r.taken ? base : r.taken) - r.taken));
                g_hi = wave_owner(give0, req, uint32_t(end - 1 - r.taken)) + 1;
            }
            int32_t id[E];
            int32_t *to[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int64_t i = base + 64 * e + lane_id();
                to[e] = nullptr;
                if (i < r.taken) {
                    const int b = owner(take0, t_lo, t_hi, uint32_t(i));
                    to[e] = a.table + (b * a.ts + first[b] + (i - take0[b]));
                    id[e] = i < r.there ? a.ring[wrap(r.head + i, a.ring_size)] : given_id(uint32_t(i - r.there), 0, req);
                } else if (i < end) {
                    const uint32_t g = uint32_t(i - r.taken);
                    to[e] = a.ring + wrap(r.head + r.there + g, a.ring_size);   // (head + there + given <= head + size)
                    id[e] = given_id(g, g_lo, g_hi);
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (to[e])
                    *to[e] = id[e];
        }
    };
    // a step of decoding moves few ids: one a lane, so that all are under way at once; else several,
    // which share the search for the requests
    if (moves <= int64_t(threads))
        deal(std::integral_constant<int, 1>());
    else
        deal(std::integral_constant<int, tune::kMoveEach>());
}

// Two launches, for outputs that are the inputs and for more requests: one
// block scans them, leaves the plans, and writes held_out and state_out.
template <int B>
__global__ __launch_bounds__(B) void k_tables_scan(TablesArgs a)
{
    __shared__ int64_t part[2][2][B / 64], part_over[B / 64];
    const int64_t head = a.state[0], tail = a.state[1];
    int64_t gives = 0, takes = 0, over = 0, take0 = 0;
    Asks asks;
    int turn = 0;
    for (int64_t base = 0; base < a.req; base += 4 * B, turn ^= 1) {
        const int64_t b = base + 4 * int64_t(threadIdx.x);
        asks.load(a, b);
        int64_t give = 0, take = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            give += asks.q[i].give();
            take += asks.q[i].take();
            over += asks.q[i].over;
        }
        int64_t g, t;
        int64_t give0 = gives + block_prefix<B>(give, part[turn][0], &g);
        take0 = takes + block_prefix<B>(take, part[turn][1], &t);
        gives += g;
        takes += t;
        int64_t at = take0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Ask &q = asks.q[i];
            if (b + i < a.req)
                a.plan[b + i] = TablesPlan{give0, at, q.held, q.need};
            give0 += q.give();
            at += q.take();
        }
    }
    int64_t beyond;
    block_prefix<B>(over, part_over, &beyond);    // (state and held have been read before they may be written)
    const Ring r(head, tail, a.ring_size, gives, takes);
    for (int64_t base = 0; base < a.req; base += 4 * B) {
        const int64_t b = base + 4 * int64_t(threadIdx.x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (b + i >= a.req)
                continue;
            if (a.req > 4 * B) {              // (otherwise the one round above has left asks and take0)
                const TablesPlan p = a.plan[b + i];
                asks.q[i] = Ask{p.held, p.need, 0};
                take0 = p.take0;
            }
            a.held_out[b + i] = asks.q[i].after(r.taken - take0);
            take0 += asks.q[i].take();
        }
    }
    if (threadIdx.x == 0) {
        *a.totals = TablesTotals{gives, takes, head, tail};
        write_state(a, r, head, tail, gives, takes, beyond);
    }
}

__global__ __launch_bounds__(tune::kMoveBlock) void k_tables_move(TablesArgs a)
{
    const uint32_t w = blockIdx.x * (tune::kMoveBlock / 64) + uint32_t(__builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)));
    const uint32_t b = divide(w, a.waves);
    if (b >= uint32_t(a.req))
        return;
    const TablesPlan p = a.plan[b];
    const TablesTotals t = *a.totals;
    const Ring r(t.head, t.tail, a.ring_size, t.gives, t.takes);
    move(a, b, p, r, w - b * a.waves.d, a.waves.d, [&](int64_t g) {
        int64_t lo = 0, hi = a.req;           // the last request whose gives begin at or before g
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) / 2;
            if (a.plan[mid].give0 <= g)
                lo = mid;
            else
                hi = mid;
        }
        return a.table[lo * a.ts + a.plan[lo].need + (g - a.plan[lo].give0)];
    });
}

// ------------------------------------------------------------------ slots

__device__ __forceinline__ int fresh_of(int fresh, int len)
{
    len = len > 0 ? len : 0;
    return fresh < 0 ? 0 : fresh < len ? fresh : len;
}

// Sums of token counts saturate at 2^31 - 1 (adding that way is associative
// for counts that are not negative).
__device__ __forceinline__ uint32_t sat_add(uint32_t x, uint32_t y)
{
    const uint32_t s = x + y;
    return s < 0x7fffffffu ? s : 0x7fffffffu;
}

struct SatPlus {
    __device__ __forceinline__ static uint32_t apply(uint32_t a, uint32_t b) { return sat_add(a, b); }
};

// More requests than a block keeps in LDS: their offsets, by one block.
__global__ __launch_bounds__(tune::kScanBlock) void k_slot_starts(SlotArgs a)
{
    constexpr int B = tune::kScanBlock;
    __shared__ uint32_t part[2][B / 64];
    uint32_t sum = 0;
    int turn = 0;
    for (int64_t base = 0; base < a.req; base += B, turn ^= 1) {
        const int64_t b = base + threadIdx.x;
        uint32_t t;
        const uint32_t v = b < a.req ? uint32_t(fresh_of(a.fresh[b], a.lens[b])) : 0u;
        const uint32_t s = sat_add(sum, block_prefix<B, SatPlus>(v, part[turn], &t));
        if (b < a.req)
            a.starts[b] = int32_t(s);
        sum = sat_add(sum, t);
    }
    if (threadIdx.x == 0)
        a.starts[a.req] = int32_t(sum);
}

// What a block keeps in LDS of every request, req + 1 words each.
struct Kept {
    uint32_t *start;          // tokens before it
    int32_t *first;           // position of its first new token
    int32_t *blocks;          // blocks of its table line that count
};

__device__ __forceinline__ int counted(int held, int max_blocks) { return held < max_blocks ? held : max_blocks; }

// The block's own scan of all requests, four a thread at a time.  `lo` and
// `hi`: the requests of the block's tokens `from` and `to` - 1.
template <int B>
__device__ __forceinline__ void scan_requests(const SlotArgs &a, const Kept &k, int64_t from, int64_t to, int *lo, int *hi)
{
    __shared__ uint32_t part[2][B / 64];
    const int req = int(a.req);
    uint32_t sum = 0;
    int turn = 0;
    for (int base = 0; base < req; base += 4 * B, turn ^= 1) {
        const int b = base + 4 * int(threadIdx.x);
        int len[4], fresh[4], held[4];
        if (b + 4 <= req) {
            const u32x4 l = load16(a.lens + b), f = load16(a.fresh + b), h = load16(a.held + b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                len[i] = int(l[i]);
                fresh[i] = int(f[i]);
                held[i] = int(h[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = b + i < req ? b + i : req - 1;
                len[i] = a.lens[c];
                fresh[i] = a.fresh[c];
                held[i] = a.held[c];
            }
        }
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fresh[i] = b + i < req ? fresh_of(fresh[i], len[i]) : 0;
            mine = sat_add(mine, uint32_t(fresh[i]));
        }
        uint32_t all;
        uint32_t at = sat_add(sum, block_prefix<B, SatPlus>(mine, part[turn], &all));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t end = sat_add(at, uint32_t(fresh[i]));
            if (b + i < req) {
                k.start[b + i] = at;
                k.first[b + i] = len[i] - fresh[i];
                k.blocks[b + i] = counted(held[i], a.max_blocks);
                if (blockIdx.x == 0)
                    a.starts[b + i] = int32_t(at);
                if (from >= at && from < end)
                    *lo = b + i;
                if (to - 1 >= at && to - 1 < end)
                    *hi = b + i;
            }
            at = end;
        }
        sum = sat_add(sum, all);
    }
    if (threadIdx.x == 0) {
        k.start[req] = sum;
        if (blockIdx.x == 0)
            a.starts[req] = int32_t(sum);
    }
}

// T tokens a thread, 16 bytes of slots, at a time: every store of a wave covers
// one run of whole lines.  LDS: the block scans the requests itself and looks
// them up there; otherwise a.starts holds the sums.
template <class Slot, bool LDS, bool STREAM>
__global__ __launch_bounds__(tune::kSlotBlock) void k_slots(SlotArgs a)
{
    constexpr int B = tune::kSlotBlock, T = 16 / int(sizeof(Slot));
    extern __shared__ uint32_t lds[];
    __shared__ int s_lo, s_hi;
    const int req = int(a.req);
    const int64_t from = int64_t(blockIdx.x) * a.per_block;
    const int64_t to = from + a.per_block < a.capacity ? from + a.per_block : a.capacity;
    const Kept kept{lds, reinterpret_cast<int32_t *>(lds + req + 1), reinterpret_cast<int32_t *>(lds + 2 * (a.req + 1))};
    if (threadIdx.x == 0) {
        s_lo = 0;
        s_hi = req - 1;
    }
    if constexpr (LDS) {
        __syncthreads();
        scan_requests<B>(a, kept, from, to, &s_lo, &s_hi);
    }
    __syncthreads();
    const auto start = [&](int b) { return int64_t(LDS ? kept.start[b] : uint32_t(a.starts[b])); };
    const int64_t total = start(req);
    const int s0 = s_lo, s1 = s_hi + 1;
    Slot *slots = static_cast<Slot *>(a.slots);
    for (int64_t t = from + int64_t(threadIdx.x) * T; t < to; t += int64_t(B) * T) {
        Slot slot[T];
        int pos[T], who[T], off[T];
        int32_t id[T];
        int b = t < total ? last_start(start, s0, s1, t) : s0;    // start(s0) <= t < start(s1)
        int64_t begin = start(b), end = t < total ? start(b + 1) : begin;
#pragma unroll
        for (int k = 0; k < T; ++k) {
            const int64_t i = t + k;
            id[k] = -1;
            pos[k] = 0;
            off[k] = 0;
            who[k] = -1;
            if (i < total && i < to) {
                while (i >= end) {
                    ++b;
                    begin = end;
                    end = start(b + 1);
                }
                int first, blocks;
                if constexpr (LDS) {
                    first = kept.first[b];
                    blocks = kept.blocks[b];
                } else {
                    const int len = a.lens[b];
                    first = len - fresh_of(a.fresh[b], len);
                    blocks = counted(a.held[b], a.max_blocks);
                }
                who[k] = b;
                pos[k] = first + int(i - begin);
                const int blk = int(divide(uint32_t(pos[k]), a.block));
                off[k] = pos[k] - blk * int(a.block.d);
                if (blk < blocks)
                    id[k] = a.table[int64_t(b) * a.ts + blk];
            }
        }
#pragma unroll
        for (int k = 0; k < T; ++k)
            slot[k] = id[k] >= 0 && id[k] < a.n_blocks ? Slot(int64_t(id[k]) * a.block.d + off[k]) : Slot(-1);
        if (t + T <= to) {
            Words<4>::template store<STREAM>(slots + t, words_of<4>(slot));
            if (a.positions)
                Words<T>::template store<STREAM>(a.positions + t, words_of<T>(pos));
            if (a.requests)
                Words<T>::template store<STREAM>(a.requests + t, words_of<T>(who));
        } else {
#pragma unroll
            for (int k = 0; k < T; ++k)
                if (t + k < to) {
                    slots[t + k] = slot[k];
                    if (a.positions)
                        a.positions[t + k] = pos[k];
                    if (a.requests)
                        a.requests[t + k] = who[k];
                }
        }
    }
}

template <class Slot>
int run_slots(const SlotLaunch &L)
{
    const dim3 grid(uint32_t(L.grid)), block(tune::kSlotBlock);
    if (L.a.req <= tune::kSlotLdsRequests) {
        const size_t lds = size_t(slots_lds_bytes(L.a.req));
        if (L.stream_out)
            launch_timed(k_slots<Slot, true, true>, grid, block, lds, L.stream, L.ev_begin, L.ev_end, L.a);
        else
            launch_timed(k_slots<Slot, true, false>, grid, block, lds, L.stream, L.ev_begin, L.ev_end, L.a);
    } else {
        launch_timed(k_slot_starts, dim3(1), dim3(tune::kScanBlock), 0, L.stream, L.ev_begin, L.ev_end, L.a);
        launch_timed(k_slots<Slot, false, false>, grid, block, 0, L.stream, nullptr, nullptr, L.a);
    }
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

}  // namespace

int launch_tables(const TablesLaunch &L)
{
    const dim3 grid(uint32_t(L.grid)), block(tune::kMoveBlock);
    if (L.one_launch) {
        launch_timed(k_tables, grid, block, size_t(tables_lds_bytes(L.a.req)), L.stream, L.ev_begin, L.ev_end, L.a);
    } else {
        if (L.a.req <= 1024)
            launch_timed(k_tables_scan<256>, dim3(1), dim3(256), 0, L.stream, L.ev_begin, L.ev_end, L.a);
        else
            launch_timed(k_tables_scan<1024>, dim3(1), dim3(1024), 0, L.stream, L.ev_begin, L.ev_end, L.a);
        if (L.grid > 0)
            launch_timed(k_tables_move, grid, block, 0, L.stream, nullptr, nullptr, L.a);
    }
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

int launch_slots(const SlotLaunch &L)
{
    return L.slot_dtype == I64 ? run_slots<int64_t>(L) : run_slots<int32_t>(L);
}

}  // namespace rk
