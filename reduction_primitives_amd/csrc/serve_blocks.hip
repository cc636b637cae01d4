// serve_blocks.hip -- block tables and slot maps from request lengths.
//
// block_tables.  Request b needs need_b = ceil(len_b / block) blocks and holds
// held_b.  With give_b = max(held_b - need_b, 0), take_b = max(need_b - held_b, 0)
// and their exclusive sums over the requests G_b, T_b, block number i of those
// b gives back goes to place tail + G_b + i of the ring of free blocks, and
// block number i of those it takes comes from place head + T_b + i.  A place
// at or behind the old tail holds a block given back in this very call: it
// is read from the giver's table row, never from the ring, so no block waits
// for another's store.  The first launch, one block, scans the requests; the
// second moves the ids, any number of blocks on any request's.
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


__device__ __forceinline__ int64_t ring_place(int64_t v, int64_t size)
{
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
};

__device__ __forceinline__ Ask ask(int len, int held, const TablesArgs &a)
{
    Ask q;
    const int want = blocks_of(len, a.block);
    q.need = want < a.max_blocks ? want : a.max_blocks;
    q.over = want - q.need;
    q.held = held < 0 ? 0 : held > a.max_blocks ? a.max_blocks : held;
    return q;
}

// First launch, one block: four requests a thread at a time.
__global__ __launch_bounds__(tune::kScanBlock) void k_tables_scan(TablesArgs a)
{
    constexpr int B = tune::kScanBlock;
    __shared__ int64_t part[2][2][B / 64];
    __shared__ int64_t part_over[B / 64];
    const int64_t head = a.state[0], tail = a.state[1];
    int64_t gives = 0, takes = 0, over = 0;
    Ask q[4];
    int64_t g0[4], t0[4];
    int turn = 0;
    for (int64_t base = 0; base < a.req; base += 4 * B, turn ^= 1) {
        const int64_t b = base + 4 * int64_t(threadIdx.x);
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
        int64_t give = 0, take = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = ask(len[i], held[i], a);
            g0[i] = give;
            t0[i] = take;
            give += q[i].give();
            take += q[i].take();
            over += q[i].over;
        }
        int64_t g, t;
        const int64_t gb = gives + block_prefix<B>(give, part[turn][0], &g);
        const int64_t tb = takes + block_prefix<B>(take, part[turn][1], &t);
        gives += g;
        takes += t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g0[i] += gb;
            t0[i] += tb;
            if (b + i < a.req)
                a.plan[b + i] = TablesPlan{g0[i], t0[i], q[i].held, q[i].need};
        }
    }
    int64_t missing;
    block_prefix<B>(over, part_over, &missing);   // (state and held have been read before they may be written)
    const int64_t size = a.ring_size;
    int64_t there = tail - head;
    there = there < 0 ? 0 : there > size ? size : there;
    const int64_t given = gives < size - there ? gives : size - there;
    const int64_t taken = takes < there + given ? takes : there + given;
    for (int64_t base = 0; base < a.req; base += 4 * B) {
        const int64_t b = base + 4 * int64_t(threadIdx.x);
        int out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (a.req > 4 * B && b + i < a.req) {   // (otherwise the one round above has left q and t0)
                const TablesPlan p = a.plan[b + i];
                q[i] = Ask{p.held, p.need, 0};
                t0[i] = p.take0;
            }
            const int64_t left = taken - t0[i];
            const int take = q[i].take();
            out[i] = (q[i].need < q[i].held ? q[i].need : q[i].held) + (left < 0 ? 0 : left < take ? int(left) : take);
        }
        if (b + 4 <= a.req) {
            Words<4>::template store<false>(a.held_out + b, words_of<4>(out));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (b + i < a.req)
                    a.held_out[b + i] = out[i];
        }
    }
    if (threadIdx.x == 0) {
        a.plan[a.req] = TablesPlan{gives, takes, 0, 0};
        *a.totals = TablesTotals{taken, given, there, ring_place(head, size)};
        a.state_out[0] = head + taken;
        a.state_out[1] = tail + given;
        a.state_out[2] = takes - taken + missing;
        a.state_out[3] = gives - given;
    }
}

// The block id of give number g: of the last request whose gives begin at or
// before it.
__device__ __forceinline__ int32_t given_id(const TablesArgs &a, int64_t g)
{
    int64_t lo = 0, hi = a.req;               // give0 of lo <= g < give0 of hi
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (a.plan[mid].give0 <= g)
            lo = mid;
        else
            hi = mid;
    }
    return a.table[lo * a.ts + a.plan[lo].need + (g - a.plan[lo].give0)];
}

// Second launch: a.waves waves move a request's blocks, kMoveEach entries a lane
// at a time.
__global__ __launch_bounds__(tune::kMoveBlock) void k_tables_move(TablesArgs a)
{
    constexpr int E = tune::kMoveEach;
    const uint32_t w = blockIdx.x * (tune::kMoveBlock / 64) + uint32_t(__builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)));
    const uint32_t b = divide(w, a.waves);
    if (b >= uint32_t(a.req))
        return;
    const TablesPlan p = a.plan[b];
    const TablesTotals all = *a.totals;
    int32_t *line = a.table + int64_t(b) * a.ts;
    const bool gives = p.held > p.need;
    const int64_t from = gives ? p.give0 : p.take0;
    const int64_t limit = (gives ? all.given : all.taken) - from;
    int64_t count = gives ? p.held - p.need : p.need - p.held;
    count = count < limit ? count : limit;
    const int first = gives ? p.need : p.held;
    for (int64_t k = int64_t(w - b * a.waves.d) * (64 * E) + lane_id(); k < count; k += int64_t(a.waves.d) * (64 * E)) {
        int32_t id[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t i = k + 64 * e;
            if (i < count) {
                if (gives)
                    id[e] = line[first + i];
                else if (from + i < all.there)
                    id[e] = a.ring[wrap(all.head + from + i, a.ring_size)];
                else
                    id[e] = given_id(a, from + i - all.there);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t i = k + 64 * e;
            if (i < count) {
                if (gives)                    // (head + there + given <= head + size < 2 * size)
                    a.ring[wrap(all.head + all.there + from + i, a.ring_size)] = id[e];
                else
                    line[first + i] = id[e];
            }
        }
    }
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
    const Kept kept{lds, reinterpret_cast<int32_t *>(lds + req + 1), reinterpret_cast<int32_t *>(lds + 2 * (req + 1))};
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
        int b = s0;
        if (t < total) {                      // start(lo) <= t < start(hi)
            int hi = s1;
            while (hi - b > 1) {
                const int mid = (b + hi) >> 1;
                if (start(mid) <= t)
                    b = mid;
                else
                    hi = mid;
            }
        }
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
        const size_t lds = (size_t(L.a.req) + 1) * 12;
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
    launch_timed(k_tables_scan, dim3(1), dim3(tune::kScanBlock), 0, L.stream, L.ev_begin, L.ev_end, L.a);
    if (L.grid > 0)
        launch_timed(k_tables_move, dim3(uint32_t(L.grid)), dim3(tune::kMoveBlock), 0, L.stream, nullptr, nullptr, L.a);
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

int launch_slots(const SlotLaunch &L)
{
    return L.slot_dtype == I64 ? run_slots<int64_t>(L) : run_slots<int32_t>(L);
}

}  // namespace rk
