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


// Workspace (see kTablesHeader): pairs (given back before, taken before) of
// every request and of the end, then the blocks each request held.
__device__ __forceinline__ int64_t *offsets_of(const TablesArgs &a) { return a.offsets + kTablesHeader; }
__device__ __forceinline__ int32_t *held_of(const TablesArgs &a)
{
    return reinterpret_cast<int32_t *>(offsets_of(a) + 2 * (a.req + 1));
}

__device__ __forceinline__ int64_t ring_place(int64_t v, int64_t size)
{
    const int64_t m = v % size;
    return m < 0 ? m + size : m;
}

__global__ __launch_bounds__(tune::kScanBlock) void k_tables_scan(TablesArgs a)
{
    constexpr int B = tune::kScanBlock;
    __shared__ int64_t part[2][2][B / 64];
    __shared__ unsigned long long s_over;
    int64_t *off = offsets_of(a);
    int32_t *before = held_of(a);
    if (threadIdx.x == 0)
        s_over = 0;
    int64_t gives = 0, takes = 0, over = 0;
    int turn = 0;
    for (int64_t base = 0; base < a.req; base += B, turn ^= 1) {
        const int64_t b = base + threadIdx.x;
        int64_t give = 0, take = 0;
        int held = 0;
        if (b < a.req) {
            const int want = blocks_of(a.lens[b], a.block);
            const int need = want < a.max_blocks ? want : a.max_blocks;
            held = a.held[b];
            held = held < 0 ? 0 : held > a.max_blocks ? a.max_blocks : held;
            give = held > need ? held - need : 0;
            take = need > held ? need - held : 0;
            over += want - need;
            before[b] = held;
        }
        int64_t g, t;
        const int64_t g0 = gives + block_prefix<B>(give, part[turn][0], &g);
        const int64_t t0 = takes + block_prefix<B>(take, part[turn][1], &t);
        gives += g;
        takes += t;
        if (b < a.req) {
            off[2 * b] = g0;
            off[2 * b + 1] = t0;
        }
    }
    if (over)
        atomicAdd(&s_over, (unsigned long long)over);
    const int64_t head = a.state[0], tail = a.state[1];
    __syncthreads();                          // state and held are read before they may be written
    const int64_t size = a.ring_size;
    int64_t there = tail - head;
    there = there < 0 ? 0 : there > size ? size : there;
    const int64_t given = gives < size - there ? gives : size - there;
    const int64_t taken = takes < there + given ? takes : there + given;
    for (int64_t b = threadIdx.x; b < a.req; b += B) {
        const int want = blocks_of(a.lens[b], a.block);
        const int need = want < a.max_blocks ? want : a.max_blocks;
        const int held = before[b];
        const int64_t left = taken - off[2 * b + 1];
        const int64_t take = need > held ? need - held : 0;
        const int64_t got = left < 0 ? 0 : left < take ? left : take;
        a.held_out[b] = (need < held ? need : held) + int(got);
    }
    if (threadIdx.x == 0) {
        off[2 * a.req] = gives;
        off[2 * a.req + 1] = takes;
        a.offsets[0] = taken;
        a.offsets[1] = given;
        a.offsets[2] = there;
        a.offsets[3] = ring_place(head, size);
        a.state_out[0] = head + taken;
        a.state_out[1] = tail + given;
        a.state_out[2] = takes - taken + int64_t(s_over);
        a.state_out[3] = gives - given;
    }
}

// The last request whose offset (0: given back, 1: taken) is <= i; off holds
// an end entry, and i < the end.
__device__ __forceinline__ int64_t owner(const int64_t *off, int64_t req, int64_t i, int which)
{
    int64_t lo = 0, hi = req;                 // off[lo] <= i < off[hi]
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) / 2;
        if (off[2 * mid + which] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The block id of give number g.
__device__ __forceinline__ int32_t given_id(const TablesArgs &a, const int64_t *off, int64_t g)
{
    const int64_t b = owner(off, a.req, g, 0);
    const int64_t need = blocks_of(a.lens[b], a.block);      // b gives back: need < held <= max_blocks
    return a.table[b * a.ts + need + (g - off[2 * b])];
}

__global__ __launch_bounds__(tune::kMoveBlock) void k_tables_move(TablesArgs a)
{
    const int64_t *off = offsets_of(a);
    const int32_t *held = held_of(a);
    const int64_t taken = a.offsets[0], given = a.offsets[1], there = a.offsets[2], head = a.offsets[3];
    const int64_t stride = int64_t(gridDim.x) * tune::kMoveBlock;
    for (int64_t i = int64_t(blockIdx.x) * tune::kMoveBlock + threadIdx.x; i < taken + given; i += stride) {
        if (i < taken) {
            int32_t id;
            if (i < there) {
                int64_t at = head + i;
                at = at >= a.ring_size ? at - a.ring_size : at;
                id = a.ring[at];
            } else {
                id = given_id(a, off, i - there);
            }
            const int64_t b = owner(off, a.req, i, 1);
            a.table[b * a.ts + held[b] + (i - off[2 * b + 1])] = id;
        } else {
            const int64_t g = i - taken;
            int64_t at = head + there + g;    // < 2 * ring_size
            at = at >= a.ring_size ? at - a.ring_size : at;
            a.ring[at] = given_id(a, off, g);
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


// Exclusive saturating scan over a block; total: the block's sum.
template <int BLOCK>
__device__ __forceinline__ uint32_t block_prefix_sat(uint32_t v, uint32_t *part, uint32_t *total)
{
    constexpr int NW = BLOCK / 64;
    const int lane = lane_id();
    uint32_t incl = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(incl, d);
        if (lane >= d)
            incl = sat_add(incl, o);
    }
    uint32_t excl = __shfl_up(incl, 1);
    if (lane == 0)
        excl = 0;
    const int w = int(threadIdx.x >> 6);
    if (lane == 63)
        part[w] = incl;
    __syncthreads();
    uint32_t before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
        const uint32_t s = part[i];
        if (i < w)
            before = sat_add(before, s);
        sum = sat_add(sum, s);
    }
    *total = sum;
    return sat_add(before, excl);
}

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
        const uint32_t s = sat_add(sum, block_prefix_sat<B>(v, part[turn], &t));
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
        uint32_t at = sat_add(sum, block_prefix_sat<B>(mine, part[turn], &all));
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
template <class Slot, bool LDS>
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
            Words<4>::template store<false>(slots + t, words_of<4>(slot));
            if (a.positions)
                Words<T>::template store<false>(a.positions + t, words_of<T>(pos));
            if (a.requests)
                Words<T>::template store<false>(a.requests + t, words_of<T>(who));
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
        launch_timed(k_slots<Slot, true>, grid, block, (size_t(L.a.req) + 1) * 12, L.stream, L.ev_begin, L.ev_end, L.a);
    } else {
        launch_timed(k_slot_starts, dim3(1), dim3(tune::kScanBlock), 0, L.stream, L.ev_begin, L.ev_end, L.a);
        launch_timed(k_slots<Slot, false>, grid, block, 0, L.stream, nullptr, nullptr, L.a);
    }
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

}  // namespace

int launch_tables(const TablesLaunch &L)
{
    launch_timed(k_tables_scan, dim3(1), dim3(tune::kScanBlock), 0, L.stream, L.ev_begin, L.ev_end, L.a);
    launch_timed(k_tables_move, dim3(uint32_t(L.grid)), dim3(tune::kMoveBlock), 0, L.stream, nullptr, nullptr, L.a);
    return hipGetLastError() == hipSuccess ? ST_OK : ST_HIP;
}

int launch_slots(const SlotLaunch &L)
{
    return L.slot_dtype == I64 ? run_slots<int64_t>(L) : run_slots<int32_t>(L);
}

}  // namespace rk
