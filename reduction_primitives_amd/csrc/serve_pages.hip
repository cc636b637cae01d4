// serve_pages.hip -- blocks of a paged cache that several rows name: block tables
// forked to a beam search's next rows, compacted, and the blocks copied.
//
// fork_blocks.  Row r of the new table is what row parents[r] was.  A row with a
// child is alive, and its first child keeps all of its blocks, so what falls
// free are the blocks that only rows without children name.  The first launch
// copies the rows and marks the dead rows' entries, the second lets every dead
// entry claim its block for the lowest entry's number while rows alive store 0
// (no order matters: the least value stays), the third keeps a bit for each entry
// that gives its block back and counts them by row, and in the fourth every block
// scans these counts, and the rows that want a fresh block, for itself, as the
// block tables do.  Most entries of a request's beams are shared at the same
// position: an entry that the nearest row alive before it, or for a dead row the
// nearest dead one, names at the same position is settled without touching the
// block's word.  A wave holds 64 positions of eight rows, so the table is read
// once a launch.  256 rows of 4 k tokens: 5 + 6 + 4 + 5 us, latency; 2048 rows of
// 64 k tokens: 23 + 34 + 15 + 17 us, bound by the words' single stores and loads
// all over the pool (with a store that is no atomic one the second took 44 us,
// with a byte for alive beside the word 30, but the first and third 11 more).
//
// compact_blocks.  A flag for each id in use, packed to words of 64 bits with the
// number of ids in use before each: the rank of any id is then one load and a
// population count, and the k-th used id beyond their number u and the k-th
// free one below it are what their own ranks say, so no search is needed.
// Entries that the row before names at the same position are marked and looked up
// once.  Up to 65536 ids every block packs and ranks for itself: 256 rows of 4 k
// tokens take 2 + 3 + 8 us in three launches, latency (2 + 3 + 3 + 6 + 5 in five);
// 4096 rows of 16 k tokens in a pool of 4 times what is used: 4 + 16 + 4 + 12 + 18
// us, bound by single bytes and words all over the pool (each row by itself, with
// three loads a rank: 5 + 24 + 7 + 10 + 32 and a launch for the sums).
//
// copy_blocks.  Pairs are read 256 at a time, those that name blocks kept in LDS
// in their order and dealt to the `parts` thread blocks that read the same ones.
#define RK_UNIT unit_serve_pages
#include "rk_serve_device.hpp"

namespace rk {
namespace {

constexpr int kB = tune::kPageBlock;
constexpr int kSeg = tune::kPageSeg;
constexpr int32_t kNoChild = 0x7fffffff;

__device__ __forceinline__ int clamp_held(int held, int width) { return held < 0 ? 0 : held < width ? held : width; }

__device__ __forceinline__ int64_t wave_number() { return (int64_t(blockIdx.x) * kB + __builtin_amdgcn_readfirstlane(int(threadIdx.x))) >> 6; }
__device__ __forceinline__ int64_t wave_count() { return int64_t(gridDim.x) * (kB / 64); }

// ----------------------------------------------------------------------- fork

// A new row's parent and what it has of it.
struct Child {
    int64_t parent;           // -1: none
    int held, keep;           // blocks of the parent; of these, those that the row names itself
    int len;
    bool first, wants;        // wants: one more block after those, its own copy of the parent's number `keep`
};

template <class First>
__device__ __forceinline__ Child child_of(const ForkArgs &a, int64_t r, First &&first)
{
    Child c{-1, 0, 0, 0, false, false};
    const int64_t p = a.parents[r];
    if (p < 0 || p >= a.rows)
        return c;
    c.parent = p;
    c.held = clamp_held(a.held[p], a.max_blocks);
    c.len = a.lens[p] < 0 ? 0 : a.lens[p];
    c.first = first(p) == r;
    const int full = int(divide(uint32_t(c.len), a.block));
    c.wants = !c.first && uint32_t(full) * a.block.d != uint32_t(c.len) && full < c.held;
    c.keep = c.first || full > c.held ? c.held : full;
    return c;
}

__device__ __forceinline__ int low_lane(uint64_t lanes) { return __builtin_ctzll(lanes); }
__device__ __forceinline__ uint64_t lanes_before(int l) { return (uint64_t(1) << l) - 1; }

constexpr int kRows = tune::kPageRows;

// The 64 entries at the same positions of kRows rows in a row, all on their way at
// once: id[r] is entry col of row row0 + r, -1 where it names no block of the pool.
// (Wider tiles are longer code that runs once: 256 entries took 14 us where these
// take 5, at 256 rows.)
struct Tile {
    int64_t row0;
    int seg, n, col;                           // n: rows that there are
    int32_t id[kRows];

    __device__ __forceinline__ Tile(int64_t item, int64_t rows, int segs)
        : row0(int64_t(uint32_t(item) / uint32_t(segs)) * kRows), seg(int(uint32_t(item) % uint32_t(segs))),
          n(int(rows - row0 < kRows ? rows - row0 : kRows)), col(seg * 64 + lane_id()) {}
    template <class Args>
    __device__ __forceinline__ int32_t read(const Args &a, int64_t row, int held) const
    {
        return col < held ? a.table[row * a.ts + col] : -1;
    }
    template <class Args>
    static __device__ __forceinline__ int32_t in_pool(const Args &a, int32_t v)
    {
        asm volatile("" : "+v"(v));            // (the loads stay before the first of these, together)
        return v >= 0 && v < a.n_blocks ? v : -1;
    }
    // held: of row row0 + r in lane lane0 + r
    template <class Args>
    __device__ __forceinline__ void load(const Args &a, int held, int lane0)
    {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            id[r] = read(a, r < n ? row0 + r : 0, r < n ? read_lane(held, lane0 + r) : 0);
    }
    template <class Args>
    __device__ __forceinline__ void settle(const Args &a)
    {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            id[r] = in_pool(a, id[r]);
    }
};

// A tile of the old rows, and what the nearest rows before it name at the same
// positions: an entry that a row alive before its own names there too, or for a dead
// row a dead one, is settled without touching the block's word.  Every launch goes
// through the same tiles, so that it takes the same entries for settled.
struct Old : Tile {
    static constexpr int kLane0 = 64 - kRows;  // lanes before: rows before the tile
    uint64_t live, dead;                       // of the rows, as lanes
    int held;
    int32_t by_live, by_dead;

    template <class First>
    __device__ __forceinline__ Old(const ForkArgs &a, int64_t item, First &&first) : Tile(item, a.rows, a.segs)
    {
        const int64_t p = row0 - kLane0 + lane_id();
        const bool there = p >= 0 && p < a.rows;
        const int32_t child = there ? first(p) : 0;
        held = there ? clamp_held(a.held[p], a.max_blocks) : 0;
        live = __ballot(there && child != kNoChild);
        dead = __ballot(there && child == kNoChild);
    }
    __device__ __forceinline__ bool any_dead() const { return (dead >> kLane0) != 0; }
    __device__ __forceinline__ void load(const ForkArgs &a)
    {
        Tile::load(a, held, kLane0);
        const uint64_t l = live & lanes_before(kLane0), d = dead & lanes_before(kLane0);
        const int at_l = l ? 63 - __builtin_clzll(l) : 0, at_d = d ? 63 - __builtin_clzll(d) : 0;
        by_live = read(a, l ? row0 - kLane0 + at_l : 0, l ? read_lane(held, at_l) : 0);
        by_dead = read(a, d ? row0 - kLane0 + at_d : 0, d ? read_lane(held, at_d) : 0);
        settle(a);
        by_live = in_pool(a, by_live);
        by_dead = in_pool(a, by_dead);
    }
    // alive(id): entries of rows alive that are not settled; dying(r, id, may): all of dead rows, may: not settled
    template <class Alive, class Dying>
    __device__ __forceinline__ void walk(Alive &&alive, Dying &&dying)
    {
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int32_t v = id[r];
            const bool fresh = v >= 0 && v != by_live;
            if (live >> (kLane0 + r) & 1) {
                if (fresh)
                    alive(v);
                by_live = v >= 0 ? v : by_live;
            } else {
                dying(r, v, fresh && v != by_dead);
                by_dead = v >= 0 ? v : by_dead;
            }
        }
    }
    __device__ __forceinline__ uint32_t number(const ForkArgs &a, int r) const
    {
        return uint32_t((row0 + r) * a.max_blocks + col) + 1;
    }
};

__device__ __forceinline__ int64_t tiles_of(int64_t rows, int segs) { return (rows + kRows - 1) / kRows * segs; }

__global__ __launch_bounds__(kB) void k_fork_clear(ForkArgs a)
{
    for (int64_t r = int64_t(blockIdx.x) * kB + threadIdx.x; r < a.rows; r += int64_t(gridDim.x) * kB)
        a.child[r] = kNoChild;
}

__global__ __launch_bounds__(kB) void k_fork_children(ForkArgs a)
{
    for (int64_t r = int64_t(blockIdx.x) * kB + threadIdx.x; r < a.rows_out; r += int64_t(gridDim.x) * kB) {
        const int64_t p = a.parents[r];
        if (p >= 0 && p < a.rows)
            __hip_atomic_fetch_min(a.child + p, int32_t(r), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// New rows' entries; dead rows' blocks unclaimed.
template <bool LDS>
__global__ __launch_bounds__(kB) void k_fork_rows(ForkArgs a)
{
    extern __shared__ int32_t s_child[];
    if constexpr (LDS) {
        for (int r = int(threadIdx.x); r < a.rows; r += kB)
            s_child[r] = kNoChild;
        __syncthreads();
        constexpr int kAhead = 8;
        for (int r0 = int(threadIdx.x); r0 < a.rows_out; r0 += kAhead * kB) {
            int32_t p[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                p[k] = a.parents[r0 + k * kB < a.rows_out ? r0 + k * kB : r0];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (r0 + k * kB < a.rows_out && p[k] >= 0 && p[k] < a.rows)
                    atomicMin(s_child + p[k], r0 + k * kB);
        }
        __syncthreads();
    }
    const auto first = [&](int64_t p) { return LDS ? s_child[p] : a.child[p]; };
    for (int64_t r = int64_t(blockIdx.x) * kB + threadIdx.x; r < a.rows; r += int64_t(gridDim.x) * kB) {
        if constexpr (LDS)
            a.child[r] = s_child[r];
        a.gives[r] = 0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) { // (the last launch may write them)
        a.totals[2] = a.state[0];
        a.totals[3] = a.state[1];
    }
    const int segs = a.max_blocks > kSeg ? (a.max_blocks + kSeg - 1) / kSeg : 1;
    const int64_t tiles = tiles_of(a.rows, a.segs), items = tiles + a.rows_out * segs;
    for (int64_t i = wave_number(); i < items; i += wave_count()) {
        if (i < tiles) {
            Old t(a, i, first);
            if (!t.any_dead())
                continue;
            t.load(a);
            t.walk([](int32_t) {}, [&](int, int32_t id, bool may) {
                if (may)
                    a.owner[id] = 0xffffffffu;
            });
            continue;
        }
        const int64_t r = uint32_t(i - tiles) / uint32_t(segs);
        const int seg = int(uint32_t(i - tiles) % uint32_t(segs)), from = seg * kSeg;
        const Child c = child_of(a, r, first);
        const int32_t *src = a.table + (c.parent < 0 ? 0 : c.parent) * a.ts;
        int32_t *dst = a.table_out + r * a.tos;
        const int to = c.keep < from + kSeg ? c.keep : from + kSeg;
        constexpr int kAhead = 8;
        for (int j0 = from + lane_id(); j0 < to; j0 += kAhead * 64) {
            int32_t v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                v[k] = src[j0 + k * 64 < to ? j0 + k * 64 : j0];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (j0 + k * 64 < to)
                    dst[j0 + k * 64] = v[k];
        }
        if (seg == 0 && lane_id() == 0) {
            a.held_out[r] = c.keep;            // (its block of its own comes with the last launch)
            a.lens_out[r] = c.len;
            a.takes[r] = c.wants;
        }
    }
}

__global__ __launch_bounds__(kB) void k_fork_claim(ForkArgs a)
{
    const auto first = [&](int64_t p) { return a.child[p]; };
    const int64_t tiles = tiles_of(a.rows, a.segs);
    for (int64_t i = wave_number(); i < tiles; i += wave_count()) {
        Old t(a, i, first);
        t.load(a);
        t.walk([&](int32_t id) { __hip_atomic_store(a.owner + id, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); },
               [&](int r, int32_t id, bool may) {
                   if (may)
                       __hip_atomic_fetch_min(a.owner + id, t.number(a, r), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
               });
    }
}

// What is given back: a bit for each entry, and their number.
__global__ __launch_bounds__(kB) void k_fork_count(ForkArgs a)
{
    const auto first = [&](int64_t p) { return a.child[p]; };
    const int64_t tiles = tiles_of(a.rows, a.segs);
    const int lane = lane_id();
    for (int64_t i = wave_number(); i < tiles; i += wave_count()) {
        Old t(a, i, first);
        uint64_t mine = 0;                     // of row row0 + lane
        if (t.any_dead()) {
            t.load(a);
            uint32_t owner[kRows];             // of what is not settled, all on their way at once
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                owner[r] = 0;
            t.walk([](int32_t) {}, [&](int r, int32_t id, bool may) {
                if (may)
                    owner[r] = a.owner[id];
            });
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                asm volatile("" : "+v"(owner[r]));
                const uint64_t m = __ballot(owner[r] == t.number(a, r));
                mine = lane == r ? m : mine;
            }
        }
        if (lane < t.n) {
            a.masks[(t.row0 + lane) * a.segs + t.seg] = mine;
            if (mine)
                __hip_atomic_fetch_add(a.gives + t.row0 + lane, __popcll(mine), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
}

// Exclusive sums of n counts, count(i), into to[i]; the whole sum in every thread.
template <int BLOCK, class Count, class To>
__device__ __forceinline__ int32_t scan_counts(int64_t n, Count &&count, To *to, int32_t *part)
{
    const int64_t each = (n + BLOCK - 1) / BLOCK, from = int64_t(threadIdx.x) * each < n ? int64_t(threadIdx.x) * each : n,
                  end = from + each < n ? from + each : n;
    int32_t sum = 0, total;
    for (int64_t i = from; i < end; ++i)
        sum += count(i);
    int32_t run = block_prefix<BLOCK>(sum, part, &total);
    for (int64_t i = from; i < end; ++i) {
        const int32_t v = count(i);
        to[i] = run;
        run += v;
    }
    __syncthreads();
    return total;
}

// Counts read into LDS, several at once.
__device__ __forceinline__ void counts_to(int32_t *to, const int32_t *from, int n)
{
    constexpr int kAhead = 8;
    for (int i0 = int(threadIdx.x); i0 < n; i0 += kAhead * kB) {
        int32_t v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            v[k] = from[i0 + k * kB < n ? i0 + k * kB : i0];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i0 + k * kB < n)
                to[i0 + k * kB] = v[k];
    }
}

// Many rows: one block's sums for all.
__global__ __launch_bounds__(tune::kScanBlock) void k_fork_plan(ForkArgs a)
{
    __shared__ int32_t part[tune::kScanBlock / 64];
    const int32_t given = scan_counts<tune::kScanBlock>(a.rows, [&](int64_t r) { return a.gives[r]; }, a.gives, part);
    const int32_t wanted = scan_counts<tune::kScanBlock>(a.rows_out, [&](int64_t r) { return a.takes[r]; }, a.takes, part);
    if (threadIdx.x == 0) {
        a.totals[0] = given;
        a.totals[1] = wanted;
    }
}

// Blocks given back go to the ring, fresh ones come from it.
template <bool LDS>
__global__ __launch_bounds__(kB) void k_fork_move(ForkArgs a)
{
    extern __shared__ int32_t s_sums[];
    __shared__ int32_t part[kB / 64];
    int64_t given, wanted;
    int32_t *s_gives = s_sums, *s_takes = s_sums + a.rows;
    if constexpr (LDS) {
        counts_to(s_gives, a.gives, int(a.rows));
        counts_to(s_takes, a.takes, int(a.rows_out));
        __syncthreads();
        given = scan_counts<kB>(a.rows, [&](int64_t r) { return s_gives[r]; }, s_gives, part);
        wanted = scan_counts<kB>(a.rows_out, [&](int64_t r) { return s_takes[r]; }, s_takes, part);
    } else {
        given = a.totals[0];
        wanted = a.totals[1];
    }
    const auto gives_before = [&](int64_t r) { return int64_t(LDS ? s_gives[r] : a.gives[r]); };
    const auto takes_before = [&](int64_t r) { return int64_t(LDS ? s_takes[r] : a.takes[r]); };
    const int64_t head = a.totals[2], tail = a.totals[3];
    const Ring ring(head, tail, a.ring_size, given, wanted);

    // 64 words of a row a wave, those that give something four at a time
    const int words = (a.segs + 63) / 64;
    if (given > 0)
        for (int64_t i = wave_number(); i < a.rows * words; i += wave_count()) {
            const int64_t row = uint32_t(i) / uint32_t(words), base = row * a.segs;
            const int seg0 = int(uint32_t(i) % uint32_t(words)) * 64;
            const uint64_t m = seg0 + lane_id() < a.segs ? a.masks[base + seg0 + lane_id()] : 0;
            uint64_t some = __ballot(m != 0);
            if (!some)
                continue;
            int32_t before = 0;
            for (int s = lane_id(); s < seg0; s += 64)
                before += __popcll(a.masks[base + s]);
            const int32_t count = __popcll(m);
            const int64_t g0 = gives_before(row) + (seg0 ? wave_reduce<OpSum>(before) : 0);
            const int32_t g = wave_prefix<Plus>(count) - count;
            while (some) {
                constexpr int kAhead = 4;
                int l[kAhead];
                int32_t id[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    l[k] = some ? low_lane(some) : -1;
                    some &= some - 1;
                    const int j = (seg0 + (l[k] < 0 ? l[0] : l[k])) * 64 + lane_id();
                    id[k] = a.table[row * a.ts + (j < a.max_blocks ? j : 0)];
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const uint64_t mk = l[k] < 0 ? 0 : read_lane(m, l[k] < 0 ? 0 : l[k]);
                    const int64_t at = g0 + read_lane(g, l[k] < 0 ? 0 : l[k]) + __popcll(mk & lanes_before(lane_id()));
                    if ((mk >> lane_id() & 1) && at < ring.given)
                        a.ring[wrap(ring.head + ring.there + at, a.ring_size)] = id[k];   // (head + there + given <= head + size)
                }
            }
        }

    // the id of give number g
    const auto given_id = [&](int64_t g) {
        int64_t row = 0, hi = a.rows;          // the last row with at most g given before it
        while (hi - row > 1) {
            const int64_t mid = row + ((hi - row) >> 1);
            if (gives_before(mid) <= g)
                row = mid;
            else
                hi = mid;
        }
        int64_t k = g - gives_before(row), i = row * a.segs;
        uint64_t m = a.masks[i];
        for (; k >= __popcll(m); m = a.masks[++i])
            k -= __popcll(m);
        for (; k > 0; --k)
            m &= m - 1;
        return a.table[row * a.ts + (i - row * a.segs) * 64 + low_lane(m)];
    };
    for (int64_t r = int64_t(blockIdx.x) * kB + threadIdx.x; r < a.rows_out; r += int64_t(gridDim.x) * kB) {
        const int64_t t = takes_before(r), next = r + 1 < a.rows_out ? takes_before(r + 1) : wanted;
        int32_t from = -1, fresh = -1;
        if (next > t && t < ring.taken) {
            const int keep = a.held_out[r];
            from = a.table[a.parents[r] * a.ts + keep];
            fresh = t < ring.there ? a.ring[wrap(ring.head + t, a.ring_size)] : given_id(t - ring.there);
            a.table_out[r * a.tos + keep] = fresh;
            a.held_out[r] = keep + 1;
        }
        a.pairs[2 * r] = from;
        a.pairs[2 * r + 1] = fresh;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.state_out[0] = head + ring.taken;
        a.state_out[1] = tail + ring.given;
        a.state_out[2] = wanted - ring.taken;
        a.state_out[3] = given - ring.given;
    }
}

// -------------------------------------------------------------------- compact

__global__ __launch_bounds__(kB) void k_compact_clear(CompactArgs a)
{
    const int64_t n = a.chunks * (tune::kCompactChunk / 16);
    for (int64_t i = int64_t(blockIdx.x) * kB + threadIdx.x; i < n; i += int64_t(gridDim.x) * kB)
        reinterpret_cast<u32x4 *>(a.used)[i] = u32x4{0, 0, 0, 0};
}

__global__ __launch_bounds__(kB) void k_compact_mark(CompactArgs a)
{
    const int64_t tiles = tiles_of(a.rows, a.segs);
    for (int64_t i = wave_number(); i < tiles; i += wave_count()) {
        Tile t(i, a.rows, a.segs);
        const int64_t p = t.row0 - 1 + lane_id();
        const int held = p >= 0 && p < a.rows ? clamp_held(a.held[p], a.max_blocks) : 0;
        t.load(a, held, 1);
        int32_t by = t.read(a, t.row0 > 0 ? t.row0 - 1 : 0, read_lane(held, 0));   // (that row's wave marks it)
        t.settle(a);
        by = Tile::in_pool(a, by);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int32_t v = t.id[r];
            if (v >= 0 && v != by)
                a.used[v] = 1;
            by = v >= 0 ? v : by;
        }
    }
}

// Flags to words, a chunk of kCompactChunk ids a block.
__global__ __launch_bounds__(kB) void k_compact_pack(CompactArgs a)
{
    constexpr int kWords = tune::kCompactChunk / 64, kMine = kWords / (kB / 64);
    static_assert(kWords == 64 && kMine == 16, "a wave packs the words whose numbers its lanes 0 .. 15 hold");
    __shared__ int32_t counts[kWords];
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)), lane = lane_id();
    const int64_t base = int64_t(blockIdx.x) * tune::kCompactChunk, word = int64_t(blockIdx.x) * kWords;
    uint8_t flag[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        flag[i] = a.used[base + (wave * kMine + i) * 64 + lane];
    uint64_t mine = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const uint64_t m = __ballot(flag[i] != 0);
        mine = lane == i ? m : mine;
    }
    if (lane < kMine)
        counts[wave * kMine + lane] = __popcll(mine);
    __syncthreads();
    const int32_t count = counts[lane], incl = wave_prefix<Plus>(count), before = incl - count;
    const int32_t at = int32_t(bpermute32(uint32_t(before), wave * kMine + (lane & (kMine - 1))));
    if (lane < kMine)
        a.words[word + wave * kMine + lane] = CompactWord{mine, at, 0};
    if (wave == 0 && lane == 63)
        a.chunk[blockIdx.x] = incl;
}

// Many chunks: one block's sums for all.
__global__ __launch_bounds__(tune::kScanBlock) void k_compact_scan(CompactArgs a)
{
    __shared__ int32_t part[tune::kScanBlock / 64];
    const int32_t all = scan_counts<tune::kScanBlock>(a.chunks, [&](int64_t c) { return a.chunk[c]; }, a.chunk, part);
    if (threadIdx.x == 0)
        a.chunk[a.chunks] = all;
}

// Sums over chunks [0, end) and [0, all), in every thread.
__device__ __forceinline__ int2 sum_chunks(const CompactArgs &a, int64_t end, int64_t all, int2 *part)
{
    int2 v = make_int2(0, 0);
    for (int64_t c = threadIdx.x; c < all; c += kB) {
        const int32_t n = a.chunk[c];
        v.x += c < end ? n : 0;
        v.y += n;
    }
    v = make_int2(wave_reduce<OpSum>(v.x), wave_reduce<OpSum>(v.y));
    __syncthreads();
    if (lane_id() == 0)
        part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
    for (int w = 1; w < kB / 64; ++w)
        v = make_int2(v.x + part[w].x, v.y + part[w].y);
    return v;
}

// The moves, and the ring of what is free after them; each word's rank.  A chunk a block.
template <bool SCANNED>
__global__ __launch_bounds__(kB) void k_compact_pairs(CompactArgs a)
{
    __shared__ int2 part[kB / 64];
    constexpr int kWords = tune::kCompactChunk / 64;
    const int64_t own = blockIdx.x;
    int64_t base, u, kept = 0;                 // used before the chunk; in all; below u
    if constexpr (SCANNED) {
        base = a.chunk[own];
        u = a.chunk[a.chunks];
    } else {
        const int2 v = sum_chunks(a, own, a.chunks, part);
        base = v.x;
        u = v.y;
    }
    if (u < a.n_blocks) {
        const int64_t c = u / tune::kCompactChunk;
        kept = SCANNED ? a.chunk[c] : sum_chunks(a, c, c, part).x;
        const CompactWord w = a.words[u >> 6];
        kept += w.before + __popcll(w.used & lanes_before(int(u & 63)));
    } else {
        kept = u;
    }
    const int64_t moves = u - kept;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)), lane = lane_id();
    const int64_t word0 = own * kWords + wave * (kWords / (kB / 64));
    constexpr int kMine = kWords / (kB / 64);
    if (own < a.chunks) {
        const CompactWord mine = a.words[word0 + (lane & (kMine - 1))];
        const int32_t rank = int32_t(base) + mine.before;
        if (lane < kMine)
            a.words[word0 + lane].rank = rank;
#pragma unroll 4
        for (int i = 0; i < kMine; ++i) {
            const uint64_t m = read_lane(mine.used, i);
            const int64_t r = read_lane(rank, i) + __popcll(m & lanes_before(lane)), id = (word0 + i) * 64 + lane;
            const bool used = m >> lane & 1;
            if (id < a.n_blocks) {
                if (used && id >= u)
                    a.pairs[2 * (r - kept)] = int32_t(id);
                else if (!used && id < u)
                    a.pairs[2 * (id - r) + 1] = int32_t(id);
                if (id >= u)
                    a.ring[id - u] = int32_t(id);
            }
        }
    }
    for (int64_t k = moves + int64_t(blockIdx.x) * kB + threadIdx.x; k < a.max_pairs; k += int64_t(gridDim.x) * kB) {
        a.pairs[2 * k] = -1;
        a.pairs[2 * k + 1] = -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.totals[0] = u;
        a.totals[1] = kept;
        a.state_out[0] = 0;
        a.state_out[1] = a.n_blocks - u;
        a.state_out[2] = moves;
        a.state_out[3] = 0;
    }
}

// (The row before a tile is not looked at: it may have its new ids already.)
__global__ __launch_bounds__(kB) void k_compact_tables(CompactArgs a)
{
    const int64_t u = a.totals[0], kept = a.totals[1], tiles = tiles_of(a.rows, a.segs);
    for (int64_t i = wave_number(); i < tiles; i += wave_count()) {
        Tile t(i, a.rows, a.segs);
        const int64_t p = t.row0 + lane_id();
        const int held = p < a.rows && lane_id() < kRows ? clamp_held(a.held[p], a.max_blocks) : 0;
        t.load(a, held, 0);
        // three rounds of loads, each for all rows at once: entries, their words, their places
        uint64_t used[kRows];
        int32_t rank[kRows], to[kRows], by = -1;
        bool look[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            asm volatile("" : "+v"(t.id[r]));
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int32_t v = t.id[r];
            look[r] = v >= u && v < a.n_blocks && v != by;   // (u >= 0; entries that are not there are -1)
            by = v >= u && v < a.n_blocks ? v : by;
            used[r] = 0;
            rank[r] = 0;
            if (look[r]) {
                used[r] = a.words[v >> 6].used;
                rank[r] = a.words[v >> 6].rank;
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            asm volatile("" : "+v"(used[r]), "+v"(rank[r]));
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            to[r] = 0;
            if (look[r])
                to[r] = a.pairs[2 * (int64_t(rank[r]) + __popcll(used[r] & lanes_before(t.id[r] & 63)) - kept) + 1];
        }
        int32_t last = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int32_t v = t.id[r];
            last = look[r] ? to[r] : last;
            if (t.col < read_lane(held, r))
                a.table_out[(t.row0 + r) * a.tos + t.col] = v >= u && v < a.n_blocks ? last : v;
        }
    }
}

// Small pools, all of it after the marks in one launch: every block packs the flags and
// ranks the words for itself, and finds the k-th free id by bisection.
__global__ __launch_bounds__(kB) void k_compact_own(CompactArgs a)
{
    constexpr int kWords = tune::kCompactOwn / 64, kMine = kWords / kB;
    __shared__ __attribute__((aligned(16))) uint64_t s_used[kWords];
    __shared__ int32_t s_rank[kWords], s_part[kB / 64];
    const int tid = int(threadIdx.x), lane = lane_id(), words = int(a.chunks) * (tune::kCompactChunk / 64);
    {
        constexpr int kAhead = tune::kCompactOwn / 16 / kB;
        u32x4 f[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = tid + k * kB;
            f[k] = reinterpret_cast<const u32x4 *>(a.used)[i < words * 4 ? i : 0];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            uint32_t m = 0;                    // four bytes of 0 or 1 to the bits 24 .. 27 of the product
#pragma unroll
            for (int j = 0; j < 4; ++j)
                m |= (f[k][j] * 0x01020408u >> 24 & 0xf) << (4 * j);
            const int i = tid + k * kB;
            reinterpret_cast<uint16_t *>(s_used)[i] = uint16_t(i < words * 4 ? m : 0);
        }
    }
    __syncthreads();
    int32_t sum = 0, u;
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        sum += __popcll(s_used[tid * kMine + k]);
    int32_t run = block_prefix<kB>(sum, s_part, &u);
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        s_rank[tid * kMine + k] = run;
        run += __popcll(s_used[tid * kMine + k]);
    }
    __syncthreads();
    const auto rank = [&](int id) { return s_rank[id >> 6] + int(__popcll(s_used[id >> 6] & lanes_before(id & 63))); };
    const int n = int(a.n_blocks), kept = u < n ? rank(u) : u, moves = u - kept;
    // the k-th free ids, N at a time
    const auto places = [&](auto &k) {
        constexpr int N = sizeof(k) / sizeof(k[0]);
        int w[N];
#pragma unroll
        for (int r = 0; r < N; ++r)
            w[r] = 0;
#pragma unroll
        for (int d = kWords / 2; d > 0; d /= 2)
#pragma unroll
            for (int r = 0; r < N; ++r)
                w[r] += (w[r] + d) * 64 - s_rank[w[r] + d] <= k[r] ? d : 0;
#pragma unroll
        for (int r = 0; r < N; ++r) {
            uint64_t m = ~s_used[w[r]];
            int left = k[r] - (w[r] * 64 - s_rank[w[r]]), at = 0;
#pragma unroll
            for (int d = 32; d > 0; d /= 2) {
                const int c = __popcll(m & ((uint64_t(1) << d) - 1));
                const bool up = left >= c;
                left -= up ? c : 0;
                at += up ? d : 0;
                m = up ? m >> d : m;
            }
            k[r] = w[r] * 64 + at;
        }
    };
    for (int id = int(blockIdx.x) * kB + tid; id < n; id += int(gridDim.x) * kB) {
        if (id < u)
            continue;
        a.ring[id - u] = id;
        if (s_used[id >> 6] >> (id & 63) & 1) {
            int k[1] = {rank(id) - kept};
            const int64_t pair = 2 * int64_t(k[0]);
            places(k);
            a.pairs[pair] = id;
            a.pairs[pair + 1] = k[0];
        }
    }
    for (int64_t k = moves + int64_t(blockIdx.x) * kB + tid; k < a.max_pairs; k += int64_t(gridDim.x) * kB) {
        a.pairs[2 * k] = -1;
        a.pairs[2 * k + 1] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.state_out[0] = 0;
        a.state_out[1] = n - u;
        a.state_out[2] = moves;
        a.state_out[3] = 0;
    }
    const int64_t tiles = tiles_of(a.rows, a.segs);
    for (int64_t i = wave_number(); i < tiles; i += wave_count()) {
        Tile t(i, a.rows, a.segs);
        const int64_t p = t.row0 + lane;
        const int held = p < a.rows && lane < kRows ? clamp_held(a.held[p], a.max_blocks) : 0;
        t.load(a, held, 0);
        int to[kRows];
        bool moved[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            asm volatile("" : "+v"(t.id[r]));
            moved[r] = t.id[r] >= u && t.id[r] < n;
            to[r] = moved[r] ? rank(t.id[r]) - kept : 0;
        }
        places(to);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (t.col < read_lane(held, r))
                a.table_out[(t.row0 + r) * a.tos + t.col] = moved[r] ? to[r] : t.id[r];
    }
}

// ----------------------------------------------------------------------- copy

typedef u32x4 AnyVec __attribute__((aligned(1)));

__global__ __launch_bounds__(kB) void k_copy(CopyArgs a)
{
    __shared__ int2 s_pair[kB];
    __shared__ int s_counts[kB / 64];
    const CopyCache c = a.cache[blockIdx.y];
    const int part = int(blockIdx.x % uint32_t(a.parts)), wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int64_t from = int64_t(blockIdx.z) * tune::kCopyChunk;
    const int64_t left = c.bytes - from, n = left < tune::kCopyChunk ? left : tune::kCopyChunk;
    if (n <= 0)
        return;
    for (int64_t p0 = int64_t(blockIdx.x / uint32_t(a.parts)) * kB; p0 < a.n_pairs;
         p0 += int64_t(gridDim.x / uint32_t(a.parts)) * kB) {
        const int64_t p = p0 + threadIdx.x;
        int2 q = make_int2(-1, -1);
        if (p < a.n_pairs)
            q = make_int2(a.pairs[2 * p], a.pairs[2 * p + 1]);
        const bool there = q.x >= 0 && q.y >= 0 && q.x < c.blocks && q.y < c.blocks && q.x != q.y;
        const uint64_t m = __ballot(there);
        if (lane_id() == 0)
            s_counts[wave] = __popcll(m);
        __syncthreads();
        int before = 0, count = 0;
        for (int w = 0; w < kB / 64; ++w) {
            before += w < wave ? s_counts[w] : 0;
            count += s_counts[w];
        }
        if (there)
            s_pair[before + __popcll(m & ((uint64_t(1) << lane_id()) - 1))] = q;
        __syncthreads();
        for (int i = part; i < count; i += a.parts) {
            const char *src = c.data + s_pair[i].x * c.stride + from;
            char *dst = c.data + s_pair[i].y * c.stride + from;
            int64_t at = int64_t(threadIdx.x) * 16;
#pragma unroll 4
            for (; at + 16 <= n; at += kB * 16)
                *reinterpret_cast<AnyVec *>(dst + at) = *reinterpret_cast<const AnyVec *>(src + at);
            if (at < n)
                for (int64_t b = at; b < n; ++b)
                    dst[b] = src[b];
        }
        __syncthreads();
    }
}

int64_t blocks_for(int64_t waves, int64_t cap)
{
    const int64_t b = (waves + kB / 64 - 1) / (kB / 64);
    return b < 1 ? 1 : b < cap ? b : cap;
}

bool launched() { return hipGetLastError() == hipSuccess; }

}  // namespace

int launch_fork(const ForkLaunch &L)
{
    const ForkArgs &a = L.a;
    hipStream_t st = static_cast<hipStream_t>(L.stream);
    const dim3 block(kB);
    if (!L.in_lds) {
        const int64_t n = a.rows > a.rows_out ? a.rows : a.rows_out;
        const dim3 grid(uint32_t(blocks_for((n + 63) / 64, L.grid)));
        hipLaunchKernelGGL(k_fork_clear, grid, block, 0, st, a);
        hipLaunchKernelGGL(k_fork_children, grid, block, 0, st, a);
        if (!launched())
            return ST_HIP;
    }
    const int64_t tiles = (a.rows + kRows - 1) / kRows * a.segs, items = tiles + a.rows_out * (a.max_blocks > kSeg ? (a.max_blocks + kSeg - 1) / kSeg : 1);
    const dim3 grid(uint32_t(blocks_for(items, L.grid))), grid_old(uint32_t(blocks_for(tiles, L.grid)));
    const int64_t old = a.rows * ((a.segs + 63) / 64), moving = old > (a.rows_out + 63) / 64 ? old : (a.rows_out + 63) / 64;
    const dim3 grid_move(uint32_t(blocks_for(moving, L.grid)));
    if (L.in_lds)
        launch_timed(k_fork_rows<true>, grid, block, size_t(a.rows) * 4, L.stream, L.ev_begin, L.ev_end, a);
    else
        launch_timed(k_fork_rows<false>, grid, block, 0, L.stream, L.ev_begin, L.ev_end, a);
    hipLaunchKernelGGL(k_fork_claim, grid_old, block, 0, st, a);
    hipLaunchKernelGGL(k_fork_count, grid_old, block, 0, st, a);
    if (L.in_lds) {
        hipLaunchKernelGGL(k_fork_move<true>, grid_move, block, size_t(a.rows + a.rows_out) * 4, st, a);
    } else {
        hipLaunchKernelGGL(k_fork_plan, dim3(1), dim3(tune::kScanBlock), 0, st, a);
        hipLaunchKernelGGL(k_fork_move<false>, grid_move, block, 0, st, a);
    }
    return launched() ? ST_OK : ST_HIP;
}

int launch_compact(const CompactLaunch &L)
{
    const CompactArgs &a = L.a;
    hipStream_t st = static_cast<hipStream_t>(L.stream);
    const dim3 block(kB), rows(uint32_t(blocks_for((a.rows + kRows - 1) / kRows * a.segs, L.grid)));
    const dim3 chunks(uint32_t(a.chunks > 0 ? a.chunks : 1));
    launch_timed(k_compact_clear, chunks, block, 0, L.stream, L.ev_begin, L.ev_end, a);
    hipLaunchKernelGGL(k_compact_mark, rows, block, 0, st, a);
    if (a.n_blocks <= tune::kCompactOwn) {     // (two blocks a CU at most: each reads all flags)
        const int64_t by_id = (a.n_blocks + 63) / 64, by_tile = (a.rows + kRows - 1) / kRows * a.segs;
        hipLaunchKernelGGL(k_compact_own, dim3(uint32_t(blocks_for(by_id > by_tile ? by_id : by_tile, L.grid / 4))), block, 0, st, a);
        return launched() ? ST_OK : ST_HIP;
    }
    if (a.chunks > 0)
        hipLaunchKernelGGL(k_compact_pack, chunks, block, 0, st, a);
    if (a.chunks > tune::kCompactSums) {
        hipLaunchKernelGGL(k_compact_scan, dim3(1), dim3(tune::kScanBlock), 0, st, a);
        hipLaunchKernelGGL(k_compact_pairs<true>, chunks, block, 0, st, a);
    } else {
        hipLaunchKernelGGL(k_compact_pairs<false>, chunks, block, 0, st, a);
    }
    hipLaunchKernelGGL(k_compact_tables, rows, block, 0, st, a);
    return launched() ? ST_OK : ST_HIP;
}

int launch_copy(const CopyLaunch &L)
{
    launch_timed(k_copy, dim3(uint32_t(L.grid_x), uint32_t(L.a.caches), uint32_t(L.a.chunks)), dim3(kB), 0, L.stream,
                 L.ev_begin, L.ev_end, L.a);
    return launched() ? ST_OK : ST_HIP;
}

}  // namespace rk
