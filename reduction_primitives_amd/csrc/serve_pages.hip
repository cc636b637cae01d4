// serve_pages.hip -- blocks of a paged cache that several rows name: block tables
// forked to a beam search's next rows, compacted, and the blocks copied.
//
// fork_blocks.  Row r of the new table is what row parents[r] was.  A row with a
// child is alive, and its first child keeps all of its blocks, so what falls
// free are the blocks that only rows without children name.  The first launch
// copies the rows and marks the dead rows' entries, the second lets every dead
// entry claim its block for the lowest entry's number while rows alive store 0
// (no order matters: the least value stays), the third counts what each row
// gives back, and in the fourth every block scans these counts, and the rows
// that want a fresh block, for itself, as the block tables do.  Most entries of
// a request's beams are shared at the same position: an entry that the nearest
// row alive before it, or for a dead row the nearest dead one, names at the
// same position is settled without touching the blocks' words.
//
// compact_blocks.  A flag for each id in use, packed to 64-bit words with the
// number of ids in use before each: the rank of any id is then two loads and a
// population count, and the k-th used id beyond their number u and the k-th
// free one below it are what their own ranks say, so no search is needed.
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

// The entries of one segment of a row, `of` the row's length: f(j, there), all
// lanes at a time, j rising.
template <class F>
__device__ __forceinline__ void for_segment(int seg, int of, F &&f)
{
    const int from = seg * kSeg, to = from + kSeg < of ? from + kSeg : of;
    for (int j = from; j < to; j += 64)
        f(j + lane_id(), j + lane_id() < to);
}

// Rows near a row whose entries at the same position settle its own: the
// nearest row alive before it, and the nearest dead one.
struct Near {
    static constexpr int kReach = 16;
    int64_t alive = -1, dead = -1;
    int alive_held = 0, dead_held = 0;

    template <class First>
    __device__ __forceinline__ Near(const ForkArgs &a, int64_t row, First &&first)
    {
        for (int64_t p = row - 1; p >= 0 && p >= row - kReach && (alive < 0 || dead < 0); --p) {
            const bool live = first(p) != kNoChild;
            if (live && alive < 0) {
                alive = p;
                alive_held = clamp_held(a.held[p], a.max_blocks);
            } else if (!live && dead < 0) {
                dead = p;
                dead_held = clamp_held(a.held[p], a.max_blocks);
            }
        }
    }
    __device__ __forceinline__ bool alive_names(const ForkArgs &a, int j, int32_t id) const
    {
        return j < alive_held && a.table[alive * a.ts + j] == id;
    }
    __device__ __forceinline__ bool dead_names(const ForkArgs &a, int j, int32_t id) const
    {
        return j < dead_held && a.table[dead * a.ts + j] == id;
    }
};

__device__ __forceinline__ bool in_pool(const ForkArgs &a, int32_t id) { return id >= 0 && id < a.n_blocks; }

__device__ __forceinline__ uint32_t entry_number(const ForkArgs &a, int64_t row, int j)
{
    return uint32_t(row * a.max_blocks + j) + 1;
}

// Whether a dead row's entry may give its block back: nothing near settles it.
__device__ __forceinline__ bool may_give(const ForkArgs &a, const Near &n, int j, int32_t id)
{
    return in_pool(a, id) && !n.alive_names(a, j, id) && !n.dead_names(a, j, id);
}

__device__ __forceinline__ bool gives(const ForkArgs &a, const Near &n, int64_t row, int j, bool there, int32_t *id)
{
    if (!there)
        return false;
    *id = a.table[row * a.ts + j];
    return may_give(a, n, j, *id) && a.owner[*id] == entry_number(a, row, j);
}

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
        for (int r = int(threadIdx.x); r < a.rows_out; r += kB) {
            const int64_t p = a.parents[r];
            if (p >= 0 && p < a.rows)
                atomicMin(s_child + p, r);
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
    const int64_t items = a.rows_out * a.segs, more = a.rows * a.segs;
    for (int64_t i = wave_number(); i < items + more; i += wave_count()) {
        if (i < items) {
            const int64_t r = i / a.segs;
            const Child c = child_of(a, r, first);
            const int32_t *from = a.table + (c.parent < 0 ? 0 : c.parent) * a.ts;
            int32_t *to = a.table_out + r * a.tos;
            for_segment(int(i - r * a.segs), c.keep, [&](int j, bool there) {
                if (there)
                    to[j] = from[j];
            });
        } else {
            const int64_t row = (i - items) / a.segs;
            if (first(row) != kNoChild)
                continue;
            const Near n(a, row, first);
            for_segment(int(i - items - row * a.segs), clamp_held(a.held[row], a.max_blocks), [&](int j, bool there) {
                const int32_t id = there ? a.table[row * a.ts + j] : -1;
                if (may_give(a, n, j, id))
                    a.owner[id] = 0xffffffffu;
            });
        }
    }
}

__global__ __launch_bounds__(kB) void k_fork_claim(ForkArgs a)
{
    const auto first = [&](int64_t p) { return a.child[p]; };
    for (int64_t i = wave_number(); i < a.rows * a.segs; i += wave_count()) {
        const int64_t row = i / a.segs;
        const int seg = int(i - row * a.segs), held = clamp_held(a.held[row], a.max_blocks);
        const Near n(a, row, first);
        const bool alive = first(row) != kNoChild;
        for_segment(seg, held, [&](int j, bool there) {
            const int32_t id = there ? a.table[row * a.ts + j] : -1;
            if (!in_pool(a, id) || n.alive_names(a, j, id))
                return;
            if (alive)
                __hip_atomic_store(a.owner + id, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            else if (!n.dead_names(a, j, id))
                __hip_atomic_fetch_min(a.owner + id, entry_number(a, row, j), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        });
    }
}

__global__ __launch_bounds__(kB) void k_fork_count(ForkArgs a)
{
    const auto first = [&](int64_t p) { return a.child[p]; };
    for (int64_t i = wave_number(); i < a.rows * a.segs; i += wave_count()) {
        const int64_t row = i / a.segs;
        if (first(row) != kNoChild)
            continue;
        const Near n(a, row, first);
        int32_t sum = 0;
        for_segment(int(i - row * a.segs), clamp_held(a.held[row], a.max_blocks), [&](int j, bool there) {
            int32_t id;
            sum += __popcll(__ballot(gives(a, n, row, j, there, &id)));
        });
        if (lane_id() == 0) {
            a.parts[i] = sum;
            if (sum)
                __hip_atomic_fetch_add(a.gives + row, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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

// Many rows: one block's sums for all.
__global__ __launch_bounds__(tune::kScanBlock) void k_fork_plan(ForkArgs a)
{
    __shared__ int32_t part[tune::kScanBlock / 64];
    const auto first = [&](int64_t p) { return a.child[p]; };
    const int32_t given = scan_counts<tune::kScanBlock>(a.rows, [&](int64_t r) { return a.gives[r]; }, a.gives, part);
    const int32_t wanted = scan_counts<tune::kScanBlock>(a.rows_out, [&](int64_t r) { return int32_t(child_of(a, r, first).wants); },
                                                         a.takes, part);
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
    const auto first = [&](int64_t p) { return a.child[p]; };
    int64_t given, wanted;
    int32_t *s_gives = s_sums, *s_takes = s_sums + a.rows;
    if constexpr (LDS) {
        given = scan_counts<kB>(a.rows, [&](int64_t r) { return a.gives[r]; }, s_gives, part);
        wanted = scan_counts<kB>(a.rows_out, [&](int64_t r) { return int32_t(child_of(a, r, first).wants); }, s_takes, part);
    } else {
        given = a.totals[0];
        wanted = a.totals[1];
    }
    const auto gives_before = [&](int64_t r) { return int64_t(LDS ? s_gives[r] : a.gives[r]); };
    const auto takes_before = [&](int64_t r) { return int64_t(LDS ? s_takes[r] : a.takes[r]); };
    const int64_t head = a.totals[2], tail = a.totals[3];
    const Ring ring(head, tail, a.ring_size, given, wanted);

    if (given > 0)
        for (int64_t i = wave_number(); i < a.rows * a.segs; i += wave_count()) {
            const int64_t row = i / a.segs;
            const int seg = int(i - row * a.segs);
            if (first(row) != kNoChild || seg * kSeg >= clamp_held(a.held[row], a.max_blocks) || a.parts[i] == 0)
                continue;
            const Near n(a, row, first);
            int64_t g = gives_before(row);
            for (int s = 0; s < seg; ++s)
                g += a.parts[row * a.segs + s];
            for_segment(seg, clamp_held(a.held[row], a.max_blocks), [&](int j, bool there) {
                int32_t id = -1;
                const bool out = gives(a, n, row, j, there, &id);
                const uint64_t m = __ballot(out);
                const int64_t at = g + __popcll(m & ((uint64_t(1) << lane_id()) - 1));
                if (out && at < ring.given)
                    a.ring[wrap(ring.head + ring.there + at, a.ring_size)] = id;   // (head + there + given <= head + size)
                g += __popcll(m);
            });
        }

    // the id of give number g, found by a whole wave (g the same in all lanes)
    const auto given_id = [&](int64_t g) {
        int64_t row = 0, hi = a.rows;          // the last row with at most g given before it
        while (hi - row > 1) {
            const int64_t mid = row + ((hi - row) >> 1);
            if (gives_before(mid) <= g)
                row = mid;
            else
                hi = mid;
        }
        int64_t k = g - gives_before(row);
        int seg = 0;
        while (seg + 1 < a.segs && k >= a.parts[row * a.segs + seg]) {
            k -= a.parts[row * a.segs + seg];
            ++seg;
        }
        const Near n(a, row, first);
        int32_t found = -1;
        for_segment(seg, clamp_held(a.held[row], a.max_blocks), [&](int j, bool there) {
            int32_t id = -1;
            const bool out = gives(a, n, row, j, there, &id);
            const uint64_t m = __ballot(out);
            const bool it = out && k == __popcll(m & ((uint64_t(1) << lane_id()) - 1));
            const uint64_t at = __ballot(it);
            if (at)
                found = read_lane(id, __builtin_ctzll(at));
            k -= __popcll(m);
        });
        return found;
    };
    for (int64_t r0 = wave_number() * 64; r0 < a.rows_out; r0 += wave_count() * 64) {
        const int64_t r = r0 + lane_id();
        Child c{-1, 0, 0, 0, false, false};
        int32_t fresh = -1;
        int64_t t = 0;
        bool got = false;
        if (r < a.rows_out) {
            c = child_of(a, r, first);
            t = takes_before(r);
            got = c.wants && t < ring.taken;
            if (got && t < ring.there)
                fresh = a.ring[wrap(ring.head + t, a.ring_size)];
        }
        for (uint64_t rest = __ballot(got && t >= ring.there); rest; rest &= rest - 1) {
            const int l = __builtin_ctzll(rest);
            const int32_t id = given_id(read_lane(t, l) - ring.there);
            if (lane_id() == l)
                fresh = id;
        }
        if (r < a.rows_out) {
            a.held_out[r] = c.keep + got;
            a.lens_out[r] = c.len;
            a.pairs[2 * r] = got ? a.table[c.parent * a.ts + c.keep] : -1;
            a.pairs[2 * r + 1] = got ? fresh : -1;
            if (got)
                a.table_out[r * a.tos + c.keep] = fresh;
        }
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
    for (int64_t i = wave_number(); i < a.rows * a.segs; i += wave_count()) {
        const int64_t row = i / a.segs;
        for_segment(int(i - row * a.segs), clamp_held(a.held[row], a.max_blocks), [&](int j, bool there) {
            const int32_t id = there ? a.table[row * a.ts + j] : -1;
            if (id >= 0 && id < a.n_blocks)
                a.used[id] = 1;
        });
    }
}

// Flags to words, a chunk of kCompactChunk ids a block.
__global__ __launch_bounds__(kB) void k_compact_pack(CompactArgs a)
{
    constexpr int kWords = tune::kCompactChunk / 64, kEach = kWords / (kB / 64);
    __shared__ int32_t counts[kWords];
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int64_t base = int64_t(blockIdx.x) * tune::kCompactChunk, word = int64_t(blockIdx.x) * kWords;
#pragma unroll 4
    for (int i = 0; i < kEach; ++i) {
        const int w = wave * kEach + i;
        const uint64_t m = __ballot(a.used[base + w * 64 + lane_id()] != 0);
        if (lane_id() == 0) {
            a.bits[word + w] = m;
            counts[w] = __popcll(m);
        }
    }
    __syncthreads();
    static_assert(kWords == 64, "one wave scans a chunk's words");
    if (wave == 0) {
        const int32_t incl = wave_prefix<Plus>(counts[lane_id()]);
        a.before[word + lane_id()] = uint16_t(incl - counts[lane_id()]);
        if (lane_id() == 63)
            a.chunk[blockIdx.x] = incl;
    }
}

__global__ __launch_bounds__(tune::kScanBlock) void k_compact_scan(CompactArgs a)
{
    __shared__ int32_t part[tune::kScanBlock / 64];
    const int32_t all = scan_counts<tune::kScanBlock>(a.chunks, [&](int64_t c) { return a.chunk[c]; }, a.chunk, part);
    if (threadIdx.x == 0)
        a.chunk[a.chunks] = all;
}

// Blocks in use below an id (0 <= id < chunks * kCompactChunk).
__device__ __forceinline__ int64_t rank_of(const CompactArgs &a, int64_t id, uint64_t *word)
{
    *word = a.bits[id >> 6];
    return int64_t(a.chunk[id / tune::kCompactChunk]) + a.before[id >> 6] + __popcll(*word & ((uint64_t(1) << (id & 63)) - 1));
}

__device__ __forceinline__ int64_t used_below(const CompactArgs &a, int64_t id)
{
    uint64_t w;
    return id < a.n_blocks ? rank_of(a, id, &w) : a.chunk[a.chunks];
}

// The moves, and the ring of what is free after them.
__global__ __launch_bounds__(kB) void k_compact_pairs(CompactArgs a)
{
    const int64_t u = a.chunk[a.chunks], kept = used_below(a, u), moves = u - kept;
    for (int64_t id = int64_t(blockIdx.x) * kB + threadIdx.x; id < a.n_blocks; id += int64_t(gridDim.x) * kB) {
        uint64_t w;
        const int64_t r = rank_of(a, id, &w);
        const bool used = (w >> (id & 63)) & 1;
        if (used && id >= u)
            a.pairs[2 * (r - kept)] = int32_t(id);
        else if (!used && id < u)
            a.pairs[2 * (id - r) + 1] = int32_t(id);
        if (id >= u)
            a.ring[id - u] = int32_t(id);
    }
    for (int64_t k = moves + int64_t(blockIdx.x) * kB + threadIdx.x; k < a.max_pairs; k += int64_t(gridDim.x) * kB) {
        a.pairs[2 * k] = -1;
        a.pairs[2 * k + 1] = -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.state_out[0] = 0;
        a.state_out[1] = a.n_blocks - u;
        a.state_out[2] = moves;
        a.state_out[3] = 0;
    }
}

__global__ __launch_bounds__(kB) void k_compact_tables(CompactArgs a)
{
    const int64_t u = a.chunk[a.chunks], kept = used_below(a, u);
    for (int64_t i = wave_number(); i < a.rows * a.segs; i += wave_count()) {
        const int64_t row = i / a.segs;
        for_segment(int(i - row * a.segs), clamp_held(a.held[row], a.max_blocks), [&](int j, bool there) {
            if (!there)
                return;
            int32_t id = a.table[row * a.ts + j];
            if (id >= u && id < a.n_blocks) {
                uint64_t w;
                id = a.pairs[2 * (rank_of(a, id, &w) - kept) + 1];
            }
            a.table_out[row * a.tos + j] = id;
        });
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
    const int64_t old = a.rows * a.segs, items = old + a.rows_out * a.segs;
    const dim3 grid(uint32_t(blocks_for(items, L.grid))), grid_old(uint32_t(blocks_for(old, L.grid)));
    const int64_t moving = old > (a.rows_out + 63) / 64 ? old : (a.rows_out + 63) / 64;
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
    const dim3 block(kB), rows(uint32_t(blocks_for(a.rows * a.segs, L.grid)));
    const dim3 ids(uint32_t(blocks_for((a.n_blocks + 63) / 64, L.grid)));
    launch_timed(k_compact_clear, ids, block, 0, L.stream, L.ev_begin, L.ev_end, a);
    hipLaunchKernelGGL(k_compact_mark, rows, block, 0, st, a);
    if (a.chunks > 0)
        hipLaunchKernelGGL(k_compact_pack, dim3(uint32_t(a.chunks)), block, 0, st, a);
    hipLaunchKernelGGL(k_compact_scan, dim3(1), dim3(tune::kScanBlock), 0, st, a);
    hipLaunchKernelGGL(k_compact_pairs, ids, block, 0, st, a);
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
