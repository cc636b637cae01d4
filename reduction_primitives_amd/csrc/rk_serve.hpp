// rk_serve.hpp -- plans and kernel arguments of the serving operators: softmax
// of lines, verification of drafted tokens, block tables and slot maps.  Pure
// C++ (no HIP), like rk_plan.hpp.
#pragma once

#include <cstddef>
#include <cstdint>

#include "rk_plan.hpp"

namespace rk {
namespace tune {
// ---- softmax of lines
// A line of up to kSoftLanes * kSoftPer entries is one block's (a wave's up to
// 64 * kSoftPer), in one launch; longer ones are split over two.  Measured,
// one block against split: 5 x 8192 f32 3.4 / 5.2 us, 512 x 8192 8.2 / 11.1,
// 128 x 20000 6.5 / 9.5, 512 x 32768 bf16 to f32 20.0 / 21.4, 5 x 32768 5.5 / 5.4;
// with 64 entries a thread 5 x 65536 took 10.9 us against 5.4.
constexpr int kSoftPer = 32;              // entries a thread holds of a line kept in registers
constexpr int kSoftLanes = 1024;          // most threads that share such a line
// Lines of up to this many entries share a wave, 16 lanes each.  Against a wave
// a line: 5 x 64 f32 2.2 / 2.4 us, 16384 x 64 3.4 / 6.7, 100000 x 64 10.2 / 28.8, x 256 38.1 /
// 40.0 (bf16 19.0 / 33.3), x 512 74.1 / 71.0, 5 x 512 2.8 / 2.5.
constexpr int kSoftRowEntries = 256;
constexpr int kSoftBlock = 256;           // threads of a split line's blocks
// Entries of a wave's tile of a split line.  4096: 5 x 131072 f32 6.7 us,
// 320 x 131072 bf16 to f32 49.1; 2048: 5.7, 50.6; 1024: 5.6, 50.5.
constexpr int kSoftTile = 2048;
// Every wave of the writing launch folds its line's statistics, 64 tiles at a
// time, for itself; past this many tiles (a million entries) a launch between
// folds them once a line.
constexpr int kSoftFoldTiles = 512;
// Outputs beyond the eight L2s together (32 MB) are stored past the caches, so
// the input stays there for its second reading: 320 x 131072 bf16 to f32 (168
// MB out) 59.5 us with plain stores, 48.2 us with streaming ones.  Smaller
// ones stay cached for whoever reads the probabilities next.
constexpr int64_t kSoftStreamBytes = int64_t(32) << 20;
// ---- draft verification
constexpr int kVerifyBlock = 256;
constexpr int kVerifyTile = 2048;         // vocabulary entries one wave sums at a time
constexpr int kVerifyBlocksPerCu = 16;    // grid cap = CUs * this (256 x 131072 f32: 8 34.7 us, 16 and 32 32.7)
// Up to a request a CU and this many blocks a CU the last block of a request
// finishes it; beyond, a second launch does, whose blocks do not wait behind
// those that still read.  One launch against two, x 131072 f32: 64 requests 12.5 /
// 13.1 us, 128 19.2 / 19.5, 192 25.0 / 24.6, 256 32.1 / 30.5; bf16: 64 9.8 / 10.7, 128
// 15.1 / 14.9, 256 26.6 / 22.4; x 32000 f32: 64 8.0 / 9.5, 256 13.1 / 13.4, 384 19.6 / 17.7.
constexpr int kVerifyFusedBlocksPerCu = 8;
// ---- block tables and slot maps
constexpr int kScanBlock = 1024;          // threads of the one block that scans a slot map's many requests
constexpr int kMoveBlock = 256;           // threads of the blocks that move block ids
// Ids a lane moves at a time.  2048 requests moving 840,000 ids each way: 1
// 14.0 us, 2 11.5, 4 10.6, 8 12 and more; but a step of decoding, which moves
// few, 5.2 us with 1, 6.2 with 2, 8.2 with 4: it takes 1.
constexpr int kMoveEach = 4;
// Grid cap = CUs * this (two launches: past a wave a request), or what their
// LDS lets run at once: every block scans all requests.  2048 requests: 2 20.8
// us, 4 14.0, 8 16.0; 4096 (48 KB of LDS): 3 10.4, 4 14.4.
constexpr int kMoveBlocksPerCu = 4;
// Requests a one-launch call takes, 12 bytes of LDS each.  Against two
// launches: 64 requests 4.1 / 5.6 us, 1024 5.8 / 6.9, 2048 7.2 / 10.0.
constexpr int kMoveLdsRequests = 4096;
constexpr int kSlotBlock = 256;
// Requests a slot map's blocks keep in LDS (12 bytes each), against a launch of
// its own that scans them: 256 requests 3.9 / 5.2 us, 1024 4.0 / 7.1, 4096 7.0 / 10.7.
constexpr int kSlotLdsRequests = 4096;
constexpr int kSlotBlocksPerCu = 8;       // grid cap = CUs * this, or what their LDS lets run at once
constexpr int kLdsBytes = 160 << 10;      // of a CU
// Outputs beyond the eight L2s together are stored past the caches (3.1M tokens,
// 50 MB: 11.9 us with plain stores, 11.1 us without); smaller ones stay there
// for the kernels that write the cache.
constexpr int64_t kSlotStreamBytes = int64_t(32) << 20;
}  // namespace tune

enum SoftmaxKernel { VK_NONE = 0, VK_SOFT_LINE = 1, VK_SOFT_SPLIT = 2 };

// Division of 0 <= x < 2^31 by d >= 1 as a multiplication: with l the bits
// of d - 1 and m = floor(2^(31+l) / d) + 1, x / d = (x * m) >> (31 + l).
// (m d exceeds 2^(31+l) by e with 1 <= e <= d <= 2^l, so x e < 2^(31+l), and
// m < 2^32 since 2^(l-1) < d for d > 1, so the product fits 64 bits.)
struct Divider {
    uint32_t d;
    uint32_t m;               // d = 1: unused, shift 0
    int shift;
};
Divider make_divider(uint32_t d);

// The last i of [lo, hi) with start(i) <= t, where start does not fall and
// start(lo) <= t.  (lo + hi passes 2^31 from 2^30 requests on.)
template <class Start>
constexpr int last_start(const Start &start, int lo, int hi, int64_t t)
{
    while (hi - lo > 1) {
        const int mid = lo + ((hi - lo) >> 1);
        if (start(mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Blocks of `lds` bytes that a CU runs at once, at most `most`.
constexpr int64_t resident(int64_t lds, int64_t most)
{
    const int64_t fit = tune::kLdsBytes / (lds > 0 ? lds : 1);
    return fit < 1 ? 1 : fit < most ? fit : most;
}

// ------------------------------------------------------------------ softmax

struct SoftmaxPlan {
    int kernel = VK_NONE;
    int64_t grid = 0;         // blocks of the first launch
    int block = 0;
    int launches = 0;
    int lanes = 0;            // threads sharing a line (VK_SOFT_LINE)
    int chunks = 1;           // tiles of a line (VK_SOFT_SPLIT)
    int vec = 1;
    bool fold = false;        // a launch of its own folds the lines' statistics (VK_SOFT_SPLIT)
    bool stream_out = false;  // the writing launch stores past the caches (VK_SOFT_SPLIT)
    size_t ws_bytes = 0;
};

struct SoftmaxArgs {
    const void *x;
    void *out;
    const float *t;           // temperatures, or NULL (1)
    float *stats;             // split: max, sum of every tile of every line, then (fold) of every line
    int32_t *first;           // split: place of the first largest entry in every tile, then (fold) its tile
    bool fold;
    int64_t n, lines, xs, os;
    int chunks;
    Divider per_line;         // split: blocks of a line
};

int plan_softmax(int in_dtype, int out_dtype, int64_t n, int64_t lines, SoftmaxPlan *p);

struct SoftmaxLaunch {
    SoftmaxPlan plan;
    SoftmaxArgs a;
    int in, out;
    void *stream, *ev_begin, *ev_end;
};
int launch_softmax(const SoftmaxLaunch &L);

// ------------------------------------------------------- draft verification

struct VerifyPlan {
    int64_t tiles = 0;        // tiles of a line
    int chunks = 0;           // blocks of a line
    int64_t grid = 0;
    int launches = 0;
    bool fused_ok = false;    // the last block of a request finishes it
    size_t ws_bytes = 0;
};

// What is known of a request once its kept drafts are.
struct VerifyDrawn {
    int64_t lo;               // its first draft
    int64_t x;                // the token turned down (-1: none)
    int count, kept;          // its drafts, and how many are kept
};

struct VerifyArgs {
    const void *p, *q;        // q NULL: drafts without probabilities
    int64_t ps, qs;           // line strides
    int64_t n;                // vocabulary
    int64_t req, drafts;      // requests; drafted tokens of all requests
    int max_draft;
    const int32_t *starts;    // NULL: max_draft drafts for every request
    const void *drafted;
    const float *u, *r;
    void *tokens;
    int32_t *accepted;
    double *sums;             // [req][tiles]
    VerifyDrawn *drawn;       // [req], written for a second launch
    int64_t tiles;
    int chunks;
    int slot;                 // >= 0: the last block of a request finishes it
};

int plan_verify(int prob_dtype, int64_t n, int64_t req, int cus, VerifyPlan *p);

struct VerifyLaunch {
    VerifyPlan plan;
    VerifyArgs a;
    int dtype, token_dtype;
    void *stream, *ev_begin, *ev_end;
};
int launch_verify(const VerifyLaunch &L);

// -------------------------------------------------- block tables, slot maps

// What the first launch of a block_tables call leaves for the second.
struct TablesPlan {
    int64_t give0, take0;     // blocks given back, blocks wanted by the requests before this one
    int32_t held, need;
};
struct TablesTotals {
    int64_t gives, takes;     // blocks given back and wanted in all
    int64_t head, tail;       // of the ring, before the call
};

struct TablesArgs {
    const int32_t *lens, *held;
    int32_t *held_out;
    int64_t req;
    Divider block;
    int32_t *table;
    int64_t ts;               // table stride
    int max_blocks;
    int32_t *ring;
    int64_t ring_size;
    const int64_t *state;
    int64_t *state_out;
    TablesTotals *totals;     // the workspace: the totals, then a plan for every request
    TablesPlan *plan;
    Divider waves;            // waves that move one request's blocks
};
// LDS of a one-launch call's block: three words a request, two more, and its scans' sums.
constexpr int64_t tables_lds_bytes(int64_t req) { return (3 * req + 2) * 4; }
constexpr int64_t kTablesLdsFixed = 256;
constexpr int64_t tables_ws_bytes(int64_t req) { return int64_t(sizeof(TablesTotals)) + req * int64_t(sizeof(TablesPlan)); }

struct TablesLaunch {
    TablesArgs a;
    bool one_launch;
    int64_t grid;             // blocks that move ids
    void *stream, *ev_begin, *ev_end;
};
int launch_tables(const TablesLaunch &L);

struct SlotArgs {
    const int32_t *lens, *fresh;
    int64_t req;
    Divider block;
    const int32_t *table;
    int64_t ts;
    int max_blocks;
    const int32_t *held;
    int64_t n_blocks;
    int64_t capacity;
    void *slots;
    int32_t *positions, *requests, *starts;
    int64_t per_block;        // tokens of a block
};
constexpr int64_t slots_lds_bytes(int64_t req) { return (req + 1) * 12; }
constexpr int64_t kSlotsLdsFixed = 256;
struct SlotLaunch {
    SlotArgs a;
    int slot_dtype;
    bool stream_out;          // store past the caches
    int64_t grid;
    void *stream, *ev_begin, *ev_end;
};
int launch_slots(const SlotLaunch &L);

}  // namespace rk
