// rk_recur.hpp -- plan and kernel arguments of the gated linear recurrence and
// its backward pass.  Pure C++ (no HIP), like rk_plan.hpp.
#pragma once

#include <cstddef>
#include <cstdint>

#include "rk_serve.hpp"

namespace rk {
namespace tune {
constexpr int kRecurBlock = 256;          // threads
constexpr int kRecurVec = 4;              // channels of a lane (1 where there are fewer)
// Most channels of a tile, so that a row of it is a whole 128-byte line of 16-bit
// elements (32, in an earlier version: 65536 x 2048 bf16 forward 272 us against 260,
// 512 x 64 x 2048 backward 250 against 178).
constexpr int kRecurStrip = 64;
// Sequences of so many tokens, up to so many of them, are columns of their own:
// the tiles that run at the same time are then mostly other sequences', not the
// ones a tile waits for.  Apart and one after the other, bf16 forward, us a call: 64 x
// 512 x 2048 102 and 112, 32 x 1024 x 2048 107 and 117, 1024 x 512 x 128 96 and 119
// (backward 187 and 193, 192 and 198, 181 and 199); 64 x 256 x 2048 55 and 57, 2 x 256
// x 2048 12.2 and 11.9.  The borders are rough: sequences that fill a tile together
// gain nothing (4096 x 512 x 4: 41 and 20), and beyond 4096 of them some still would
// (8192 x 512 x 32: 171 and 196).
constexpr int64_t kRecurApart = 512, kRecurApartMost = 4096;
// Polls of a look-back (a microsecond each) before its block does the work of one
// that has not been started.
constexpr uint32_t kRecurPatience = 4096;
// And of a block that has done so: where blocks have been held back there may be
// hundreds of such tiles in a column, one behind the other, and 4096 polls each
// seconds in all.  (A block that is under way ends after some 15 us: 16384 of them
// take 247, 1024 at a time.)
constexpr uint32_t kRecurPatienceAgain = 64;
static_assert(kRecurPatienceAgain <= kRecurPatience, "polls begin at the difference");
}  // namespace tune

// Most tokens of a lane: what leaves the registers for kRecurWaves waves.  The bytes
// that blocks have on their way bound the rate: with three waves a SIMD, in an earlier
// version, 8 x 4096 x 2048 bf16 backward took 219 us, with four 204; forward with 12
// tokens, gates computed twice to make room for them, 16 x 4096 x 2048 took 233 us,
// with 8 and gates kept 207.
constexpr int recur_rows(int x_size, int gate_size, bool backward)
{
    return backward && gate_size + 3 * x_size > 8 ? 4 : 8;
}
constexpr int kRecurWaves = 4;            // of a SIMD

enum RecurKind { RECUR_VALUE = 0, RECUR_LOG = 1, RECUR_SIGMOID = 2 };

// A tensor of tokens x channels: elements between sequences (or 0 where they
// follow each other) and between tokens; channels are contiguous.
struct RecurTensor {
    const void *p;
    int64_t bs, ts;
};

struct RecurArgs {
    RecurTensor gate, x, h, dout;     // h: the forward pass's outputs, read by the backward pass
    RecurTensor out, dgate;           // written: the outputs, or the gradients of x and of the gates
    const float *state;               // [n_states][channels] or NULL
    const float *dlast;               // backward: gradients of the last states, or NULL
    float *state_out;                 // forward: the last states; backward: the gradients of the first ones
    const int32_t *sources;           // line of `state` a sequence starts from, NULL: its own
    int64_t n_states;
    const int32_t *starts;            // n_seq + 1 offsets of the sequences in the rows, or NULL
    int64_t n_seq;
    int64_t rows, segs;               // tokens of a segment, segments (tensors' bs apart)
    Divider period;                   // without starts: tokens of a sequence
    int64_t channels;
    int kind;
    bool blend;
    int lanes_log2;                   // lanes across a tile's channels
    int strips;                       // tiles across the channels
    int64_t tiles;                    // tiles along a segment's tokens
    int tile_rows;                    // tokens of a tile
    bool linked;                      // a tile may begin inside a sequence: states pass from tile to tile
    uint32_t *ws;
    uint32_t patience;
    bool force_help;                  // every block that looks back computes the tile before its own, too (a test hook)
};

// Look-back state: two words for every channel of every tile, and kRecurBatch - 1
// tiles' more that a look-back may load with the last one's.
constexpr int kRecurBatch = 4;            // records that a wave has on their way at a time (8 spill registers)
constexpr int kRecurRecBytes = 2 * 8 * tune::kRecurStrip;

struct RecurPlan {
    int vec = 0, lanes_log2 = 0, per_lane = 0;   // channels of a lane, lanes across, tokens of a lane
    int strips = 0;
    int64_t tiles = 0;
    int tile_rows = 0;
    bool linked = false;
    bool step = false;        // one token a sequence, forward: a lane a row's four channels, no tiles
    int64_t grid = 0;
    int launches = 0;
    size_t ws_bytes = 0;
};

// rows, segs: as in RecurArgs; period: tokens of a sequence, 0 where they are packed
int plan_recur(int x_dtype, int gate_dtype, int64_t rows, int64_t segs, int64_t period, int64_t channels, bool backward,
               int cus, RecurPlan *p);

struct RecurLaunch {
    RecurPlan plan;
    RecurArgs a;
    int gate_dtype;
    bool backward;
    const float *state;       // first states that are copied to `kept` before the tiles are begun, or NULL
    float *kept;
    void *stream, *ev_begin, *ev_end;
};
int launch_recur_f32(const RecurLaunch &L);
int launch_recur_bf16(const RecurLaunch &L);
int launch_recur_f16(const RecurLaunch &L);

}  // namespace rk
