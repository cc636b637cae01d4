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
constexpr int kRecurStrip = 64;           // most channels of a tile
constexpr uint32_t kRecurSpinLimit = 1u << 24;   // look-back: sleeps per wait before giving up (about a second)
}  // namespace tune

// Most tokens of a lane: 16, or 8 where its inputs of 16 would not fit the
// registers (the backward pass reads a gate and three of x's type).
constexpr int recur_rows(int x_size, int gate_size, bool backward)
{
    return backward && gate_size + 3 * x_size > 8 ? 8 : 16;
}

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
    uint32_t spin_limit, force_wait;
};

// Look-back state of a tile: a line for its flag, then the map's factor and
// addend and the state behind the tile, a float each for every channel.
constexpr int kRecurHeaderBytes = 256;
constexpr int kRecurRecBytes = 128 + 3 * 4 * tune::kRecurStrip;

struct RecurPlan {
    int vec = 0, lanes_log2 = 0, per_lane = 0;   // channels of a lane, lanes across, tokens of a lane
    int strips = 0;
    int64_t tiles = 0;
    int tile_rows = 0;
    bool linked = false;
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
    void *stream, *ev_begin, *ev_end;
};
int launch_recur_f32(const RecurLaunch &L);
int launch_recur_bf16(const RecurLaunch &L);
int launch_recur_f16(const RecurLaunch &L);

}  // namespace rk
