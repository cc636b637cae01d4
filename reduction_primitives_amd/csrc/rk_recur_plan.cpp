// rk_recur_plan.cpp -- launch plan of the gated linear recurrence (pure C++).
#include "rk_recur.hpp"

namespace rk {

size_t round_up_256(size_t b);

int plan_recur(int x_dtype, int gate_dtype, int64_t rows, int64_t segs, int64_t period, int64_t channels, bool backward,
               int cus, RecurPlan *p)
{
    *p = RecurPlan();
    if (!dtype_known(x_dtype) || !dtype_known(gate_dtype) || rows < 0 || segs < 0 || channels < 0)
        return ST_INVALID;
    if ((x_dtype != F32 && x_dtype != BF16 && x_dtype != F16) || (gate_dtype != x_dtype && gate_dtype != F32))
        return ST_UNSUPPORTED;
    if (rows > 0x7fffffff || segs > 0x7fffffff || channels > 0x7fffffff)
        return ST_UNSUPPORTED;
    if (segs == 0 || channels == 0)
        return ST_OK;
    p->launches = 1;
    if (rows == 0)
        return ST_OK;
    cus = cus > 0 ? cus : tune::kDefaultCus;
    if (period == 1 && !backward && segs == 1) {
        const int64_t lanes = (channels + tune::kRecurVec - 1) / tune::kRecurVec;
        int log2 = 0;
        while ((1 << log2) < lanes && (1 << log2) < tune::kRecurBlock)
            ++log2;
        const int64_t strips = ((lanes - 1) >> log2) + 1, rows_a_block = tune::kRecurBlock >> log2,
                      blocks = (rows + rows_a_block - 1) / rows_a_block;
        if (blocks <= 0xffffff / strips) {    // (more rows go through tiles of several)
            p->step = true;
            p->vec = tune::kRecurVec;
            p->per_lane = 1;
            p->lanes_log2 = log2;
            p->strips = int(strips);
            p->tile_rows = int(rows_a_block);
            p->tiles = blocks;
            p->grid = blocks * strips;
            return ST_OK;
        }
    }
    p->vec = channels < tune::kRecurVec ? 1 : tune::kRecurVec;
    while ((p->vec << p->lanes_log2) < channels && (p->vec << p->lanes_log2) < tune::kRecurStrip)
        ++p->lanes_log2;
    const int64_t strip = int64_t(p->vec) << p->lanes_log2, strips = (channels + strip - 1) / strip;
    if (strips * segs > 0xffffff)
        return ST_UNSUPPORTED;                // blocks of 256 threads of a launch
    const int64_t groups = tune::kRecurBlock >> p->lanes_log2;
    // One token a lane where more would leave half of the CUs without a block.  With and without, bf16, us a call:
    // 1 x 256 x 2048 backward 12.6 and 14.3, 1 x 64 x 2048 10.1 and 10.0.  Forward it wins nothing (12.1 and 11.6, 10.1
    // and 8.2), and where there are few channels the look-back goes through eight times as many tiles: 1 x 8192 x 64
    // forward 52 and 17, backward 52 and 19.
    p->per_lane = p->vec == 1 ? 4 : recur_rows(dtype_size(x_dtype), dtype_size(gate_dtype), backward);
    if (p->vec > 1 && (rows + groups * p->per_lane - 1) / (groups * p->per_lane) * strips * segs < cus / 2)
        p->per_lane = 1;
    int64_t tile = groups * p->per_lane;
    // whole sequences a tile, where at most a quarter of its lanes is left idle: no state passes between tiles then
    p->linked = period == 0 || (tile % period != 0 && 4 * period > tile);
    if (!p->linked)
        tile = tile / period * period;
    p->tile_rows = int(tile);
    p->strips = int(strips);
    p->tiles = (rows + tile - 1) / tile;
    p->linked = p->linked && p->tiles > 1;
    if (p->tiles * strips * segs > 0xffffff)
        return ST_UNSUPPORTED;
    p->grid = p->tiles * strips * segs;
    if (p->linked) {
        p->launches = 2;
        p->ws_bytes = round_up_256(size_t(p->grid + kRecurBatch - 1) * kRecurRecBytes);
    }
    return ST_OK;
}

}  // namespace rk
