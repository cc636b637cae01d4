// rk_serve_plan.cpp -- launch plans of the serving operators (pure C++).
#include "rk_serve.hpp"

namespace rk {

size_t round_up_256(size_t b);

namespace {

bool prob_dtype_ok(int d) { return d == F32 || d == BF16 || d == F16; }

constexpr int64_t kMaxLines = 0x7fffffff;
constexpr int64_t kMaxThreads = 0xffffffff;   // of one launch
constexpr int64_t kMaxLine = 0x7fffffff;

}  // namespace

int plan_softmax(int in_dtype, int out_dtype, int64_t n, int64_t lines, SoftmaxPlan *p)
{
    *p = SoftmaxPlan();
    if (!dtype_known(in_dtype) || !dtype_known(out_dtype) || n < 0 || lines < 0)
        return ST_INVALID;
    if (!prob_dtype_ok(in_dtype) || !prob_dtype_ok(out_dtype))
        return ST_UNSUPPORTED;
    if (n > kMaxLine || lines > kMaxLines)
        return ST_UNSUPPORTED;
    // 16 bytes of the wider type (the first launch of a split line reads 16 bytes of input)
    const int in_vec = 16 / dtype_size(in_dtype), out_vec = 16 / dtype_size(out_dtype);
    p->vec = in_vec < out_vec ? in_vec : out_vec;
    if (n == 0 || lines == 0)
        return ST_OK;
    p->launches = 1;
    p->kernel = VK_SOFT_LINE;
    if (n <= 64 * tune::kSoftPer) {
        p->lanes = n <= tune::kSoftRowEntries ? 16 : 64;
        p->block = 256;
        p->grid = (lines + 256 / p->lanes - 1) / (256 / p->lanes);
    } else if (n <= tune::kSoftLanes * tune::kSoftPer) {
        p->lanes = 256;
        while (p->lanes * tune::kSoftPer < n)
            p->lanes *= 2;
        p->block = p->lanes;
        p->grid = lines;
    } else {
        constexpr int waves = tune::kSoftBlock / 64;
        p->kernel = VK_SOFT_SPLIT;
        p->vec = in_vec;
        p->block = tune::kSoftBlock;
        p->chunks = int((n + tune::kSoftTile - 1) / tune::kSoftTile);
        p->grid = lines * ((p->chunks + waves - 1) / waves);
        p->fold = p->chunks > tune::kSoftFoldTiles;
        p->launches = p->fold ? 3 : 2;
        p->stream_out = lines * n * dtype_size(out_dtype) > tune::kSoftStreamBytes;
        p->ws_bytes = round_up_256(size_t(lines) * size_t(p->chunks + (p->fold ? 1 : 0)) * 12);
    }
    return p->grid > kMaxThreads / p->block ? ST_UNSUPPORTED : ST_OK;
}

int plan_verify(int prob_dtype, int64_t n, int64_t req, int cus, VerifyPlan *p)
{
    *p = VerifyPlan();
    if (!dtype_known(prob_dtype) || n < 1 || req < 0)
        return ST_INVALID;
    if (!prob_dtype_ok(prob_dtype) || n > kMaxLine || req > kMaxLines)
        return ST_UNSUPPORTED;
    constexpr int waves = tune::kVerifyBlock / 64;
    p->tiles = (n + tune::kVerifyTile - 1) / tune::kVerifyTile;
    // a wave a tile while the blocks fit the chip at once; beyond that, more tiles a wave
    cus = cus > 0 ? cus : tune::kDefaultCus;
    const int64_t most = int64_t(cus) * tune::kVerifyBlocksPerCu;
    int64_t chunks = (p->tiles + waves - 1) / waves, fit = req > 0 ? most / req : chunks;
    fit = fit < 1 ? 1 : fit;
    p->chunks = int(chunks < fit ? chunks : fit);
    p->grid = req * p->chunks;
    if (p->grid > kMaxThreads / tune::kVerifyBlock)
        return ST_UNSUPPORTED;
    p->fused_ok = req * arrive_counters(p->chunks) <= kArriveCapacity && req <= cus &&
                  p->grid <= int64_t(cus) * tune::kVerifyFusedBlocksPerCu;
    p->launches = req == 0 ? 0 : p->chunks == 1 || p->fused_ok ? 1 : 2;
    p->ws_bytes = round_up_256(size_t(req) * (size_t(p->tiles) * 8 + sizeof(VerifyDrawn)));
    return ST_OK;
}

int plan_beams(int dtype, int64_t n, int64_t req, int64_t beams, int64_t count, int cus, BeamPlan *p)
{
    *p = BeamPlan();
    if (!dtype_known(dtype) || n < 1 || req < 0 || beams < 1 || count < 1)
        return ST_INVALID;
    if (!prob_dtype_ok(dtype) || n > kMaxLine || beams > tune::kBeamLines || count > tune::kBeamMost ||
        req > kMaxLines / beams)
        return ST_UNSUPPORTED;
    if (req == 0)
        return ST_OK;
    const int64_t lines = req * beams, tiles = (n + tune::kBeamTile - 1) / tune::kBeamTile;
    int64_t waves = int64_t(cus > 0 ? cus : tune::kDefaultCus) * tune::kBeamWavesPerCu / lines;
    waves = waves < 1 ? 1 : waves < tiles ? waves : tiles;
    const int64_t each = (tiles + waves - 1) / waves;
    p->chunks = (tiles + each - 1) / each;
    p->per_wave = each * tune::kBeamTile;
    p->items = lines * p->chunks;
    p->grid = (p->items + tune::kBeamBlock / 64 - 1) / (tune::kBeamBlock / 64);
    if (p->grid > kMaxThreads / tune::kBeamBlock || req > kMaxThreads / tune::kBeamBlock ||
        beams * p->chunks * count > 0x7fffffff - 4 * tune::kBeamBlock)
        return ST_UNSUPPORTED;
    p->ws_bytes = round_up_256(size_t(p->items) * (12 + 8 * size_t(count)));
    return ST_OK;
}

size_t fork_ws_bytes(int64_t rows, int64_t rows_out, int64_t max_blocks, int64_t n_blocks)
{
    return round_up_256(32 + 8 * size_t(rows * ((max_blocks + 63) / 64)) + 4 * size_t(2 * rows + rows_out + n_blocks));
}

size_t compact_ws_bytes(int64_t n_blocks)
{
    const size_t chunks = size_t((n_blocks + tune::kCompactChunk - 1) / tune::kCompactChunk);
    return round_up_256(16 + chunks * (tune::kCompactChunk + tune::kCompactChunk / 64 * sizeof(CompactWord)) + (chunks + 1) * 4);
}

Divider make_divider(uint32_t d)
{
    Divider r{d, 0, 0};
    if (d > 1) {
        int l = 0;
        while ((uint64_t(1) << l) < d)
            ++l;
        r.shift = 31 + l;
        r.m = uint32_t((uint64_t(1) << r.shift) / d + 1);
    }
    return r;
}

}  // namespace rk
