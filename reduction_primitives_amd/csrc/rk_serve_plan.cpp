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
