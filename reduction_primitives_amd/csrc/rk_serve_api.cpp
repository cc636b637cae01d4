// rk_serve_api.cpp -- the serving operators of the C ABI (include/rk.h):
// argument checks, plans, launches.
#include "rk.h"

#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstring>

#include "rk_host.hpp"
#include "rk_serve.hpp"

namespace {

using namespace rk;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Span {
    uintptr_t from, to;       // bytes [from, to)
};

Span span(const void *p, int64_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p && bytes > 0 ? a + uintptr_t(bytes) : a};
}

Span line_span(const void *p, int64_t n, int64_t lines, int64_t stride, int size)
{
    return span(p, n > 0 && lines > 0 ? ((lines - 1) * stride + n) * size : 0);
}

bool overlap(const Span &a, const Span &b) { return a.from < b.to && b.from < a.to; }

// Lines fit the address space: lines * stride * 8 bytes stay far below 2^63.
bool lines_fit(int64_t n, int64_t lines, int64_t stride)
{
    constexpr int64_t most = int64_t(1) << 48;
    return stride >= 0 && stride <= most && n <= most && (lines <= 1 || stride == 0 || lines <= most / stride);
}

bool capturing(hipStream_t st)
{
    hipStreamCaptureStatus s = hipStreamCaptureStatusNone;
    return hipStreamIsCapturing(st, &s) != hipSuccess || s != hipStreamCaptureStatusNone;
}

}  // namespace

extern "C" {

size_t rk_softmax_workspace_size(int in_dtype, int out_dtype, int64_t n, int64_t lines)
{
    SoftmaxPlan p;
    return plan_softmax(in_dtype, out_dtype, n, lines, &p) == ST_OK ? p.ws_bytes : 0;
}

int rk_plan_softmax(int in_dtype, int out_dtype, int64_t n, int64_t lines, rk_plan_info *info)
{
    if (!info)
        return RK_ERR_INVALID_ARGUMENT;
    SoftmaxPlan p;
    const int rc = plan_softmax(in_dtype, out_dtype, n, lines, &p);
    if (rc)
        return rc;
    std::memset(info, 0, sizeof *info);
    info->kernel = p.kernel == VK_SOFT_SPLIT ? RK_KERNEL_SOFTMAX_SPLIT
                   : p.kernel == VK_SOFT_LINE ? RK_KERNEL_SOFTMAX_LINE : RK_KERNEL_NONE;
    info->launches = p.launches;
    info->grid = p.grid;
    info->block = p.block;
    info->split = p.chunks;
    info->vec = p.vec;
    info->tile_outputs = p.kernel == VK_SOFT_SPLIT ? tune::kSoftTile : p.lanes * tune::kSoftPer;
    info->n_out = n * lines;
    info->reduce_len = n;
    info->workspace_bytes = p.ws_bytes;
    return RK_OK;
}

int rk_softmax(int in_dtype, int out_dtype, const void *x, int64_t n, int64_t lines, int64_t x_stride,
               const float *temperature, void *out, int64_t out_stride, void *workspace, size_t workspace_bytes,
               void *stream)
{
    SoftmaxPlan p;
    int rc = plan_softmax(in_dtype, out_dtype, n, lines, &p);
    if (rc)
        return rc;
    if (!lines_fit(n, lines, x_stride) || !lines_fit(n, lines, out_stride) || (lines > 1 && out_stride < n))
        return RK_ERR_INVALID_ARGUMENT;
    if (n == 0 || lines == 0)
        return RK_OK;
    const int isz = dtype_size(in_dtype), osz = dtype_size(out_dtype);
    if (!x || !out || !aligned(x, isz) || !aligned(out, osz) || !aligned(temperature, 4))
        return RK_ERR_INVALID_ARGUMENT;
    if (p.ws_bytes > 0 && (!workspace || !aligned(workspace, 8) || workspace_bytes < p.ws_bytes))
        return RK_ERR_INVALID_ARGUMENT;
    const Span so = line_span(out, n, lines, out_stride, osz);
    if (overlap(so, line_span(x, n, lines, x_stride, isz))) {
        // the line itself, or the other columns of the same rows
        const int64_t row = x_stride * isz;
        bool ok = x == out && isz == osz && (lines == 1 || x_stride == out_stride);
        if (!ok && lines > 1 && row == out_stride * osz) {
            const int64_t d = int64_t(reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(x));
            const int64_t r = (d % row + row) % row;
            ok = r >= n * isz && r + n * osz <= row;
        }
        if (!ok)
            return RK_ERR_INVALID_ARGUMENT;
    }
    const Span sw = span(workspace, int64_t(p.ws_bytes)), st = span(temperature, lines * 4);
    if (overlap(sw, so) || overlap(sw, line_span(x, n, lines, x_stride, isz)) || overlap(st, so) || overlap(st, sw))
        return RK_ERR_INVALID_ARGUMENT;
    if (host::debug_enabled())
        std::fprintf(stderr, "rk_softmax: n=%lld lines=%lld kernel=%d grid=%lld chunks=%d ws=%zu\n", (long long)n,
                     (long long)lines, p.kernel, (long long)p.grid, p.chunks, p.ws_bytes);
    SoftmaxLaunch L;
    std::memset(static_cast<void *>(&L), 0, sizeof L);
    L.plan = p;
    L.a.x = x;
    L.a.out = out;
    L.a.t = temperature;
    L.a.stats = static_cast<float *>(workspace);
    L.a.first = p.ws_bytes ? reinterpret_cast<int32_t *>(static_cast<float *>(workspace) + 2 * lines * (p.chunks + p.fold))
                           : nullptr;
    L.a.fold = p.fold;
    L.a.n = n;
    L.a.lines = lines;
    L.a.xs = x_stride;
    L.a.os = out_stride;
    L.a.chunks = p.chunks;
    L.a.per_line = make_divider(uint32_t(p.kernel == VK_SOFT_SPLIT ? p.grid / lines : 1));
    L.in = in_dtype;
    L.out = out_dtype;
    L.stream = stream;
    host::launch_events(&L.ev_begin, &L.ev_end);
    if (host::injected_launch_failure())
        return RK_ERR_HIP;
    return launch_softmax(L);
}

size_t rk_draft_verify_workspace_size(int prob_dtype, int64_t vocab, int64_t n_req)
{
    VerifyPlan p;
    return plan_verify(prob_dtype, vocab, n_req, host::device_cus(), &p) == ST_OK ? p.ws_bytes : 0;
}

int rk_plan_draft_verify(int prob_dtype, int64_t vocab, int64_t n_req, int num_cus, rk_plan_info *info)
{
    if (!info)
        return RK_ERR_INVALID_ARGUMENT;
    VerifyPlan p;
    const int rc = plan_verify(prob_dtype, vocab, n_req, num_cus > 0 ? num_cus : host::device_cus(), &p);
    if (rc)
        return rc;
    std::memset(info, 0, sizeof *info);
    info->kernel = p.grid > 0 ? RK_KERNEL_DRAFT_VERIFY : RK_KERNEL_NONE;
    info->launches = p.launches == 1 && p.chunks > 1 && !host::fused_finish() ? 2 : p.launches;
    info->grid = p.grid;
    info->block = tune::kVerifyBlock;
    info->split = p.chunks;
    info->vec = 16 / dtype_size(prob_dtype);
    info->tile_outputs = tune::kVerifyTile;
    info->n_out = n_req;
    info->reduce_len = vocab;
    info->workspace_bytes = p.ws_bytes;
    return RK_OK;
}

int rk_draft_verify(int prob_dtype, int token_dtype, const void *p, int64_t p_stride, const void *q, int64_t q_stride,
                    int64_t vocab, int64_t n_req, int64_t n_draft, int max_draft, const int32_t *starts,
                    const void *drafted, const float *u, const float *r, void *tokens, int32_t *accepted,
                    void *workspace, size_t workspace_bytes, void *stream)
{
    VerifyPlan pl;
    int rc = plan_verify(prob_dtype, vocab, n_req, host::device_cus(), &pl);
    if (rc)
        return rc;
    if (!dtype_known(token_dtype) || n_draft < 0 || max_draft < 0 || max_draft > (1 << 24))
        return RK_ERR_INVALID_ARGUMENT;
    if (token_dtype != I32 && token_dtype != I64)
        return RK_ERR_UNSUPPORTED;
    if (n_draft > 0x7fffffff - n_req)
        return RK_ERR_UNSUPPORTED;
    if (!starts && n_draft != n_req * max_draft)
        return RK_ERR_INVALID_ARGUMENT;
    if (n_req == 0)
        return RK_OK;
    const int64_t rows = n_draft + n_req;
    if (!lines_fit(vocab, rows, p_stride) || (q && !lines_fit(vocab, n_draft, q_stride)))
        return RK_ERR_INVALID_ARGUMENT;
    const int psz = dtype_size(prob_dtype), tsz = dtype_size(token_dtype);
    if (!p || !r || !tokens || !accepted || (n_draft > 0 && (!drafted || !u)))
        return RK_ERR_INVALID_ARGUMENT;
    if (!aligned(p, psz) || !aligned(q, psz) || !aligned(drafted, tsz) || !aligned(tokens, tsz) || !aligned(u, 4) ||
        !aligned(r, 4) || !aligned(starts, 4) || !aligned(accepted, 4))
        return RK_ERR_INVALID_ARGUMENT;
    if (!workspace || !aligned(workspace, 8) || workspace_bytes < pl.ws_bytes)
        return RK_ERR_INVALID_ARGUMENT;
    const Span out[] = {span(tokens, n_req * (int64_t(max_draft) + 1) * tsz), span(accepted, n_req * 4),
                        span(workspace, int64_t(pl.ws_bytes))};
    const Span in[] = {line_span(p, vocab, rows, p_stride, psz), line_span(q, vocab, n_draft, q_stride, psz),
                       span(starts, (n_req + 1) * 4), span(drafted, n_draft * tsz), span(u, n_draft * 4),
                       span(r, n_req * 4)};
    for (int i = 0; i < 3; ++i) {
        for (const Span &s : in)
            if (overlap(out[i], s))
                return RK_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return RK_ERR_INVALID_ARGUMENT;
    }
    if (host::debug_enabled())
        std::fprintf(stderr, "rk_draft_verify: vocab=%lld requests=%lld drafts=%lld tiles=%lld chunks=%d ws=%zu\n",
                     (long long)vocab, (long long)n_req, (long long)n_draft, (long long)pl.tiles, pl.chunks,
                     pl.ws_bytes);
    VerifyLaunch L;
    std::memset(static_cast<void *>(&L), 0, sizeof L);
    L.plan = pl;
    L.a.p = p;
    L.a.q = n_draft > 0 ? q : nullptr;
    L.a.ps = p_stride;
    L.a.qs = q_stride;
    L.a.n = vocab;
    L.a.req = n_req;
    L.a.drafts = n_draft;
    L.a.max_draft = max_draft;
    L.a.starts = starts;
    L.a.drafted = drafted;
    L.a.u = u;
    L.a.r = r;
    L.a.tokens = tokens;
    L.a.accepted = accepted;
    L.a.sums = static_cast<double *>(workspace);
    L.a.drawn = reinterpret_cast<VerifyDrawn *>(L.a.sums + n_req * pl.tiles);
    L.a.tiles = pl.tiles;
    L.a.chunks = pl.chunks;
    // A captured call takes the second launch: it then shares no counters
    // with other graphs captured on the same stream.
    L.a.slot = pl.chunks > 1 && pl.fused_ok && !capturing(static_cast<hipStream_t>(stream))
                   ? host::stream_slot(stream) : -1;
    L.dtype = prob_dtype;
    L.token_dtype = token_dtype;
    L.stream = stream;
    host::launch_events(&L.ev_begin, &L.ev_end);
    if (host::injected_launch_failure())
        return RK_ERR_HIP;
    return launch_verify(L);
}

size_t rk_block_tables_workspace_size(int64_t n_req)
{
    return n_req < 0 || n_req > 0x7fffffff ? 0 : (size_t(tables_ws_bytes(n_req)) + 255) / 256 * 256;
}

int rk_block_tables(const int32_t *lens, int64_t n_req, int block_size, const int32_t *held, int32_t *held_out,
                    int32_t *table, int64_t table_stride, int max_blocks, int32_t *ring, int64_t ring_size,
                    const int64_t *state, int64_t *state_out, void *workspace, size_t workspace_bytes, void *stream)
{
    if (n_req < 0 || block_size < 1 || max_blocks < 0 || ring_size < 1)
        return RK_ERR_INVALID_ARGUMENT;
    if (n_req > 0x7fffffff || ring_size > 0x7fffffff)
        return RK_ERR_UNSUPPORTED;
    if (!lines_fit(max_blocks, n_req, table_stride) || (n_req > 1 && table_stride < max_blocks))
        return RK_ERR_INVALID_ARGUMENT;
    const int64_t ws = int64_t(rk_block_tables_workspace_size(n_req));
    if (!ring || !state || !state_out || !aligned(ring, 4) || !aligned(state, 8) || !aligned(state_out, 8) ||
        !workspace || !aligned(workspace, 8) || workspace_bytes < size_t(ws))
        return RK_ERR_INVALID_ARGUMENT;
    if (n_req > 0 && (!lens || !held || !held_out || (max_blocks > 0 && !table)))
        return RK_ERR_INVALID_ARGUMENT;
    if (!aligned(lens, 4) || !aligned(held, 4) || !aligned(held_out, 4) || !aligned(table, 4))
        return RK_ERR_INVALID_ARGUMENT;
    // held_out may be held and state_out state; nothing else may overlap what is written
    const Span out[] = {span(held_out, n_req * 4), span(state_out, 32), line_span(table, max_blocks, n_req, table_stride, 4),
                        span(ring, ring_size * 4), span(workspace, ws)};
    const Span sl = span(lens, n_req * 4), sh = span(held, n_req * 4), ss = span(state, 16);
    for (int i = 0; i < 5; ++i) {
        if (overlap(out[i], sl) || (overlap(out[i], sh) && !(i == 0 && held_out == held)) ||
            (overlap(out[i], ss) && !(i == 1 && state_out == state)))
            return RK_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return RK_ERR_INVALID_ARGUMENT;
    }
    const int cus = host::device_cus() > 0 ? host::device_cus() : tune::kDefaultCus;
    const bool one_launch = n_req > 0 && n_req <= tune::kMoveLdsRequests &&
                            n_req * int64_t(max_blocks) < (int64_t(1) << 31) && held_out != held && state_out != state;
    constexpr int block_waves = tune::kMoveBlock / 64, ids = 64 * tune::kMoveEach;
    const int64_t cap = int64_t(cus) * tune::kMoveBlocksPerCu;
    int64_t grid, waves = 1;
    if (one_launch) {                         // what can move, dealt to all waves
        const int64_t most = n_req * int64_t(max_blocks);
        const int64_t fit = int64_t(cus) * resident(tables_lds_bytes(n_req) + kTablesLdsFixed, tune::kMoveBlocksPerCu);
        grid = (most + ids * block_waves - 1) / (ids * block_waves);
        grid = grid < 1 ? 1 : grid < fit ? grid : fit;
    } else {                                  // a wave a request, more where requests are few and their lines long
        const int64_t useful = (int64_t(max_blocks) + ids - 1) / ids;
        waves = n_req > 0 ? cap * block_waves / n_req : 1;
        waves = waves < useful ? waves : useful;
        waves = waves < 1 ? 1 : waves;
        grid = (n_req * waves + block_waves - 1) / block_waves;
        if (grid > int64_t(0xffffffff) / tune::kMoveBlock)
            return RK_ERR_UNSUPPORTED;
    }
    if (host::debug_enabled())
        std::fprintf(stderr, "rk_block_tables: requests=%lld block=%d max_blocks=%d ring=%lld grid=%lld\n",
                     (long long)n_req, block_size, max_blocks, (long long)ring_size, (long long)grid);
    TablesLaunch L;
    std::memset(static_cast<void *>(&L), 0, sizeof L);
    L.a.lens = lens;
    L.a.held = held;
    L.a.held_out = held_out;
    L.a.req = n_req;
    L.a.block = make_divider(uint32_t(block_size));
    L.a.table = table;
    L.a.ts = table_stride;
    L.a.max_blocks = max_blocks;
    L.a.ring = ring;
    L.a.ring_size = ring_size;
    L.a.state = state;
    L.a.state_out = state_out;
    L.a.totals = static_cast<TablesTotals *>(workspace);
    L.a.plan = reinterpret_cast<TablesPlan *>(L.a.totals + 1);
    L.a.waves = make_divider(uint32_t(waves));
    L.one_launch = one_launch;
    L.grid = grid;
    L.stream = stream;
    host::launch_events(&L.ev_begin, &L.ev_end);
    if (host::injected_launch_failure())
        return RK_ERR_HIP;
    return launch_tables(L);
}

int rk_slot_map(const int32_t *lens, const int32_t *fresh, int64_t n_req, int block_size, const int32_t *table,
                int64_t table_stride, int max_blocks, const int32_t *held, int64_t n_blocks, int slot_dtype,
                int64_t capacity, void *slots, int32_t *positions, int32_t *requests, int32_t *starts, void *stream)
{
    if (n_req < 0 || block_size < 1 || max_blocks < 0 || n_blocks < 0 || capacity < 0 || !dtype_known(slot_dtype))
        return RK_ERR_INVALID_ARGUMENT;
    if (slot_dtype != I32 && slot_dtype != I64)
        return RK_ERR_UNSUPPORTED;
    if (n_req > 0x7ffffffe || capacity > 0x7fffffff || n_blocks > 0x7fffffff ||
        (slot_dtype == I32 && n_blocks * block_size > (int64_t(1) << 31)))
        return RK_ERR_UNSUPPORTED;
    if (!lines_fit(max_blocks, n_req, table_stride) || (n_req > 1 && table_stride < max_blocks))
        return RK_ERR_INVALID_ARGUMENT;
    const int ssz = dtype_size(slot_dtype);
    if (!starts || (capacity > 0 && !slots) || (n_req > 0 && (!lens || !fresh || !held || (max_blocks > 0 && !table))))
        return RK_ERR_INVALID_ARGUMENT;
    if (!aligned(lens, 4) || !aligned(fresh, 4) || !aligned(held, 4) || !aligned(table, 4) || !aligned(slots, ssz) ||
        !aligned(positions, 4) || !aligned(requests, 4) || !aligned(starts, 4))
        return RK_ERR_INVALID_ARGUMENT;
    const Span out[] = {span(slots, capacity * ssz), span(positions, capacity * 4), span(requests, capacity * 4),
                        span(starts, (n_req + 1) * 4)};
    const Span in[] = {span(lens, n_req * 4), span(fresh, n_req * 4), span(held, n_req * 4),
                       line_span(table, max_blocks, n_req, table_stride, 4)};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : in)
            if (overlap(out[i], s))
                return RK_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j]))
                return RK_ERR_INVALID_ARGUMENT;
    }
    const int cus = host::device_cus() > 0 ? host::device_cus() : tune::kDefaultCus;
    const int64_t step = int64_t(tune::kSlotBlock) * (16 / ssz);
    const int64_t most = int64_t(cus) * (n_req <= tune::kSlotLdsRequests
                                          ? resident(slots_lds_bytes(n_req) + kSlotsLdsFixed, tune::kSlotBlocksPerCu)
                                          : tune::kSlotBlocksPerCu);
    int64_t per = (capacity + most - 1) / most;
    per = (per + step - 1) / step * step;
    per = per < step ? step : per;
    const int64_t grid = capacity > 0 ? (capacity + per - 1) / per : 1;
    if (host::debug_enabled())
        std::fprintf(stderr, "rk_slot_map: requests=%lld block=%d capacity=%lld grid=%lld\n", (long long)n_req,
                     block_size, (long long)capacity, (long long)grid);
    SlotLaunch L;
    std::memset(static_cast<void *>(&L), 0, sizeof L);
    L.a.lens = lens;
    L.a.fresh = fresh;
    L.a.req = n_req;
    L.a.block = make_divider(uint32_t(block_size));
    L.a.table = table;
    L.a.ts = table_stride;
    L.a.max_blocks = max_blocks;
    L.a.held = held;
    L.a.n_blocks = n_blocks;
    L.a.capacity = capacity;
    L.a.slots = slots;
    L.a.positions = positions;
    L.a.requests = requests;
    L.a.starts = starts;
    L.a.per_block = per;
    L.slot_dtype = slot_dtype;
    L.stream_out = capacity * (ssz + (positions ? 4 : 0) + (requests ? 4 : 0)) > tune::kSlotStreamBytes;
    L.grid = grid;
    L.stream = stream;
    host::launch_events(&L.ev_begin, &L.ev_end);
    if (host::injected_launch_failure())
        return RK_ERR_HIP;
    return launch_slots(L);
}

}  // extern "C"
