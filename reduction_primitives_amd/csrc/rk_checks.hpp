// rk_checks.hpp -- argument checks that the C ABI's host files share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace rk {
namespace checks {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Span {
    uintptr_t from, to;       // bytes [from, to)
};

inline Span span(const void *p, int64_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p && bytes > 0 ? a + uintptr_t(bytes) : a};
}

inline Span line_span(const void *p, int64_t n, int64_t lines, int64_t stride, int size)
{
    return span(p, n > 0 && lines > 0 ? ((lines - 1) * stride + n) * size : 0);
}

inline bool overlap(const Span &a, const Span &b) { return a.from < b.to && b.from < a.to; }

// Lines fit the address space: lines * stride * 8 bytes stay far below 2^63.
inline bool lines_fit(int64_t n, int64_t lines, int64_t stride)
{
    constexpr int64_t most = int64_t(1) << 48;
    return stride >= 0 && stride <= most && n <= most && (lines <= 1 || stride == 0 || lines <= most / stride);
}

inline bool capturing(hipStream_t st)
{
    hipStreamCaptureStatus s = hipStreamCaptureStatusNone;
    return hipStreamIsCapturing(st, &s) != hipSuccess || s != hipStreamCaptureStatusNone;
}

}  // namespace checks
}  // namespace rk
