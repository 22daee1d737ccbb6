// checks.h -- argument checks shared by the C entry points (host only,
// internal): element sizes, byte spans and their overlap, stride bounds.
#pragma once

#include "bitlinear.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 40; // keeps per-exponent sums of |W| below 2^64
int64_t round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }

int dtype_size(int dt)
{
    switch (dt) {
    case BITLINEAR_F32: return 4;
    case BITLINEAR_BF16: return 2;
    case BITLINEAR_I8: return 1;
    case BITLINEAR_I32: return 4;
    case BITLINEAR_I8_TILED: return 1;
    default: return 0;
    }
}

struct Span {
    uintptr_t lo, hi; // [lo, hi)
};

Span span_of(const void *p, int64_t rows, int64_t ld, int64_t cols, int elem)
{
    uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    uintptr_t bytes = static_cast<uintptr_t>(((rows - 1) * ld + cols) * elem);
    return {lo, lo + bytes};
}

bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// Row strides are bounded so that no offset (rows - 1) * ld * 4 bytes, on the
// host or in a kernel, can overflow 64 bits: ld <= 2^40 elements and the
// rows span at most 2^44 elements.
constexpr int64_t kMaxLd = int64_t(1) << 40, kMaxSpan = int64_t(1) << 44;
bool stride_ok(int64_t rows, int64_t ld) { return ld <= kMaxLd && rows - 1 <= kMaxSpan / ld; }

int status_of(hipError_t e) { return e == hipSuccess ? BITLINEAR_OK : BITLINEAR_ERR_LAUNCH; }

bool valid_layout(int layout)
{
    return layout == BITLINEAR_LAYOUT_I2 || layout == BITLINEAR_LAYOUT_B3 || layout == BITLINEAR_LAYOUT_B1;
}

constexpr int64_t kTiledMaxK = 65536; // the tiled quantiser keeps a row's pieces in registers

} // namespace
