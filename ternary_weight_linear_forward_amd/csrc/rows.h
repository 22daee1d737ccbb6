// rows.h -- eight consecutive elements of a row of fp32 or bf16 values at any
// element alignment (global memory serves 16-byte accesses at 2-byte steps), for
// the kernels around the BitLinears.
#pragma once

#include "common.h"

#include <type_traits>

namespace bl {

typedef uint32_t u4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u2_any __attribute__((ext_vector_type(2), aligned(1)));

// Elements idx .. idx + 7 of p, those at or past 'left' as 0 (and not read).
template <int DT>
__device__ __forceinline__ void load8(const void *p, int64_t idx, int64_t left, float (&v)[8])
{
    if (left >= 8) {
        if constexpr (DT == DT_F32) {
            const u4_any *q = reinterpret_cast<const u4_any *>(static_cast<const float *>(p) + idx);
            const u4_any a = q[0], b = q[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = __uint_as_float(a[e]);
                v[4 + e] = __uint_as_float(b[e]);
            }
        } else {
            const u4_any a = *reinterpret_cast<const u4_any *>(static_cast<const uint16_t *>(p) + idx);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(a[e] << 16);
                v[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < left ? load_x<DT>(p, idx + e) : 0.0f;
    }
}

// Stores v[e] at idx + e for e < left, rounded to nearest even for bf16.
template <int DT>
__device__ __forceinline__ void store8(void *p, int64_t idx, int64_t left, const float (&v)[8])
{
    if (left >= 8) {
        if constexpr (DT == DT_F32) {
            u4_any *q = reinterpret_cast<u4_any *>(static_cast<float *>(p) + idx);
            u4_any a, b;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = __float_as_uint(v[e]);
                b[e] = __float_as_uint(v[4 + e]);
            }
            q[0] = a;
            q[1] = b;
        } else {
            u4_any a;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                a[e] = float_to_bf16_rne(v[2 * e]) | static_cast<uint32_t>(float_to_bf16_rne(v[2 * e + 1])) << 16;
            *reinterpret_cast<u4_any *>(static_cast<uint16_t *>(p) + idx) = a;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) {
                if constexpr (DT == DT_F32) static_cast<float *>(p)[idx + e] = v[e];
                else static_cast<uint16_t *>(p)[idx + e] = float_to_bf16_rne(v[e]);
            }
    }
}

} // namespace bl
