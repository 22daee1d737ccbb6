// cache.hip -- keys and values quantised to int8 as they are written into the
// paged cache, and read back.  Per token and head: scale = max|x| / 127, byte =
// rint(x s) with s = 127 (1 / max|x|), every operation rounded to binary32.
//
// Both directions move tiles of 64 tokens (in the caller's order) of one head, K
// or V: a thread takes a quad of tokens 16 T + 4 g + {0..3} and 8 columns, LPR
// threads cover a row.  V's block order makes a quad of one column one 32-bit
// word, so the 4 x 8 bytes of a thread are transposed in registers (16
// v_perm_b32) and move as 8 words; the four T of a g are 16 neighbouring bytes.
// A quad whose slots are not four consecutive, 4-aligned ones moves by bytes.
// Bound: HBM for prompts, latency for a decode step's few tokens.
// Measured: 16000 tokens x 8 heads x 128 bf16, 98 MB a direction: write 26 us (3.8
// TB/s), read 21 us (4.7 TB/s); 1999 x 32 x 100 fp32, 64 MB: 15 and 17 us; 16 x 8 x
// 128: 5.6 and 4.7 us; 2000 x 8 x 128 from slot 0: 6.2 and 5.8 us, from slot 333, where
// no quad is a run, 10.4 and 8.3 us.  Tokens one by one, without tiles, took 3.6 times as long.
#include "cache_core.h"
#include "common.h"
#include "launch.h"
#include "rows.h"

namespace bl {

// x s within 127 (1 + 2^-24)^3 < 127.5, so quant4_bounded's rounding applies.
// Rows below 2^-96 are brought up by 2^64 first, as in token_quant, so that 1 /
// max|x| stays finite.
__device__ __forceinline__ TokenQuant cache_quant(float top)
{
    TokenQuant t;
    t.pre = top < 0x1p-96f ? 0x1p64f : 1.0f;
    t.s = top > 0.0f ? 127.0f * (1.0f / (top * t.pre)) : 0.0f;
    return t;
}

// Maximum over groups of LPR lanes (a power of two up to 32), in every lane.
template <int LPR>
__device__ __forceinline__ float group_max(float v)
{
    auto step = [&](int x) { v = fmaxf(v, __int_as_float(x)); };
    if constexpr (LPR >= 2) step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xb1, 0xf, 0xf, true));   // quad_perm xor 1
    if constexpr (LPR >= 4) step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4e, 0xf, 0xf, true));   // quad_perm xor 2
    if constexpr (LPR >= 8) step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));  // row_half_mirror
    if constexpr (LPR >= 16) step(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true)); // row_mirror
    if constexpr (LPR >= 32) v = fmaxf(v, __shfl_xor(v, 16));
    return v;
}

// 4 x 4 bytes, rows to columns (its own inverse).
__device__ __forceinline__ void transpose4(uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d)
{
    const uint32_t l0 = __builtin_amdgcn_perm(b, a, 0x05010400u), h0 = __builtin_amdgcn_perm(b, a, 0x07030602u);
    const uint32_t l1 = __builtin_amdgcn_perm(d, c, 0x05010400u), h1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
    a = __builtin_amdgcn_perm(l1, l0, 0x05040100u);
    b = __builtin_amdgcn_perm(l1, l0, 0x07060302u);
    c = __builtin_amdgcn_perm(h1, h0, 0x05040100u);
    d = __builtin_amdgcn_perm(h1, h0, 0x07060302u);
}

// The four slots of a quad: place of each token (row of the head's K, -1 for
// none), and whether they are one aligned run.
struct Quad {
    int64_t row[4]; // token's row in units of tokens, or -1
    bool run;
};

__device__ __forceinline__ Quad quad_of(const CacheView &c, const int64_t *slots, int64_t tokens, int64_t m0, int head)
{
    Quad q;
    int64_t s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] = m0 + r < tokens ? slots[m0 + r] : -1;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const bool ok = s[r] >= 0 && s[r] < c.slots;
        // (page_tokens and slots / 64 fit 32 bits: slots <= 2^36)
        const uint32_t blk = ok ? static_cast<uint32_t>(s[r] / CACHE_BLOCK) : 0u, bpp = c.page_tokens / CACHE_BLOCK;
        const uint32_t page = blk / bpp;
        q.row[r] = ok ? cache_row0(c, page, head) + (blk - page * bpp) * CACHE_BLOCK + s[r] % CACHE_BLOCK : -1;
    }
    q.run = s[0] >= 0 && s[0] < c.slots && s[0] % 4 == 0 && s[1] == s[0] + 1 && s[2] == s[0] + 2 && s[3] == s[0] + 3;
    return q;
}

// Byte of token row 'row' (of its head), column d of V.
__device__ __forceinline__ int64_t v_at(const CacheView &c, int64_t row, int d)
{
    const int t = static_cast<int>(row % CACHE_BLOCK);
    return (row - t) * c.Dp + d * CACHE_BLOCK + cache_v_byte(t);
}

template <int DT, int LPR>
__global__ __launch_bounds__(256) void k_cache_write(const CacheView c, const CacheRows rows, const int64_t *slots,
                                                     int64_t tokens)
{
    const int64_t base = static_cast<int64_t>(blockIdx.x) * CACHE_BLOCK;
    const int head = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    const void *src = is_v ? rows.V : rows.K;
    const int64_t ld_t = is_v ? rows.ldv_t : rows.ldk_t, off = head * (is_v ? rows.ldv_h : rows.ldk_h);
    for (int id = threadIdx.x; id < 16 * LPR; id += 256) {
        const int L = id % LPR, T = id / LPR % 4, g = id / LPR / 4, d0 = 8 * L;
        const int64_t m0 = base + 16 * T + 4 * g;
        if (m0 >= tokens) continue; // (whole groups of LPR lanes)
        const Quad q = quad_of(c, slots, tokens, m0, head);
        float x[4][8];
#pragma unroll
        for (int r = 0; r < 4; ++r) load8<DT>(src, off + (q.row[r] >= 0 ? m0 + r : m0) * ld_t + d0, c.D - d0, x[r]);
        uint32_t w[4][2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[r][e]));
            top = group_max<LPR>(top);
            const TokenQuant s = cache_quant(top);
            w[r][0] = quant4_bounded(x[r][0], x[r][1], x[r][2], x[r][3], s);
            w[r][1] = quant4_bounded(x[r][4], x[r][5], x[r][6], x[r][7], s);
            if (L == 0 && q.row[r] >= 0) (is_v ? c.Vs : c.Ks)[q.row[r]] = top / 127.0f;
        }
        if (d0 >= c.Dp) continue;
        if (!is_v) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (q.row[r] >= 0) *reinterpret_cast<uint2 *>(c.K + q.row[r] * c.Dp + d0) = make_uint2(w[r][0], w[r][1]);
            continue;
        }
        if (q.run) {
            uint32_t *dst = reinterpret_cast<uint32_t *>(c.V + v_at(c, q.row[0], d0));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                transpose4(w[0][h], w[1][h], w[2][h], w[3][h]);
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[(4 * h + e) * (CACHE_BLOCK / 4)] = w[e][h];
            }
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (q.row[r] >= 0) {
                    int8_t *dst = c.V + v_at(c, q.row[r], d0);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dst[e * CACHE_BLOCK] = static_cast<int8_t>(w[r][e / 4] >> (8 * (e % 4)));
                }
        }
    }
}

template <int DT, int LPR>
__global__ __launch_bounds__(256) void k_cache_read(const CacheView c, const CacheRows rows, const int64_t *slots,
                                                    int64_t tokens)
{
    const int64_t base = static_cast<int64_t>(blockIdx.x) * CACHE_BLOCK;
    const int head = blockIdx.y;
    const bool is_v = blockIdx.z != 0;
    void *dst = is_v ? rows.V : rows.K;
    const int64_t ld_t = is_v ? rows.ldv_t : rows.ldk_t, off = head * (is_v ? rows.ldv_h : rows.ldk_h);
    for (int id = threadIdx.x; id < 16 * LPR; id += 256) {
        const int L = id % LPR, T = id / LPR % 4, g = id / LPR / 4, d0 = 8 * L;
        const int64_t m0 = base + 16 * T + 4 * g;
        if (m0 >= tokens || d0 >= c.D) continue;
        const Quad q = quad_of(c, slots, tokens, m0, head);
        uint32_t w[4][2];
        float s[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            w[r][0] = w[r][1] = 0;
            s[r] = q.row[r] >= 0 ? (is_v ? c.Vs : c.Ks)[q.row[r]] : 0.0f;
        }
        if (!is_v) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (q.row[r] >= 0) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(c.K + q.row[r] * c.Dp + d0);
                    w[r][0] = u.x;
                    w[r][1] = u.y;
                }
        } else if (q.run) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(c.V + v_at(c, q.row[0], d0));
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e][h] = p[(4 * h + e) * (CACHE_BLOCK / 4)];
#pragma unroll
            for (int h = 0; h < 2; ++h) transpose4(w[0][h], w[1][h], w[2][h], w[3][h]);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (q.row[r] >= 0) {
                    const int8_t *p = c.V + v_at(c, q.row[r], d0);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[r][e / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(p[e * CACHE_BLOCK])) << (8 * (e % 4));
                }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (m0 + r >= tokens) continue;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(static_cast<int8_t>(w[r][e / 4] >> (8 * (e % 4)))) * s[r];
            store8<DT>(dst, off + (m0 + r) * ld_t + d0, c.D - d0, x);
        }
    }
}

// Threads a row (8 columns each).
template <class F>
static void by_lanes(int Dp, const F &f)
{
    if (Dp <= 32) f(std::integral_constant<int, 4>());
    else if (Dp <= 64) f(std::integral_constant<int, 8>());
    else if (Dp <= 128) f(std::integral_constant<int, 16>());
    else f(std::integral_constant<int, 32>());
}

hipError_t launch_cache_write(const CacheView &c, const CacheRows &r, int dtype, int64_t tokens, const int64_t *slots,
                              hipStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((tokens + CACHE_BLOCK - 1) / CACHE_BLOCK), static_cast<unsigned>(c.heads), 2),
        block(256);
    by_lanes(c.Dp, [&](auto lpr) {
        if (dtype == DT_F32) hipLaunchKernelGGL((k_cache_write<DT_F32, lpr>), grid, block, 0, stream, c, r, slots, tokens);
        else hipLaunchKernelGGL((k_cache_write<DT_BF16, lpr>), grid, block, 0, stream, c, r, slots, tokens);
    });
    return hipGetLastError();
}

hipError_t launch_cache_read(const CacheView &c, const CacheRows &r, int dtype, int64_t tokens, const int64_t *slots,
                             hipStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((tokens + CACHE_BLOCK - 1) / CACHE_BLOCK), static_cast<unsigned>(c.heads), 2),
        block(256);
    by_lanes(c.Dp, [&](auto lpr) {
        if (dtype == DT_F32) hipLaunchKernelGGL((k_cache_read<DT_F32, lpr>), grid, block, 0, stream, c, r, slots, tokens);
        else hipLaunchKernelGGL((k_cache_read<DT_BF16, lpr>), grid, block, 0, stream, c, r, slots, tokens);
    });
    return hipGetLastError();
}

} // namespace bl
