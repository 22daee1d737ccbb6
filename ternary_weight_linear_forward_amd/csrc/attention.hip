// attention.hip -- attention of a batch of sequences that share a prefix, over
// the int8 cache.  o = softmax(scale q k^T) v over the prefix's keys and the
// sequence's own, in one pass with a running maximum m and sum l:
//   m' = max(m, s),  l' = l e^(m - m') + e^(s - m'),  o' = o e^(m - m') + e^(s - m') v.
//
// The keys are cut into parts.  A part's rows are the (query, head) pairs that
// see the same keys of one kv head: for the prefix those of every sequence
// (row = token * G + head in group), so that its keys are read once for the
// whole batch; for a sequence's own keys those of its query tokens.  Every part
// leaves (o, m, l) of its rows in the workspace and k_attn_join adds them with
// weights 2^(m - max m).
//
// Arithmetic.  int8 bytes are exact in binary16, so both products run on the
// f16 matrix cores with fp32 accumulation, and no scale touches the operands:
//  - a query row is multiplied by a power of two that brings its largest value
//    into [2^13, 2^14), or up to 2^4 below (rows that share k_attn_tile's power),
//    and rounded to binary16: bf16 queries keep their 8 bits down to 2^-24 of the
//    row's size; fp32 queries are two binary16 terms (22
//    bits).  Scores are then t = <q', k> * K_scale and softmax runs in base 2 on
//    c t with c = scale log2(e) 2^-e per row.
//  - weights p = 2^(c t - m) are multiplied by V_scale / ref * PSCALE, ref a
//    power of two above the V_scales seen, and rounded to binary16 (11 bits; with
//    fp32 queries two terms, 22 bits).  m is any reference, not the maximum: it
//    starts as the first block's, is raised to a block's maximum when a weight of
//    that block overflows binary16, and is lowered, so that the row's largest weight
//    so far comes to 2^13, when one falls below a full binary16 number (p below
//    2^-21 of the reference's): blocks form no maximum unless one of that happens.
//    Weights that are too small even then are multiplied in further rounds, brought
//    up by STEP each, into sums of their own.  l sums the unrounded p.
//    This form costs where scores spread: at a standard deviation of 1.6, 3 and 5 nats
//    11264 rows on 8000 keys of 8 heads of 128 take 84, 324 and 418 us (k_attn_tile,
//    bf16), 5 x 8 rows on 60001 keys 54, 98 and 114 us (k_attn_stream).
#include "attn_plan.h"
#include "cache_core.h"
#include "common.h"
#include "launch.h"
#include "rows.h"

namespace bl {

static_assert(ATTN_BLOCK == CACHE_BLOCK, "the plan counts blocks of the cache");

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr float ATTN_LOG2E = 1.4426950408889634f, ATTN_LN2 = 0.6931471805599453f;

// Range of the weights (see above) for one and for two binary16 terms.
template <int NS>
struct WeightRange;
template <>
struct WeightRange<1> {
    static constexpr float PSCALE = 0x1p7f, LEAST = 0x1p-14f, STEP = 0x1p29f;
};
template <>
struct WeightRange<2> { // the second term of 2^-3 still has a full 2^-24 of its own
    static constexpr float PSCALE = 0x1p14f, LEAST = 0x1p-3f, STEP = 0x1p18f;
};

// A weight to NS binary16 terms.  With two the weight is a binary32 number before it
// is split: the compiler may otherwise form a product's first term twice, once from
// the product rounded to binary32 and once (v_fma_mixlo_f16) from the exact one, which
// differ by a step of binary16 where the first rounding meets a middle, and the second
// term would be that of the other.
template <int NS>
__device__ __forceinline__ void split_weight(float w, h8 (&p)[NS], int e)
{
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (NS == 2) asm("" : "+v"(w));
#endif
    const _Float16 hi = static_cast<_Float16>(w);
    p[0][e] = hi;
    if constexpr (NS == 2) p[1][e] = static_cast<_Float16>(w - static_cast<float>(hi));
}

template <int NS>
__device__ __forceinline__ void split_weights(const float (&w)[8], h8 (&p)[NS])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) split_weight<NS>(w[e], p, e);
}

// A weight's share of a round: brought up by 'up' = STEP, STEP^2, .. into [LEAST,
// LEAST STEP), 0 in the other rounds; up = 1: the weights of at least LEAST.
// more: smaller ones are left.
template <int NS>
__device__ __forceinline__ float round_share(float w, float up, bool &more)
{
    using WR = WeightRange<NS>;
    const float y = w * up;
    more = more || (y > 0.0f && y < WR::LEAST);
    return y >= WR::LEAST && (up == 1.0f || y < WR::LEAST * WR::STEP) ? y : 0.0f;
}

// Largest and smallest of NT operands' first terms (NaN if one is NaN).
template <int NT, int NS>
__device__ __forceinline__ void weight_range(const h8 (&p)[NT][NS], float &big, float &small)
{
    h2 hi, lo;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        union {
            h8 v;
            h2 x[4];
        } u;
        u.v = p[t][0];
        if (t == 0) {
            hi = __builtin_elementwise_maximum(u.x[0], u.x[1]);
            lo = __builtin_elementwise_minimum(u.x[0], u.x[1]);
        } else {
            hi = __builtin_elementwise_maximum(__builtin_elementwise_maximum(hi, u.x[0]), u.x[1]);
            lo = __builtin_elementwise_minimum(__builtin_elementwise_minimum(lo, u.x[0]), u.x[1]);
        }
        hi = __builtin_elementwise_maximum(__builtin_elementwise_maximum(hi, u.x[2]), u.x[3]);
        lo = __builtin_elementwise_minimum(__builtin_elementwise_minimum(lo, u.x[2]), u.x[3]);
    }
    big = static_cast<float>(__builtin_elementwise_maximum(hi[0], hi[1]));
    small = static_cast<float>(__builtin_elementwise_minimum(lo[0], lo[1]));
}
constexpr float H_MAX = 65504.0f;   // largest binary16
constexpr float SUM_MAX = 0x1p100f; // a block's sum of p beyond which the reference is raised

// Whether a block's weights ask for the general form (bit operators: no branches).
__device__ __forceinline__ bool calls_for_general(bool unset, float big, float sum, bool small)
{
    return unset | !(big <= H_MAX) | !(sum <= SUM_MAX) | small;
}

// What the compiler may not put off: it would keep all the terms until then.
__device__ __forceinline__ void pin(float &v)
{
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(v));
#endif
}

// Power of two at or above v > 0 (as a factor that never overflows).
__device__ __forceinline__ float pow2_above(float v)
{
    const uint32_t e = (__float_as_uint(v) + 0x007fffffu) >> 23;
    return __uint_as_float(min(max(e, 16u), 253u) << 23);
}

// Small weights: what a row's weights can be multiplied with so that the largest so
// far, have, comes to [2^13, 2^14) (a power of two, at least 1; sums stay in range).
__device__ __forceinline__ float lift(float have, float sum)
{
    const float f = 0x1p13f / pow2_above(fmaxf(have, 0x1p-80f)), room = 0x1p90f / pow2_above(fmaxf(sum, 1.0f));
    return fmaxf(1.0f, fminf(f, room));
}

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Own keys query i of a sequence sees: own_len - n + i + 1, within [0, own_len].
__device__ __forceinline__ int attn_own_limit(int own_len, int n, int i)
{
    const int64_t v = static_cast<int64_t>(own_len) - n + i + 1;
    return v < 0 ? 0 : (v > own_len ? own_len : static_cast<int>(v));
}

// Eight int8 (two words) to binary16, exactly: byte x + 128 below the exponent
// byte of 1024 is the binary16 number 1024 + x + 128.
__device__ __forceinline__ h8 bytes_to_h8(uint32_t a, uint32_t b)
{
    const h2 off = {static_cast<_Float16>(-1152.0f), static_cast<_Float16>(-1152.0f)};
    a ^= 0x80808080u;
    b ^= 0x80808080u;
    union {
        h2 p[4];
        h8 v;
    } r;
    r.p[0] = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, a, 0x04010400u)) + off;
    r.p[1] = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u)) + off;
    r.p[2] = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u)) + off;
    r.p[3] = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)) + off;
    return r.v;
}

// v of this lane and of lane ^ 32 (lane ^ 16), in both lanes: the swap of a
// register's halves (rows) with a copy's.
__device__ __forceinline__ void halves32(float v, float &a, float &b)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
#else
    a = b = v;
#endif
}
__device__ __forceinline__ void halves16(float v, float &a, float &b)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    a = __uint_as_float(r[0]);
    b = __uint_as_float(r[1]);
#else
    a = b = v;
#endif
}
__device__ __forceinline__ float max_across32(float v)
{
    float a, b;
    halves32(v, a, b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float max_across16(float v)
{
    float a, b;
    halves16(v, a, b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float sum_across32(float v)
{
    float a, b;
    halves32(v, a, b);
    return a + b;
}
__device__ __forceinline__ float sum_across16(float v)
{
    float a, b;
    halves16(v, a, b);
    return a + b;
}

// A load at a uniform address and a lane's offset in bytes: global_load with a
// scalar base, so that no 64-bit sums are kept across a loop.  The address space is
// named because the compiler may not see through the empty asm, and a flat load
// would count among the LDS's: every wait for an operand read would wait for it.
template <class T>
__device__ __forceinline__ T load_at(const void *base, uint32_t offset)
{
#if defined(__HIP_DEVICE_COMPILE__)
    typedef const __attribute__((address_space(1))) uint8_t *bytes_t;
    typedef const __attribute__((address_space(1))) T *at_t;
    bytes_t p = reinterpret_cast<bytes_t>(reinterpret_cast<uintptr_t>(base));
    asm volatile("" : "+s"(p), "+v"(offset));
    return *reinterpret_cast<at_t>(p + offset);
#else
    return T();
#endif
}

// One part's rows and keys, the same for a whole workgroup.  The keys are a list
// of blocks of 64: nbp blocks of the prefix (0: none of them in this part's list),
// then blocks of the sequence's own keys.
struct AttnJob {
    int kvh, row0, rows, tok0, n; // head, rows of the tile, first token, query tokens
    int nbp, prefix, own;         // prefix blocks and keys, own keys
    int blk0, blk1;               // this part's blocks
    int part;
    const int32_t *prefix_pages, *own_pages;
};

__device__ __forceinline__ bool attn_job(const AttnArgs &a, const AttnPlan &pl, int tile_rows, int wg, AttnJob &j)
{
    const int G = a.heads / a.c.heads, nbp = (a.prefix + CACHE_BLOCK - 1) / CACHE_BLOCK;
    j.prefix_pages = a.prefix_pages;
    j.prefix = a.prefix;
    if (wg < pl.wgs_prefix) {
        // the rows of every sequence against a piece of the prefix; consecutive workgroups
        // take other heads and pieces, so that the row tiles of one piece lie on one XCD
        const int per = a.c.heads * pl.splits_prefix;
        const int tile = wg / per, r = wg % per;
        j.kvh = r % a.c.heads;
        j.part = r / a.c.heads;
        j.tok0 = 0;
        j.n = a.tokens;
        j.row0 = tile * tile_rows;
        j.rows = min(tile_rows, a.tokens * G - j.row0);
        if (j.rows <= 0) return false; // (no plan has such a tile; its queries would lie past Q)
        j.nbp = nbp;
        j.own = 0;
        j.own_pages = nullptr;
        j.blk0 = j.part * pl.chunk_prefix;
        j.blk1 = min(j.blk0 + pl.chunk_prefix, nbp);
        return true;
    }
    // a sequence's rows against its own keys, after the prefix's where the plan joins them
    int r = wg - pl.wgs_prefix;
    j.kvh = r % a.c.heads;
    r /= a.c.heads;
    const int s = r % pl.splits_own;
    r /= pl.splits_own;
    const int tile = r % pl.tiles_own, b = r / pl.tiles_own;
    int first = b * a.max_q, n = a.max_q;
    if (a.q_start) {
        first = a.q_start[b];
        n = min(max(a.q_start[b + 1] - first, 0), a.max_q);
        if (first < 0 || first > a.tokens - n) return false;
    }
    j.tok0 = first;
    j.n = n;
    j.row0 = tile * tile_rows;
    j.rows = min(tile_rows, n * G - j.row0);
    if (j.rows <= 0) return false;
    j.nbp = pl.joint ? nbp : 0;
    j.own = min(max(a.own_len[b], 0), a.max_own);
    const int last = attn_own_limit(j.own, n, (j.row0 + j.rows - 1) / G); // the tile's furthest key
    j.blk0 = s * pl.chunk_own;
    j.blk1 = min(j.blk0 + pl.chunk_own, j.nbp + (last + CACHE_BLOCK - 1) / CACHE_BLOCK);
    j.part = pl.splits_prefix + s;
    j.own_pages = a.own_pages + b * a.ld_pages;
    return true;
}

// Own keys row rho (of the tile) sees; 0 past the tile's rows.
__device__ __forceinline__ int row_limit(const AttnJob &j, int G, int rho)
{
    return rho < j.rows ? attn_own_limit(j.own, j.n, (j.row0 + rho) / G) : 0;
}

// Workspace: o of every (part, token, head) [Dp], then (m, l) of every one.
__device__ __forceinline__ int64_t part_index(const AttnArgs &a, int part, int64_t tok, int head)
{
    return (static_cast<int64_t>(part) * a.tokens + tok) * a.heads + head;
}

// Four columns of a row's result: o / l, rounded once to the output's type.
template <int DT>
__device__ __forceinline__ void store_result(const AttnArgs &a, int64_t tok, int head, int col, f4 v)
{
    const int64_t at = tok * a.ldo_t + head * a.ldo_h + col;
    if (col + 4 <= a.c.D) {
        if constexpr (DT == DT_F32) {
            typedef float f4_any __attribute__((ext_vector_type(4), aligned(4)));
            *reinterpret_cast<f4_any *>(static_cast<float *>(a.O) + at) = v;
        } else {
            const uint32_t lo = float_to_bf16_rne(v[0]) | static_cast<uint32_t>(float_to_bf16_rne(v[1])) << 16,
                           hi = float_to_bf16_rne(v[2]) | static_cast<uint32_t>(float_to_bf16_rne(v[3])) << 16;
            *reinterpret_cast<u2_any *>(static_cast<uint16_t *>(a.O) + at) = u2_any{lo, hi};
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (col + e < a.c.D) {
            if constexpr (DT == DT_F32) static_cast<float *>(a.O)[at + e] = v[e];
            else static_cast<uint16_t *>(a.O)[at + e] = float_to_bf16_rne(v[e]);
        }
}

// log(sum e^s) from a base-2 reference and sum.
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.0f ? (m + log2f(l)) * ATTN_LN2 : neg_inf(); }

// Where 64 blocks of a job lie, lane x holding block first + step x: the number of
// the block among all blocks of the cache (page, head and place in the page), 0 for a
// page outside the cache or a block past the job's, whose bit of valid is 0.  A block
// is then one read of a lane, with no page list, division or test in the loop.
struct BlockTable {
    int unit;
    unsigned long long valid;
    __device__ __forceinline__ void load(const AttnArgs &a, const AttnJob &j, int first, int step)
    {
        const int blk = first + step * lane_id(), bpp = a.c.page_tokens / CACHE_BLOCK;
        int page = -1;
        unit = 0;
        if (blk < j.blk1) {
            const int rel = blk < j.nbp ? blk : blk - j.nbp, pi = rel / bpp;
            page = (blk < j.nbp ? j.prefix_pages : j.own_pages)[pi];
            if (page >= 0 && page < a.c.pages)
                unit = static_cast<int>(cache_row0(a.c, page, j.kvh) / CACHE_BLOCK) + rel - pi * bpp;
            else page = -1;
        }
        valid = __ballot(page >= 0);
    }
    __device__ __forceinline__ uint32_t at(int x) const { return __builtin_amdgcn_readlane(unit, x); } // x uniform
    __device__ __forceinline__ bool there(int x) const { return valid >> x & 1; }
};
// A block's first byte of K (and V), and of its K_scales (and V_scales).
__device__ __forceinline__ const int8_t *block_bytes(const int8_t *p, uint32_t unit, int Dp)
{
    return p + static_cast<uint64_t>(unit) * static_cast<uint32_t>(CACHE_BLOCK * Dp);
}
__device__ __forceinline__ const float *block_scales(const float *p, uint32_t unit)
{
    return p + static_cast<uint64_t>(unit) * CACHE_BLOCK;
}

// A row's power of two: 2^e with max|q| 2^e in [2^13, 2^14); 1 for a zero row.
__device__ __forceinline__ int row_exponent(float top)
{
    if (!(top > 0.0f)) return 0;
    int e;
    (void)frexpf(top, &e); // top = f 2^e, f in [1/2, 1)
    return 14 - e;
}

// A row's factor from scores to base-2 exponents: positive (the sign of scale,
// or 0, goes into the query) and never 0, so that 0 * inf is not formed.
__device__ __forceinline__ float row_factor(float scale, int e2)
{
    return scale != 0.0f ? fmaxf(ldexpf(fabsf(scale) * ATTN_LOG2E, -e2), 1.17549435e-38f) : 1.0f;
}

// NV times eight query values of a row, the n-th at column col(n), zeros past
// head_dim.  With head_dim a multiple of 8 the loads are unconditional (a column
// past the row reads its start), so that they go out together.
template <int DT, int NV, class Col>
__device__ __forceinline__ void load_queries(const AttnArgs &a, int64_t off, const Col &col, float (&v)[NV][8])
{
    if (a.c.D % 8 == 0) {
#pragma unroll
        for (int n = 0; n < NV; ++n) load8<DT>(a.Q, off + (col(n) < a.c.D ? col(n) : 0), 8, v[n]);
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[n][e] = col(n) < a.c.D ? v[n][e] : 0.0f;
    } else {
#pragma unroll
        for (int n = 0; n < NV; ++n) load8<DT>(a.Q, off + col(n), a.c.D - col(n), v[n]);
    }
}

// Eight query values times 2^e2 and the sign of scale as NS binary16 terms.
template <int NS>
__device__ __forceinline__ void query_terms(const float (&v)[8], int e2, float scale, h8 (&q)[NS])
{
    const float sgn = scale < 0.0f ? -1.0f : (scale > 0.0f ? 1.0f : 0.0f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = ldexpf(v[e], e2) * sgn;
        const _Float16 hi = static_cast<_Float16>(x);
        q[0][e] = hi;
        if constexpr (NS == 2) q[1][e] = static_cast<_Float16>(x - static_cast<float>(hi));
    }
}

__device__ __forceinline__ float max_abs8(const float (&v)[8])
{
    float t = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) t = fmaxf(t, fabsf(v[e]));
    return t;
}

// ---------------------------------------------------------------------------
// Few rows: k_attn_stream.  A wave takes 16 rows and streams blocks of 64 keys
// from memory straight into matrix-core operands: lane (i = lane % 16, g = lane /
// 16) loads 16 bytes of key 16 T + i (a K row's columns 64 c + 16 g ..) and 16
// bytes of V's row d = 16 dt + i (keys 4g .. 4g + 3 of the four 16-key tiles).
// S^T = K Q^T leaves keys 4g .. 4g + 3 of a tile in lane (row i, g), which is the
// operand order of O^T += V^T P^T: the weights never leave their lane.  The waves of
// a workgroup (one, two or four) take the chunk's blocks in turn and add their sums
// in LDS.
// Bound: HBM (the bytes of the cache) for 16 rows, no LDS and no barrier in the loop:
// 2 x 8 rows on 60001 keys of 8 heads of 128, 127 MB: 26 us, 4.9 TB/s.  With more row
// tiles the conversion of each (5 x 8 rows: 53 us, 376 MB through L2); with 176
// sequences' own keys of up to 512, 1408 jobs of unequal length, the longest one (31
// us for 107 MB: a wave alone takes 3 us a block).  More rows a wave (two and three
// tiles on one conversion) need registers past 256 and came to the same.
// ---------------------------------------------------------------------------
template <int DT, int DC>
__global__ __launch_bounds__(256, DC == 4 ? 1 : 2) void k_attn_stream(const AttnArgs a, const AttnPlan pl)
{
    constexpr int NS = DT == DT_F32 ? 2 : 1; // binary16 terms of queries and weights
    using WR = WeightRange<NS>;
    constexpr int DTILES = 4 * DC, DPAD = 64 * DC;
    // [waves][16 rows][DPAD] sums, then [waves][16] m, [waves][16] l, [16] l of all
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const int waves = blockDim.x / 64;
    AttnJob j;
    if (!attn_job(a, pl, 16, blockIdx.x + pl.wg0, j)) return;
    const int G = a.heads / a.c.heads, lane = lane_id(), wave = wave_id(), i = lane & 15, g = lane >> 4;
    const int Dp = a.c.Dp;

    u4 kb[4][DC], vb[DTILES];
    f4 ks[4], vs[4];
    // byte offsets of this lane inside a block (columns past Dp read column 0: the queries hold zeros there)
    uint32_t koff[DC], voff[DTILES];
#pragma unroll
    for (int cc = 0; cc < DC; ++cc) koff[cc] = i * Dp + (64 * cc + 16 * g < Dp ? 64 * cc + 16 * g : 0);
#pragma unroll
    for (int d = 0; d < DTILES; ++d) voff[d] = (16 * d < Dp ? 16 * d + i : i) * CACHE_BLOCK + 16 * g;
    auto load_k = [&](uint32_t unit) {
        const int8_t *p = block_bytes(a.c.K, unit, Dp);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int cc = 0; cc < DC; ++cc) kb[t][cc] = load_at<u4>(p + 16 * t * Dp, koff[cc]);
    };
    auto load_v = [&](uint32_t unit) { // and the scales
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            ks[t] = load_at<f4>(block_scales(a.c.Ks, unit) + 16 * t, 16 * g);
            vs[t] = load_at<f4>(block_scales(a.c.Vs, unit) + 16 * t, 16 * g);
        }
#pragma unroll
        for (int d = 0; d < DTILES; ++d) vb[d] = load_at<u4>(block_bytes(a.c.V, unit, Dp), voff[d]);
    };
    // the wave's blocks, the first one in flight while the queries are read
    BlockTable table;
    int blk = j.blk0 + wave;
    unsigned left = 0;
    uint32_t unit = 0;
    bool there = false;
    if (blk < j.blk1) {
        table.load(a, j, blk, waves);
        unit = table.at(0);
        there = table.there(0);
        load_k(unit);
        load_v(unit);
    }

    h8 q[DC][2][NS]; // 64-column chunk, k-step, term
    float c;
    {
        const int rr = i < j.rows ? j.row0 + i : j.row0;
        const int64_t off = (j.tok0 + static_cast<int64_t>(rr / G)) * a.ldq_t + (j.kvh * G + rr % G) * a.ldq_h;
        float v[2 * DC][8], top = 0.0f;
        load_queries<DT>(a, off, [&](int n) { return 64 * (n / 2) + 16 * g + 8 * (n % 2); }, v);
#pragma unroll
        for (int n = 0; n < 2 * DC; ++n) top = fmaxf(top, max_abs8(v[n]));
        top = max_across32(max_across16(top));
        const int e2 = row_exponent(top);
#pragma unroll
        for (int cc = 0; cc < DC; ++cc)
#pragma unroll
            for (int h = 0; h < 2; ++h) query_terms<NS>(v[2 * cc + h], e2, a.scale, q[cc][h]);
        c = row_factor(a.scale, e2);
    }
    // own keys the lane's row sees; below the smallest of the tile's no key is masked
    const int lim = row_limit(j, G, i);
    int lim_min = i < j.rows ? lim : 0x7fffffff;
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) lim_min = min(lim_min, __shfl_xor(lim_min, x));
    lim_min = __builtin_amdgcn_readfirstlane(lim_min);

    f4 o[DTILES];
    // m: the row's reference in base 2 (0 until it is set), have: its largest weight so far
    // (what this lane saw of it), ref: the power of two of the V_scales that the row sees (a row sees
    // what the rows before it see: where the first one's is set, all are)
    float m = 0.0f, l = 0.0f, have = 0.0f, ref = 0.0f, vscale = 0.0f;
    bool set = false;
#pragma unroll
    for (int d = 0; d < DTILES; ++d) o[d] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    for (; blk < j.blk1; blk += waves) {
        // this block's list: its first key and those the lane's row sees
        const bool pre = blk < j.nbp;
        const int k0 = (pre ? blk : blk - j.nbp) * CACHE_BLOCK;
        const int mine = there ? (pre ? j.prefix : lim) : 0;
        const bool masked = !there || k0 + CACHE_BLOCK > (pre ? j.prefix : lim_min);
        const bool next = blk + waves < j.blk1;
        if (next) {
            if (++left % 64 == 0) table.load(a, j, blk + waves, waves);
            unit = table.at(left % 64);
            there = table.there(left % 64);
        }
        f4 s[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            s[t] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int cc = 0; cc < DC; ++cc)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const h8 kf = bytes_to_h8(kb[t][cc][2 * h], kb[t][cc][2 * h + 1]);
#pragma unroll
                    for (int z = 0; z < NS; ++z) s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[cc][h][z], s[t], 0, 0, 0);
                }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) s[t] *= ks[t] * c;
        if (masked) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = k0 + 16 * t + 4 * g + e;
                    s[t][e] = key < mine ? s[t][e] : neg_inf();
                    vs[t][e] = key < mine ? vs[t][e] : 0.0f; // (a hidden one may be anything)
                }
        }
        // the next block's keys, while this block's weights are formed
        if (next) load_k(unit);
        h8 p[2][NS];
        float sum = 0.0f, big = __builtin_inff(), small = 0.0f;
        // (before any V_scale was seen, a wave's first block as a rule, the general form is all there is)
        bool rare = __builtin_amdgcn_readfirstlane(__float_as_int(ref)) == 0;
        if (!rare) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = __builtin_amdgcn_exp2f(s[2 * h + e / 4][e % 4] - m);
                    sum += x;
                    w[e] = x * (vs[2 * h + e / 4][e % 4] * vscale);
                }
                split_weights<NS>(w, p[h]);
            }
            weight_range(p, big, small);
            if (masked) { // (masked weights are 0 and call for nothing)
                small = WR::LEAST;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    small = s[e / 4][e % 4] > neg_inf() ? fminf(small, static_cast<float>(p[e / 8][0][e % 8])) : small;
            }
            rare = __any(calls_for_general(!set && k0 < mine, big, sum, small < WR::LEAST));
        }
        if (rare) {
            // the general form: references brought to this block's largest, small weights in rounds
            float vtop = 0.0f, grown = 1.0f;
#pragma unroll
            for (int t = 0; t < 4; ++t) vtop = fmaxf(fmaxf(fmaxf(vtop, vs[t][0]), fmaxf(vs[t][1], vs[t][2])), vs[t][3]);
            vtop = max_across32(max_across16(vtop));
            if (vtop > ref) {
                const float ref2 = pow2_above(vtop);
                grown = ref / ref2;
                ref = ref2;
                vscale = WR::PSCALE / ref;
            }
            float top = neg_inf();
#pragma unroll
            for (int t = 0; t < 4; ++t) top = fmaxf(fmaxf(fmaxf(top, s[t][0]), fmaxf(s[t][1], s[t][2])), s[t][3]);
            top = max_across32(max_across16(top));
            big = max_across32(max_across16(big));
            sum = max_across32(max_across16(sum));
            const bool raise = top > neg_inf() && (!set || (top > m && (!(big <= H_MAX) || !(sum <= SUM_MAX))));
            const float f = raise && set ? __builtin_amdgcn_exp2f(m - top) : 1.0f;
            m = raise ? top : m;
            set = set || raise;
            l *= f;
#pragma unroll
            for (int d = 0; d < DTILES; ++d) o[d] *= f * grown;
            sum = big = 0.0f;
            small = WR::LEAST;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[t][e] = __builtin_amdgcn_exp2f(s[t][e] - m);
                    sum += s[t][e];
                    s[t][e] *= vs[t][e] * vscale;
                    big = fmaxf(big, s[t][e]);
                    small = s[t][e] > 0.0f ? fminf(small, s[t][e]) : small;
                }
            have = max_across32(max_across16(fmaxf(have * (f * grown), big)));
            big = 0.0f; // (it is in have)
            if (__any(small < WR::LEAST)) {
                small = -max_across32(max_across16(-small));
                const float up = small < WR::LEAST ? lift(have, max_across32(max_across16(l + sum))) : 1.0f;
                m -= __builtin_log2f(up);
                l *= up;
                sum *= up;
                have *= up;
#pragma unroll
                for (int d = 0; d < DTILES; ++d) o[d] *= up;
#pragma unroll
                for (int t = 0; t < 4; ++t) s[t] *= up;
                small *= up;
            }
            const bool rounds = __any(small < WR::LEAST);
            auto share = [&](float up, bool &more) {
                more = false;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = s[2 * h + e / 4][e % 4];
                        w[e] = rounds ? round_share<NS>(y, up, more) : y;
                    }
                    split_weights<NS>(w, p[h]);
                }
                more = __any(more);
            };
            bool more;
            share(1.0f, more);
            if (more) {
                for (float up = WR::STEP, down = 1.0f / WR::STEP; more; up *= WR::STEP, down *= 1.0f / WR::STEP) {
                    share(up, more);
#pragma unroll
                    for (int d = 0; d < DTILES; ++d) {
                        f4 x = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            // (opaque: else the conversions of all tiles are shared with the product below and kept)
                            uint32_t v0 = vb[d][2 * h], v1 = vb[d][2 * h + 1];
                            asm volatile("" : "+v"(v0), "+v"(v1));
                            const h8 vv = bytes_to_h8(v0, v1);
#pragma unroll
                            for (int z = 0; z < NS; ++z) x = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, p[h][z], x, 0, 0, 0);
                        }
                        o[d] += x * down;
                        __builtin_amdgcn_sched_barrier(0); // one tile's registers at a time
                    }
                }
                share(1.0f, more);
            }
        }
        l += sum;
        have = fmaxf(have, big);
#pragma unroll
        for (int d = 0; d < DTILES; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const h8 vv = bytes_to_h8(vb[d][2 * h], vb[d][2 * h + 1]);
#pragma unroll
                for (int z = 0; z < NS; ++z) o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, p[h][z], o[d], 0, 0, 0);
            }
        if (next) load_v(unit);
    }

    // add the waves: largest m of each row, every wave's sums brought to it
    f4 *po = reinterpret_cast<f4 *>(a.ws);
    float2 *pml = reinterpret_cast<float2 *>(a.ws + pl.ml_off);
    float *ml = lds + waves * 16 * DPAD, *ll = ml + waves * 16, *sums = ll + waves * 16; // l of the rows
    l = sum_across32(sum_across16(l));
    m = set ? m : neg_inf();
    if (g == 0) {
        ml[wave * 16 + i] = m;
        ll[wave * 16 + i] = l;
    }
    __syncthreads();
    {
        float top = neg_inf();
        for (int w = 0; w < waves; ++w) top = fmaxf(top, ml[w * 16 + i]);
        const float f = m > neg_inf() ? __builtin_amdgcn_exp2f(m - top) * (ref / WR::PSCALE) : 0.0f;
        float *dst = lds + (wave * 16 + i) * DPAD;
#pragma unroll
        for (int d = 0; d < DTILES; ++d) *reinterpret_cast<f4 *>(dst + 16 * d + 4 * g) = o[d] * f;
    }
    __syncthreads();
    if (threadIdx.x < 16) {
        float top = neg_inf(), sum = 0.0f;
        for (int w = 0; w < waves; ++w) top = fmaxf(top, ml[w * 16 + threadIdx.x]);
        for (int w = 0; w < waves; ++w) {
            const float mw = ml[w * 16 + threadIdx.x];
            if (mw > neg_inf()) sum += ll[w * 16 + threadIdx.x] * __builtin_amdgcn_exp2f(mw - top);
        }
        sums[threadIdx.x] = sum;
        const int rr = j.row0 + static_cast<int>(threadIdx.x);
        if (static_cast<int>(threadIdx.x) < j.rows) {
            const int64_t tok = j.tok0 + rr / G;
            const int head = j.kvh * G + rr % G;
            if (!pl.direct) pml[part_index(a, j.part, tok, head)] = make_float2(top, sum);
            else if (a.lse) a.lse[tok * a.heads + head] = lse_of(top, sum);
        }
    }
    if (pl.direct) __syncthreads();
    for (int e = threadIdx.x; e < j.rows * (Dp / 4); e += blockDim.x) {
        const int rho = e / (Dp / 4), d4 = e % (Dp / 4), rr = j.row0 + rho;
        f4 sum = f4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int w = 0; w < waves; ++w) sum += *reinterpret_cast<const f4 *>(lds + (w * 16 + rho) * DPAD + 4 * d4);
        const int64_t tok = j.tok0 + rr / G;
        const int head = j.kvh * G + rr % G;
        if (pl.direct) store_result<DT>(a, tok, head, 4 * d4, sum * (sums[rho] > 0.0f ? 1.0f / sums[rho] : 0.0f));
        else po[part_index(a, j.part, tok, head) * (Dp / 4) + d4] = sum;
    }
}

// ---------------------------------------------------------------------------
// Many rows: k_attn_tile.  A workgroup of NW waves takes 32 NW rows (a wave 32)
// and a chunk of keys; blocks of 64 keys are converted to binary16 once for the
// workgroup and kept in LDS, two of K and two of V.  S^T = K Q^T in 32 x 32 tiles
// leaves a lane (row = lane % 32, half = lane / 32) keys 8 x + 4 half + {0..3}; two
// such quads are one operand of O^T += V^T P^T, and V is laid out in LDS in that
// order: weights never leave their lane.
//
// A block n is two phases of a wave: P(n), products (sums of block n - 1, scores of
// block n, beside the conversion of the next K and this V), and W(n), its weights.
// P keeps the matrix cores busy and W the vector ALU, so with eight waves the
// second four run one phase behind the first: of the two waves of a SIMD one is in
// P while the other is in W, with a barrier after every phase, and P has the higher
// priority (8000 keys x 11264 rows: 82 us; without the shift 87, without the
// priority 84).  What P(n) writes (K of n + 1, V of n, scales of n + 1) takes places
// that nothing has read since the barrier before either half's P(n), and is read
// from the phase after both halves' P(n) on.  With four waves the other workgroup
// of the CU fills in.  Operands are read from LDS AHEAD of their use (4 to 8 measure
// alike); the bytes converted next are in flight in registers for a whole block.
// Bound: the phases' instruction streams.  11264 rows on 8000 keys of 8 heads of 128
// (46 Gflop): 78 us sustained, 590 Tflop/s (82 in the first launches after an idle
// time, as the figures above); a block takes 5000 cycles of its CU where its
// matrix instructions need 2048 and its vector instructions 2500.  One stream that
// forms the next scores beside the weights, without phases, came to the same (91 us).
// ---------------------------------------------------------------------------
template <int DT, int DC, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_attn_tile(const AttnArgs a, const AttnPlan pl)
{
    constexpr int NS = DT == DT_F32 ? 2 : 1;
    using WR = WeightRange<NS>;
    constexpr int DPAD = 64 * DC, KSTEPS = DPAD / 16, DT32 = DPAD / 32;
    constexpr int UNITS = 4 * DC / NW; // 16-byte units of K (and V) per thread
    // K in LDS: 16-byte unit of 8 columns c8 of a key at ((c8 / 2 + KSTEPS (c8 % 2)) KROW + key); the odd
    // row puts the units of one key into different banks, and an operand's place is a constant apart
    // for every k-step
    constexpr int KROW = 65, KBYTES = 2 * KSTEPS * KROW * 16, VBYTES = 64 * DPAD * 2;
    // two blocks of K, two of V (binary16), three of K_scale and V_scale
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * KBYTES + 2 * VBYTES + 3 * 512];
    auto k_at = [&](int n) { return smem + n * KBYTES; };
    auto v_at = [&](int n) { return smem + 2 * KBYTES + n * VBYTES; };
    auto scales_at = [&](int n) { return reinterpret_cast<float *>(smem + 2 * (KBYTES + VBYTES) + n * 512); };
    AttnJob j;
    if (!attn_job(a, pl, 32 * NW, blockIdx.x + pl.wg0, j)) return;
    const int G = a.heads / a.c.heads, lane = lane_id(), wave = wave_id(), i = lane & 31, hf = lane >> 5;
    const int Dp = a.c.Dp, tid = threadIdx.x, rho = 32 * wave + i;

    u4 kreg[UNITS] = {}, vreg[UNITS] = {};
    // this thread's bytes of a block; columns past Dp read the row's start (the queries hold zeros
    // there), V's rows past Dp its first rows (their sums are not stored)
    uint32_t koff[UNITS], voff[UNITS]; // (unsigned: one register beside a uniform base)
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        const int id = tid + 64 * NW * u, col = 16 * (id % (4 * DC));
        koff[u] = id / (4 * DC) * Dp + (col < Dp ? col : 0);
        voff[u] = (id / 4 < Dp ? id : id % 4) * 16;
    }
    float ksr = 0.0f, vsr = 0.0f;
    int seen = 0; // keys of the fetched block that there are
    // A block's bytes into registers: K and the scales, and V.
    auto fetch_k = [&](int blk, uint32_t unit, bool there) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) kreg[u] = load_at<u4>(block_bytes(a.c.K, unit, Dp), koff[u]);
        ksr = load_at<float>(block_scales(a.c.Ks, unit), 4 * lane);
        vsr = load_at<float>(block_scales(a.c.Vs, unit), 4 * lane);
        // (applied where the scales are written: a use here would wait for the loads)
        seen = there ? (blk < j.nbp ? j.prefix - blk * CACHE_BLOCK : j.own - (blk - j.nbp) * CACHE_BLOCK) : 0;
    };
    auto fetch_v = [&](uint32_t unit) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) vreg[u] = load_at<u4>(block_bytes(a.c.V, unit, Dp), voff[u]);
    };
    // places of block n and of block n + 1, whose K is in registers
    BlockTable table;
    uint32_t unit0 = 0, unit1 = 0;
    bool there0 = false, there1 = false;
    if (j.blk0 < j.blk1) { // (in flight while the queries are read)
        table.load(a, j, j.blk0, 1);
        unit0 = table.at(0);
        there0 = table.there(0);
        fetch_k(j.blk0, unit0, there0);
        fetch_v(unit0);
    }

    // One power of two for all rows whose largest value is within ALIKE binades of the tile's, so that
    // their scores take one factor, held beside the K_scales (it costs such a row what lies below 2^-34
    // of its largest value: half of binary16's least step of 2^-24 against 2^9).  A smaller row has a
    // power of its own, whose difference, shift, comes out of its scores; a row that is not finite takes
    // no part in the choice.  Whatever one row holds, the others keep theirs.
    constexpr int ALIKE = 4;
    h8 q[KSTEPS][NS];
    float c;
    int shift = 0;
    {
        const int rr = rho < j.rows ? j.row0 + rho : j.row0;
        const int64_t off = (j.tok0 + static_cast<int64_t>(rr / G)) * a.ldq_t + (j.kvh * G + rr % G) * a.ldq_h;
        float v[KSTEPS][8], top = 0.0f;
        load_queries<DT>(a, off, [&](int n) { return 16 * n + 8 * hf; }, v);
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k) top = fmaxf(top, max_abs8(v[k]));
        const float row = max_across32(top);
        const bool sized = row > 0.0f && row < __builtin_inff();
        top = wave_max_nonneg(sized ? row : 0.0f);
        float *tops = reinterpret_cast<float *>(smem);
        if (lane == 0) tops[wave] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, tops[w]);
        __syncthreads();
        const int tile_e2 = row_exponent(top), e2 = sized ? row_exponent(row) : tile_e2;
        shift = min(tile_e2 - e2, 0);
        shift = shift < -ALIKE ? shift : 0;
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k) query_terms<NS>(v[k], tile_e2 - shift, a.scale, q[k]);
        c = row_factor(a.scale, tile_e2);
    }
    const bool shifted = __any(shift != 0);
    // own keys the lane's row sees, and the least of the wave's rows: below it nothing is masked
    const int lim = row_limit(j, G, rho);
    int lim_min = rho < j.rows ? lim : 0x7fffffff;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) lim_min = min(lim_min, __shfl_xor(lim_min, x));
    lim_min = __builtin_amdgcn_readfirstlane(lim_min);

    float ref = 0.0f, vscale = 0.0f, grow = 1.0f;
    // Writing the fetched bytes, step by step.  V: unit (2 T + g % 2) * DPAD + d holds
    // quads g and g + 2 of 16-key tile T.
    auto stage_k = [&](int n, uint8_t *to) {
        const int u = n / 2, part = n % 2, id = tid + 64 * NW * u, key = id / (4 * DC), cu = id % (4 * DC);
        reinterpret_cast<h8 *>(to)[(cu + KSTEPS * part) * KROW + key] = bytes_to_h8(kreg[u][2 * part], kreg[u][2 * part + 1]);
    };
    auto stage_v = [&](int n, uint8_t *to) {
        const int u = n / 2, t = 2 * (n % 2), id = tid + 64 * NW * u, d = id / 4, g = id % 4;
        uint2 *pv = reinterpret_cast<uint2 *>(to);
        union {
            h8 v;
            uint2 w[2];
        } x;
        x.v = bytes_to_h8(vreg[u][t], vreg[u][t + 1]);
        pv[((2 * t + (g & 1)) * DPAD + d) * 2 + (g >> 1)] = x.w[0];
        pv[((2 * (t + 1) + (g & 1)) * DPAD + d) * 2 + (g >> 1)] = x.w[1];
    };
    // The scales, and the reference of the V_scales with the factor it asks the sums to be multiplied
    // with before that block's are added (the same in every wave).
    auto stage_scales = [&](float *to) {
        grow = 1.0f;
        ksr = lane < seen ? ksr : 0.0f;
        vsr = lane < seen ? vsr : 0.0f;
        // A V_scale that is not finite leaves the reference as it is and counts as the largest number: its
        // key's weight overflows where a row sees it and is 0 where it is hidden.
        if (__any(vsr > ref)) {
            const float ref2 = fmaxf(pow2_above(wave_max_nonneg(vsr < __builtin_inff() ? vsr : 0.0f)), ref);
            grow = ref / ref2;
            ref = ref2;
            vscale = WR::PSCALE / ref;
        }
        if (wave == 0) {
            to[lane] = fmaxf(ksr * c, 1.17549435e-38f); // (a masked score is -inf: never times 0)
            to[64 + lane] = fminf(vsr * vscale, 3.402823466e38f);
        }
    };
    constexpr int STAGE_STEPS = 4 * UNITS + 1;

    f16v o[DT32];
#pragma unroll
    for (int d = 0; d < DT32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
    float m = 0.0f, l = 0.0f; // m: the row's reference in base 2, 0 until it is set
    bool set = false;
    float have = 0.0f; // the row's largest weight so far (what this lane saw of it)
    f16v s[2];   // the block's scores
    h8 p[4][NS]; // its weights, whose values are added in the next P
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int z = 0; z < NS; ++z)
#pragma unroll
            for (int e = 0; e < 8; ++e) p[x][z][e] = static_cast<_Float16>(0.0f);
    // element e of 16-key tile t is key 16 t + 8 (e / 4) + 4 hf + e % 4
    auto score = [&](int t, int e) { return s[t / 2][8 * (t % 2) + e]; };
    // The weights of the round 'up' (1: those of at least LEAST) as operands; whether smaller ones are left.
    auto share = [&](float up) {
        bool more = false;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = round_share<NS>(score(t, e), up, more);
            split_weights<NS>(w, p[t]);
        }
        return static_cast<bool>(__any(more));
    };
    // Operands of P's products in the order of their use: SUM_OPS of the last block's V (16-key tile by
    // 16-key tile, 32 columns by 32), then SCORE_OPS of K (k-step by k-step, 32 keys by 32), read AHEAD
    // of their use.
    constexpr int SUM_OPS = 4 * DT32, SCORE_OPS = 2 * KSTEPS, AHEAD = 6;
    h8 ring[AHEAD];
    const h8 *pk = nullptr, *pv = nullptr;
    auto read_op = [&](int n) {
        if (n < SUM_OPS) ring[n % AHEAD] = pv[(2 * (n / DT32) + hf) * DPAD + 32 * (n % DT32) + i];
        else if (n < SUM_OPS + SCORE_OPS)
            ring[n % AHEAD] = pk[((n - SUM_OPS) / 2 + KSTEPS * hf) * KROW + 32 * ((n - SUM_OPS) % 2) + i];
    };
    // Step n of adding the last block's weighted values.
    auto sum_step = [&](int n) {
#pragma unroll
        for (int z = 0; z < NS; ++z)
            o[n % DT32] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[n % AHEAD], p[n / DT32][z], o[n % DT32], 0, 0, 0);
    };

    if (j.blk0 < j.blk1) {
#pragma unroll
        for (int n = 0; n < 2 * UNITS; ++n) stage_k(n, k_at(0));
        stage_scales(scales_at(0));
        // (the first P adds zero weights of a block that is not there: its V must be finite)
        for (int n = tid; n < VBYTES / 16; n += 64 * NW) reinterpret_cast<u4 *>(v_at(1))[n] = u4{0, 0, 0, 0};
        if (j.blk0 + 1 < j.blk1) {
            unit1 = table.at(1);
            there1 = table.there(1);
            fetch_k(j.blk0 + 1, unit1, there1);
        }
    }
    __syncthreads();
    const bool behind = NW == 8 && wave >= 4; // the half that runs one phase later
    if (behind) __syncthreads();
    int kbuf = 0, sbuf = 0; // places of block n's K (V the same) and scales
    for (int blk = j.blk0; blk < j.blk1; ++blk) {
        const int snext = sbuf == 2 ? 0 : sbuf + 1;
        // this block's list: its first key and those a row sees
        const bool pre = blk < j.nbp;
        const int k0 = (pre ? blk : blk - j.nbp) * CACHE_BLOCK, mine = there0 ? (pre ? j.prefix : lim) : 0;
        const bool masked = !there0 || k0 + CACHE_BLOCK > (pre ? j.prefix : lim_min);
        // ---- P(blk) ----
        __builtin_amdgcn_s_setprio(2); // (its products go before the other wave's vector instructions)
        pk = reinterpret_cast<const h8 *>(k_at(kbuf));
        pv = reinterpret_cast<const h8 *>(v_at(kbuf ^ 1));
        const float grown = grow; // asked for by this block's scales
#pragma unroll
        for (int n = 0; n < AHEAD; ++n) read_op(n);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < SUM_OPS; ++n) {
            sum_step(n);
            read_op(n + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
#pragma unroll
        for (int n = 0; n < SCORE_OPS; ++n) {
            const int k = n / 2, t = n % 2, at = SUM_OPS + n;
#pragma unroll
            for (int z = 0; z < NS; ++z)
                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ring[at % AHEAD], q[k][z], s[t], 0, 0, 0);
            read_op(at + AHEAD);
            // (after the last block the next K is bytes nothing reads)
#pragma unroll
            for (int x = n * STAGE_STEPS / SCORE_OPS; x < (n + 1) * STAGE_STEPS / SCORE_OPS; ++x) {
                if (x < 2 * UNITS) stage_k(x, k_at(kbuf ^ 1));
                else if (x < 4 * UNITS) stage_v(x - 2 * UNITS, v_at(kbuf));
                else stage_scales(scales_at(snext));
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        const uint32_t this_unit = unit0;
        unit0 = unit1;
        there0 = there1;
        if (blk + 1 < j.blk1) fetch_v(unit1);
        if (blk + 2 < j.blk1) {
            const unsigned x = blk + 2 - j.blk0;
            if (x % 64 == 0) table.load(a, j, blk + 2, 1);
            unit1 = table.at(x % 64);
            there1 = table.there(x % 64);
            fetch_k(blk + 2, unit1, there1);
        }
        __builtin_amdgcn_s_setprio(0);
        if constexpr (NW == 8) __syncthreads();

        // ---- W(blk) ----
        {
            const f4 *sc = reinterpret_cast<const f4 *>(scales_at(sbuf));
            if (shifted) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[t][r] = __builtin_ldexpf(s[t][r], shift);
            }
            if (masked) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int key = k0 + 32 * t + 8 * (r / 4) + 4 * hf + r % 4;
                        s[t][r] = key < mine ? s[t][r] : neg_inf();
                    }
            }
            // two keys a step; scales of a quad of keys, 8 x + 4 hf .., are read two quads ahead
            f4 kq[3], vq[3];
            auto read_scales = [&](int x) {
                kq[x % 3] = sc[2 * x + hf];
                vq[x % 3] = sc[16 + 2 * x + hf];
            };
            float sums[2] = {0.0f, 0.0f}, big, small; // (two chains)
            read_scales(0);
            read_scales(1);
#pragma unroll
            for (int n = 0; n < 16; ++n) {
                const int t = n / 4, e = 2 * (n % 4), quad = n / 2;
                if (n % 2 == 0 && quad + 2 < 8) read_scales(quad + 2);
                float w[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float y =
                        __builtin_amdgcn_exp2f(__builtin_fmaf(score(t, e + x), kq[quad % 3][(e + x) % 4], -m));
                    sums[x] += y;
                    w[x] = y * vq[quad % 3][(e + x) % 4];
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) split_weight<NS>(w[x], p[t], e + x);
#pragma unroll
                for (int x = 0; x < 2; ++x) pin(sums[x]);
                if (n % 2 == 1) __builtin_amdgcn_sched_barrier(0);
            }
            float sum = sums[0] + sums[1];
            weight_range(p, big, small);
            if (masked) { // (masked weights are 0 and call for nothing)
                small = WR::LEAST;
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    small = score(e / 8, e % 8) > neg_inf() ? fminf(small, static_cast<float>(p[e / 8][0][e % 8])) : small;
            }
            if (grown != 1.0f || __any(calls_for_general(!set && k0 < mine, big, sum, small < WR::LEAST))) {
                // the general form: the references brought to the block's, small weights in rounds
                int at = hf; // (the scales are read again, not kept)
                asm volatile("" : "+v"(at));
                float top = neg_inf();
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const f4 k4 = sc[4 * t + 2 * x + at];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            s[t / 2][8 * (t % 2) + 4 * x + r] *= k4[r];
                            top = fmaxf(top, score(t, 4 * x + r));
                        }
                    }
                top = max_across32(top);
                big = max_across32(big);
                sum = max_across32(sum);
                const bool raise = top > neg_inf() && (!set || (top > m && (!(big <= H_MAX) || !(sum <= SUM_MAX))));
                const float f = raise && set ? __builtin_amdgcn_exp2f(m - top) : 1.0f;
                m = raise ? top : m;
                set = set || raise;
                l *= f;
#pragma unroll
                for (int d = 0; d < DT32; ++d) o[d] *= f * grown;
                sum = 0.0f;
                big = 0.0f;
                small = WR::LEAST;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const f4 v4 = sc[16 + 4 * t + 2 * x + at];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float y = __builtin_amdgcn_exp2f(score(t, 4 * x + r) - m);
                            const float w = y * v4[r];
                            sum += y;
                            s[t / 2][8 * (t % 2) + 4 * x + r] = w;
                            big = fmaxf(big, w);
                            small = w > 0.0f ? fminf(small, w) : small;
                        }
                    }
                have = max_across32(fmaxf(have * (f * grown), big));
                big = 0.0f; // (it is in have)
                if (__any(small < WR::LEAST)) {
                    small = -max_across32(-small);
                    const float up = small < WR::LEAST ? lift(have, max_across32(l + sum)) : 1.0f;
                    m -= __builtin_log2f(up);
                    l *= up;
                    sum *= up;
                    have *= up;
#pragma unroll
                    for (int d = 0; d < DT32; ++d) o[d] *= up;
#pragma unroll
                    for (int t = 0; t < 2; ++t) s[t] *= up;
                    small *= up;
                }
                if (!__any(small < WR::LEAST)) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) w[e] = score(t, e);
                        split_weights<NS>(w, p[t]);
                    }
                } else if (share(1.0f)) {
                    // rounds, with V's bytes from memory (another wave may not have written them to LDS yet)
                    const uint8_t *v8 = reinterpret_cast<const uint8_t *>(block_bytes(a.c.V, this_unit, Dp));
                    uint32_t lane_d = i; // (opaque: addresses are formed here, not kept across the blocks)
                    asm volatile("" : "+v"(lane_d));
                    float down = 1.0f / WR::STEP;
                    bool more = true;
                    for (float up = WR::STEP; more; up *= WR::STEP, down *= 1.0f / WR::STEP) {
                        more = share(up);
#pragma unroll
                        for (int d = 0; d < DT32; ++d) {
                            const uint32_t col = 32 * d + lane_d;
                            const uint32_t *row = reinterpret_cast<const uint32_t *>(
                                v8 + (static_cast<int>(col) < Dp ? col : 0u) * CACHE_BLOCK);
                            f16v x;
#pragma unroll
                            for (int r = 0; r < 16; ++r) x[r] = 0.0f;
#pragma unroll
                            for (int t = 0; t < 4; ++t) { // quads hf and hf + 2 of tile t
                                const h8 vv = bytes_to_h8(row[4 * hf + t], row[4 * (hf + 2) + t]);
#pragma unroll
                                for (int z = 0; z < NS; ++z)
                                    x = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, p[t][z], x, 0, 0, 0);
                            }
                            o[d] += x * down;
                            __builtin_amdgcn_sched_barrier(0); // one tile's registers at a time
                        }
                    }
                    (void)share(1.0f);
                }
            }
            l += sum;
            have = fmaxf(have, big);
        }
        kbuf ^= 1;
        sbuf = snext;
        __syncthreads();
    }
    pv = reinterpret_cast<const h8 *>(v_at(kbuf ^ 1));
    if (j.blk0 < j.blk1) {
#pragma unroll
        for (int n = 0; n < SUM_OPS; ++n) {
            if (n % AHEAD == 0) {
#pragma unroll
                for (int x = 0; x < AHEAD; ++x)
                    if (n + x < SUM_OPS) read_op(n + x);
            }
            sum_step(n);
        }
    }
    if (NW == 8 && !behind) __syncthreads();
    l = sum_across32(l);
    if (rho < j.rows) {
        const int rr = j.row0 + rho, head = j.kvh * G + rr % G;
        const int64_t tok = j.tok0 + rr / G, at = part_index(a, j.part, tok, head);
        f4 *po = reinterpret_cast<f4 *>(a.ws) + at * (Dp / 4);
        const float f = ref / WR::PSCALE * (!pl.direct ? 1.0f : (l > 0.0f ? 1.0f / l : 0.0f));
#pragma unroll
        for (int d = 0; d < DT32; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int col = 32 * d + 8 * x + 4 * hf;
                const f4 v = f4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]} * f;
                if (pl.direct) store_result<DT>(a, tok, head, col, v);
                else if (col < Dp) po[col / 4] = v;
            }
        if (hf == 0) {
            if (!pl.direct) reinterpret_cast<float2 *>(a.ws + pl.ml_off)[at] = make_float2(set ? m : neg_inf(), l);
            else if (a.lse) a.lse[tok * a.heads + head] = lse_of(m, l);
        }
    }
}

// Joins the parts of every row.  LPR lanes of four columns each cover a row.  With
// few parts (WIDE false) a group of LPR lanes takes a row and goes through its
// parts four at a time; with many, a wave takes a row, its lanes reading the (m, l)
// of 64 parts at once and 64 / LPR parts' sums side by side.  Bound: HBM / L2: 11264
// rows of 128 from 6 parts, 38 MB: 8.5 us; 320 rows from 20 parts: 5 us.
template <int DT, int LPR, bool WIDE>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a, const AttnPlan pl, int64_t row0, int64_t rows)
{
    constexpr int PER = WIDE ? 64 : LPR; // lanes a row
    const int64_t r = row0 + (blockIdx.x * (256 / PER) + threadIdx.x / PER);
    if (r >= rows) return;
    const int head = static_cast<int>(r % a.heads), lane = lane_id();
    const int64_t bi = r / a.heads;
    const int most = min(a.max_q, a.tokens); // query tokens of a sequence
    const int b = static_cast<int>(bi / most), i = static_cast<int>(bi % most);
    int first = b * a.max_q, n = a.max_q;
    if (a.q_start) {
        first = a.q_start[b];
        n = min(max(a.q_start[b + 1] - first, 0), a.max_q);
        if (first < 0 || first > a.tokens - n) return;
    }
    if (i >= n) return;
    const int64_t tok = static_cast<int64_t>(first) + i;
    const int parts = pl.splits_prefix + pl.splits_own, Dp = a.c.Dp, col = 4 * (lane % LPR);
    const float2 *pml = reinterpret_cast<const float2 *>(a.ws + pl.ml_off);
    float top = neg_inf(), l = 0.0f;
    f4 o = f4{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (!WIDE) {
        for (int p0 = 0; p0 < parts; p0 += 4) {
            float2 x[4];
            f4 v[4];
            float t = top;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t at = part_index(a, min(p0 + u, parts - 1), tok, head);
                x[u] = pml[at];
                v[u] = *reinterpret_cast<const f4 *>(a.ws + at * Dp + (col < Dp ? col : 0));
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (p0 + u >= parts) x[u] = make_float2(neg_inf(), 0.0f);
                t = fmaxf(t, x[u].x);
            }
            if (!(t > neg_inf())) continue;
            const float f = __builtin_amdgcn_exp2f(top - t);
            l *= f;
            o *= f;
            top = t;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float w = __builtin_amdgcn_exp2f(x[u].x - top); // 0 for a part without keys, whose sums are 0
                l += x[u].y * w;
                o += v[u] * w;
            }
        }
    } else {
        for (int p0 = 0; p0 < parts; p0 += 64) {
            const float2 x = p0 + lane < parts ? pml[part_index(a, p0 + lane, tok, head)] : make_float2(neg_inf(), 0.0f);
            float t = x.x;
#pragma unroll
            for (int s = 32; s > 0; s >>= 1) t = fmaxf(t, __shfl_xor(t, s));
            if (!(t > neg_inf())) continue;
            if (t > top) {
                const float f = __builtin_amdgcn_exp2f(top - t); // (0 the first time)
                l *= f;
                o *= f;
                top = t;
            }
            const float f = __builtin_amdgcn_exp2f(x.x - top); // this lane's part; 0 for one without keys
            l += x.y * f;
            const int here = min(64, parts - p0);
            for (int p = 0; p < here; p += 8 * (64 / LPR)) {
                f4 v[8];
                float w[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int q = p + u * (64 / LPR) + lane / LPR;
                    w[u] = __shfl(f, q & 63);
                    w[u] = q < here ? w[u] : 0.0f;
                    v[u] = *reinterpret_cast<const f4 *>(a.ws + part_index(a, p0 + min(q, here - 1), tok, head) * Dp +
                                                         (col < Dp ? col : 0));
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) o += v[u] * w[u];
            }
        }
#pragma unroll
        for (int s = 32; s > 0; s >>= 1) l += __shfl_xor(l, s);
#pragma unroll
        for (int s = LPR; s < 64; s <<= 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], s);
    }
    if (lane % PER < LPR) store_result<DT>(a, tok, head, col, o * (l > 0.0f ? 1.0f / l : 0.0f));
    if (a.lse && lane % PER == 0) a.lse[tok * a.heads + head] = lse_of(top, l);
}

// ---- host -------------------------------------------------------------------
namespace {

template <int DT>
hipError_t launch_part(const AttnArgs &a, AttnPlan pl, int rows, int waves, int64_t first, int64_t wgs, hipStream_t st)
{
    pl.wg0 = static_cast<int>(first);
    const int dc = a.c.Dp <= 64 ? 1 : a.c.Dp <= 128 ? 2 : 4;
    const dim3 grid(static_cast<unsigned>(wgs)), block(64 * waves);
    const size_t lds = (waves * 16 * (64 * dc + 2) + 16) * sizeof(float);
#define BL_STREAM(DC) hipLaunchKernelGGL((k_attn_stream<DT, DC>), grid, block, lds, st, a, pl)
#define BL_TILE(DC, NW) hipLaunchKernelGGL((k_attn_tile<DT, DC, NW>), grid, block, 0, st, a, pl)
    if (rows == 16) {
        if (dc == 1) BL_STREAM(1);
        else if (dc == 2) BL_STREAM(2);
        else BL_STREAM(4);
    } else if (dc == 1) {
        BL_TILE(1, 4);
    } else if constexpr (DT == DT_BF16) {
        if (rows == 128) BL_TILE(2, 4);
        else BL_TILE(2, 8);
    }
#undef BL_STREAM
#undef BL_TILE
    return hipGetLastError();
}

template <int DT>
hipError_t launch_attn(const AttnArgs &a, const AttnPlan &pl, hipStream_t st)
{
    AttnLaunch l[2];
    const int n = attn_launches(pl, l);
    for (int x = 0; x < n; ++x) {
        const hipError_t e = attn_pieces(l[x].wgs, hipSuccess, [&](int64_t at, int64_t wgs) {
            return launch_part<DT>(a, pl, l[x].rows, l[x].waves, l[x].first + at, wgs, st);
        });
        if (e != hipSuccess) return e;
    }
    if (pl.direct) return hipSuccess;
    const int64_t rows = attn_join_rows(a.tokens, a.heads, a.seqs, a.max_q);
    const bool wide = pl.splits_prefix + pl.splits_own > 12;
    const int lpr = a.c.Dp <= 64 ? 16 : a.c.Dp <= 128 ? 32 : 64, rows_wg = 256 / (wide ? 64 : lpr);
    return attn_pieces(div_up(rows, rows_wg), hipSuccess, [&](int64_t at, int64_t wgs) {
        const dim3 grid(static_cast<unsigned>(wgs)), block(256);
        const int64_t row0 = at * rows_wg;
#define BL_JOIN(LPR, WIDE) hipLaunchKernelGGL((k_attn_join<DT, LPR, WIDE>), grid, block, 0, st, a, pl, row0, rows)
        if (wide) {
            if (lpr == 16) BL_JOIN(16, true);
            else if (lpr == 32) BL_JOIN(32, true);
            else BL_JOIN(64, true);
        } else {
            if (lpr == 16) BL_JOIN(16, false);
            else if (lpr == 32) BL_JOIN(32, false);
            else BL_JOIN(64, false);
        }
#undef BL_JOIN
        return hipGetLastError();
    });
}

} // namespace

// Room for either type's plan.
int64_t attn_workspace_bytes(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t seqs,
                             int64_t max_q, int64_t max_own, int64_t prefix)
{
    int64_t most = 0;
    for (const int dtype : {DT_F32, DT_BF16}) {
        const AttnPlan p = attn_plan(tokens, heads, kv_heads, head_dim, seqs, max_q, max_own, prefix, dtype == DT_F32);
        const int64_t need = p.direct ? 0 : (p.ml_off + 2 * (p.splits_prefix + p.splits_own) * tokens * heads) * 4;
        most = need > most ? need : most;
    }
    return most;
}

hipError_t launch_attention(const AttnArgs &a, hipStream_t stream)
{
    const AttnPlan p =
        attn_plan(a.tokens, a.heads, a.c.heads, a.c.D, a.seqs, a.max_q, a.max_own, a.prefix, a.dtype == DT_F32);
    return a.dtype == DT_F32 ? launch_attn<DT_F32>(a, p, stream) : launch_attn<DT_BF16>(a, p, stream);
}

} // namespace bl
