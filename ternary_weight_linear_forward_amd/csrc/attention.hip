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
//    into [2^13, 2^14) and rounded to binary16: bf16 queries keep their 8 bits
//    down to 2^-24 of the row's size; fp32 queries are two binary16 terms (22
//    bits).  Scores are then t = <q', k> * K_scale and softmax runs in base 2 on
//    c t with c = scale log2(e) 2^-e per row.
//  - weights p = 2^(c (t - m)) are multiplied by V_scale / ref * PSCALE, ref the
//    running power of two above the largest V_scale seen, and rounded to
//    binary16 (11 bits; with fp32 queries two terms, 22 bits).  m is raised only
//    when a score passes it by more than SLACK (base 2), so products stay below
//    2^16.  Weights too small for a full binary16 number (a softmax of more than
//    2^21 from its largest to its smallest weight) are multiplied in further
//    rounds, brought up by STEP each, into sums of their own: a branch that
//    blocks without such weights do not take.  l sums the unrounded p.
#include "cache_core.h"
#include "common.h"
#include "launch.h"

namespace bl {

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
    static constexpr float PSCALE = 0x1p7f, SLACK = 8.0f, LEAST = 0x1p-14f, STEP = 0x1p29f;
};
template <>
struct WeightRange<2> { // the second term of 2^-3 still has a full 2^-24 of its own
    static constexpr float PSCALE = 0x1p14f, SLACK = 1.0f, LEAST = 0x1p-3f, STEP = 0x1p18f;
};

// Weights to NS binary16 terms.
template <int NS>
__device__ __forceinline__ void split_weights(const float (&w)[8], h8 (&p)[NS])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const _Float16 hi = static_cast<_Float16>(w[e]);
        p[0][e] = hi;
        if constexpr (NS == 2) p[1][e] = static_cast<_Float16>(w[e] - static_cast<float>(hi));
    }
}

// The weights that 'up' brings into [LEAST, LEAST STEP) (up = STEP, STEP^2, ..
// in turn); the others 0.  Whether smaller ones are left.
template <int NS>
__device__ __forceinline__ bool round_weights(const float (&w)[8], float up, h8 (&p)[NS])
{
    using WR = WeightRange<NS>;
    float x[8];
    bool more = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = w[e] * up;
        more = more || (y > 0.0f && y < WR::LEAST);
        x[e] = y >= WR::LEAST && y < WR::LEAST * WR::STEP ? y : 0.0f;
    }
    split_weights<NS>(x, p);
    return more;
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

__device__ __forceinline__ float max_across32(float v) // lanes l, l ^ 32
{
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float max_across16(float v) // lanes l, l ^ 16
{
    return fmaxf(v, __shfl_xor(v, 16));
}

// Power of two at or above v > 0 (as a factor that never overflows).
__device__ __forceinline__ float pow2_above(float v)
{
    const uint32_t e = (__float_as_uint(v) + 0x007fffffu) >> 23;
    return __uint_as_float(min(max(e, 16u), 253u) << 23);
}

// One part's rows and keys, the same for a whole workgroup.
struct AttnJob {
    int kvh, row0, rows, tok0, n; // rows of the tile, first token, query tokens (own part)
    int own;                      // own length, or -1: prefix
    int blk0, blk1;               // blocks of 64 keys
    int part;
    const int32_t *pages;
    int keys; // all keys of the list
};

__device__ __forceinline__ bool attn_job(const AttnArgs &a, const AttnPlan &pl, int tile_rows_p, int tile_rows_o,
                                         int wg, AttnJob &j)
{
    const int G = a.heads / a.c.heads;
    if (wg < pl.wgs_prefix) {
        // consecutive workgroups go to different XCDs: kv heads and splits first, so
        // that the row tiles of one piece of the cache are 8 apart or on one XCD
        const int per = a.c.heads * pl.splits_prefix;
        const int tile = wg / per, r = wg % per;
        j.kvh = r % a.c.heads;
        const int s = r / a.c.heads;
        j.own = -1;
        j.n = a.tokens;
        j.tok0 = 0;
        j.row0 = tile * tile_rows_p;
        j.rows = min(tile_rows_p, a.tokens * G - j.row0);
        j.blk0 = s * pl.chunk_prefix;
        j.keys = a.prefix;
        j.blk1 = min(j.blk0 + pl.chunk_prefix, (a.prefix + CACHE_BLOCK - 1) / CACHE_BLOCK);
        j.part = s;
        j.pages = a.prefix_pages;
        return true;
    }
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
    j.row0 = tile * tile_rows_o;
    j.rows = min(tile_rows_o, n * G - j.row0);
    if (j.rows <= 0) return false;
    j.own = min(max(a.own_len[b], 0), a.max_own);
    const int last = attn_own_limit(j.own, n, (j.row0 + j.rows - 1) / G); // the tile's furthest key
    j.keys = j.own;
    j.blk0 = s * pl.chunk_own;
    j.blk1 = min(j.blk0 + pl.chunk_own, (last + CACHE_BLOCK - 1) / CACHE_BLOCK);
    j.part = pl.splits_prefix + s;
    j.pages = a.own_pages + b * a.ld_pages;
    return true;
}

// Keys row rho (of the tile) sees; 0 past the tile's rows.
__device__ __forceinline__ int row_limit(const AttnJob &j, int G, int rho)
{
    if (rho >= j.rows) return 0;
    return j.own < 0 ? j.keys : attn_own_limit(j.own, j.n, (j.row0 + rho) / G);
}

// Workspace: o of every (part, token, head) [Dp], then (m, l) of every one.
__device__ __forceinline__ int64_t part_index(const AttnArgs &a, int part, int64_t tok, int head)
{
    return (static_cast<int64_t>(part) * a.tokens + tok) * a.heads + head;
}

// The page of block blk (bpp blocks a page), or -1 where it lies outside the cache.
__device__ __forceinline__ int page_of(const AttnArgs &a, const AttnJob &j, int blk, int bpp)
{
    const int p = j.pages[blk / bpp];
    return p >= 0 && p < a.c.pages ? p : -1;
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

template <int DT>
__device__ __forceinline__ float load_q(const AttnArgs &a, int64_t row_off, int d)
{
    return d < a.c.D ? load_x<DT>(a.Q, row_off + d) : 0.0f;
}

// ---------------------------------------------------------------------------
// Few rows: k_attn_stream.  A wave takes 16 rows and streams blocks of 64 keys
// from memory straight into matrix-core operands: lane (i = lane % 16, g = lane /
// 16) loads 16 bytes of key 16 T + i (a K row's columns 64 c + 16 g ..) and 16
// bytes of V's row d = 16 dt + i (keys 4g .. 4g + 3 of the four 16-key tiles).
// S^T = K Q^T leaves keys 4g .. 4g + 3 of a tile in lane (row i, g), which is the
// operand order of O^T += V^T P^T: the weights never leave their lane.  The four
// waves of a workgroup take the chunk's blocks in turn and add their sums in LDS.
// Bound: HBM (the bytes of the cache); no LDS and no barrier in the loop.
// ---------------------------------------------------------------------------
template <int DT, int DC>
__global__ __launch_bounds__(256, DC == 4 ? 1 : 2) void k_attn_stream(const AttnArgs a, const AttnPlan pl)
{
    constexpr int NS = DT == DT_F32 ? 2 : 1; // binary16 terms of queries and weights
    using WR = WeightRange<NS>;
    constexpr int DTILES = 4 * DC, DPAD = 64 * DC;
    // [4 waves][16 rows][DPAD] sums, then [4][16] m, l
    __shared__ __attribute__((aligned(16))) float lds[4 * 16 * (DPAD + 2)];
    AttnJob j;
    if (!attn_job(a, pl, 16, 16, blockIdx.x + pl.wg0, j)) return;
    const int G = a.heads / a.c.heads, lane = lane_id(), wave = wave_id(), i = lane & 15, g = lane >> 4;
    const int Dp = a.c.Dp, bpp = a.c.page_tokens / CACHE_BLOCK;

    h8 q[NS][DC][2]; // term, 64-column chunk, k-step
    float c;
    {
        const int rr = i < j.rows ? j.row0 + i : j.row0;
        const int64_t off = (j.tok0 + static_cast<int64_t>(rr / G)) * a.ldq_t + (j.kvh * G + rr % G) * a.ldq_h;
        float v[DC][16], top = 0.0f;
#pragma unroll
        for (int cc = 0; cc < DC; ++cc)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                v[cc][e] = load_q<DT>(a, off, 64 * cc + 16 * g + e);
                top = fmaxf(top, fabsf(v[cc][e]));
            }
        top = max_across32(max_across16(top));
        const int e2 = row_exponent(top);
        const float sgn = a.scale < 0.0f ? -1.0f : (a.scale > 0.0f ? 1.0f : 0.0f);
#pragma unroll
        for (int cc = 0; cc < DC; ++cc)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float x = ldexpf(v[cc][e], e2) * sgn;
                const _Float16 hi = static_cast<_Float16>(x);
                q[0][cc][e / 8][e % 8] = hi;
                if constexpr (NS == 2) q[1][cc][e / 8][e % 8] = static_cast<_Float16>(x - static_cast<float>(hi));
            }
        c = row_factor(a.scale, e2);
    }
    // below the smallest limit of the tile's rows no key is masked
    const int lim = row_limit(j, G, i);
    int lim_min = i < j.rows ? lim : 0x7fffffff;
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) lim_min = min(lim_min, __shfl_xor(lim_min, x));
    lim_min = __builtin_amdgcn_readfirstlane(lim_min);

    f4 o[DTILES];
#pragma unroll
    for (int d = 0; d < DTILES; ++d) o[d] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = neg_inf(), l = 0.0f, ref = 0.0f;
    u4 kb[4][DC], vb[DTILES];
    f4 ks[4], vs[4];
    // byte offsets of this lane inside a block (columns past Dp read column 0: the queries hold zeros there)
    int koff[DC], voff[DTILES];
#pragma unroll
    for (int cc = 0; cc < DC; ++cc) koff[cc] = i * Dp + (64 * cc + 16 * g < Dp ? 64 * cc + 16 * g : 0);
#pragma unroll
    for (int d = 0; d < DTILES; ++d) voff[d] = (16 * d < Dp ? 16 * d + i : i) * CACHE_BLOCK + 16 * g;
    auto row_of = [&](int page, int blk) {
        return cache_row0(a.c, page < 0 ? 0 : page, j.kvh) + blk % bpp * CACHE_BLOCK;
    };
    auto load_k = [&](int64_t row) {
        const int8_t *p = a.c.K + row * Dp;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            ks[t] = *reinterpret_cast<const f4 *>(a.c.Ks + row + 16 * t + 4 * g);
            vs[t] = *reinterpret_cast<const f4 *>(a.c.Vs + row + 16 * t + 4 * g);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int cc = 0; cc < DC; ++cc) kb[t][cc] = *reinterpret_cast<const u4 *>(p + 16 * t * Dp + koff[cc]);
    };
    auto load_v = [&](int64_t row) {
        const int8_t *p = a.c.V + row * Dp;
#pragma unroll
        for (int d = 0; d < DTILES; ++d) vb[d] = *reinterpret_cast<const u4 *>(p + voff[d]);
    };
    int blk = j.blk0 + wave;
    int page = blk < j.blk1 ? page_of(a, j, blk, bpp) : -1;
    if (blk < j.blk1) {
        const int64_t row = row_of(page, blk);
        load_k(row);
        load_v(row);
    }
    for (; blk < j.blk1; blk += 4) {
        const int next = blk + 4;
        const int npage = next < j.blk1 ? page_of(a, j, next, bpp) : -1;
        const int k0 = blk * CACHE_BLOCK;
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
                    for (int z = 0; z < NS; ++z) s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, q[z][cc][h], s[t], 0, 0, 0);
                }
        }
        f4 vf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            s[t] *= ks[t];
            vf[t] = vs[t];
        }
        if (page < 0 || k0 + CACHE_BLOCK > lim_min) {
            const int all = page < 0 ? 0 : j.keys, mine = page < 0 ? 0 : lim;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = k0 + 16 * t + 4 * g + r;
                    s[t][r] = key < mine ? s[t][r] : neg_inf();
                    vf[t][r] = key < all ? vf[t][r] : 0.0f;
                }
        }
        // the next block's keys and scales, while this block's weights are formed
        const int64_t nrow = row_of(npage, next);
        if (next < j.blk1) load_k(nrow);
        float vtop = 0.0f, top = neg_inf();
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            vtop = fmaxf(fmaxf(fmaxf(vtop, vf[t][0]), fmaxf(vf[t][1], vf[t][2])), vf[t][3]);
            top = fmaxf(fmaxf(fmaxf(top, s[t][0]), fmaxf(s[t][1], s[t][2])), s[t][3]);
        }
        vtop = max_across32(max_across16(vtop));
        top = max_across32(max_across16(top));
        // (m = -inf: any finite score raises it)
        const bool raise = top > neg_inf() && !((top - m) * c <= WR::SLACK);
        if (vtop > ref || __any(raise)) { // (vtop is the same in every lane)
            const float m2 = raise ? fmaxf(m, top) : m;
            float f = raise ? __builtin_amdgcn_exp2f((m - m2) * c) : 1.0f;
            m = m2;
            l *= f;
            if (vtop > ref) {
                const float ref2 = pow2_above(vtop);
                f *= ref / ref2;
                ref = ref2;
            }
#pragma unroll
            for (int d = 0; d < DTILES; ++d) o[d] *= f;
        }
        const float mc = m > neg_inf() ? m * c : 0.0f, vscale = ref > 0.0f ? WR::PSCALE / ref : 0.0f;
        float w[2][8], least = WR::LEAST;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], c, -mc));
                l += p;
                w[t / 2][4 * (t % 2) + r] = p * (vf[t][r] * vscale);
                least = fminf(least, w[t / 2][4 * (t % 2) + r]);
            }
        if (__any(least < WR::LEAST)) {
            // weights below LEAST: rounds of their own, each brought up by STEP
            float up = WR::STEP, down = 1.0f / WR::STEP;
            for (bool more = true; more; up *= WR::STEP, down *= 1.0f / WR::STEP) {
                h8 p[2][NS];
                more = false;
#pragma unroll
                for (int h = 0; h < 2; ++h) more = round_weights<NS>(w[h], up, p[h]) || more;
                more = __any(more);
#pragma unroll
                for (int d = 0; d < DTILES; ++d) {
                    f4 x = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // (opaque: else the conversions of all tiles are shared with the product below and kept)
                        uint32_t v0 = vb[d][2 * h], v1 = vb[d][2 * h + 1];
                        asm("" : "+v"(v0), "+v"(v1));
                        const h8 vv = bytes_to_h8(v0, v1);
#pragma unroll
                        for (int z = 0; z < NS; ++z) x = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, p[h][z], x, 0, 0, 0);
                    }
                    o[d] += x * down;
                    __builtin_amdgcn_sched_barrier(0); // one tile's registers at a time
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 8; ++e) w[h][e] = w[h][e] >= WR::LEAST ? w[h][e] : 0.0f;
        }
        h8 p[2][NS];
        split_weights<NS>(w[0], p[0]);
        split_weights<NS>(w[1], p[1]);
#pragma unroll
        for (int d = 0; d < DTILES; ++d)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const h8 vv = bytes_to_h8(vb[d][2 * h], vb[d][2 * h + 1]);
#pragma unroll
                for (int z = 0; z < NS; ++z) o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, p[h][z], o[d], 0, 0, 0);
            }
        if (next < j.blk1) load_v(nrow);
        page = npage;
    }

    // add the waves: largest m of each row, every wave's sums brought to it
    float *ml = lds + 4 * 16 * DPAD;
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    m = m > neg_inf() ? m * c : neg_inf();
    if (g == 0) {
        ml[wave * 16 + i] = m;
        ml[64 + wave * 16 + i] = l;
    }
    __syncthreads();
    {
        float top = neg_inf();
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[w * 16 + i]);
        const float f = m > neg_inf() ? __builtin_amdgcn_exp2f(m - top) * (ref / WR::PSCALE) : 0.0f;
        float *dst = lds + (wave * 16 + i) * DPAD;
#pragma unroll
        for (int d = 0; d < DTILES; ++d) *reinterpret_cast<f4 *>(dst + 16 * d + 4 * g) = o[d] * f;
    }
    __syncthreads();
    f4 *po = reinterpret_cast<f4 *>(a.ws);
    float2 *pml = reinterpret_cast<float2 *>(a.ws + pl.ml_off);
    for (int e = threadIdx.x; e < j.rows * (Dp / 4); e += 256) {
        const int rho = e / (Dp / 4), d4 = e % (Dp / 4), rr = j.row0 + rho;
        f4 sum = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += *reinterpret_cast<const f4 *>(lds + (w * 16 + rho) * DPAD + 4 * d4);
        po[part_index(a, j.part, j.tok0 + rr / G, j.kvh * G + rr % G) * (Dp / 4) + d4] = sum;
    }
    if (static_cast<int>(threadIdx.x) < j.rows) {
        const int rho = threadIdx.x, rr = j.row0 + rho;
        float top = neg_inf(), sum = 0.0f;
        for (int w = 0; w < 4; ++w) top = fmaxf(top, ml[w * 16 + rho]);
        for (int w = 0; w < 4; ++w) {
            const float mw = ml[w * 16 + rho];
            if (mw > neg_inf()) sum += ml[64 + w * 16 + rho] * __builtin_amdgcn_exp2f(mw - top);
        }
        pml[part_index(a, j.part, j.tok0 + rr / G, j.kvh * G + rr % G)] = make_float2(top, sum);
    }
}

// ---------------------------------------------------------------------------
// Many rows: k_attn_tile.  A workgroup takes 128 rows (a wave 32) and a chunk of
// keys; blocks of 64 keys are converted to binary16 once for the workgroup and
// kept in two LDS buffers: the next block's bytes are fetched into registers
// before a block is multiplied and written after it, one barrier a block.
// S^T = K Q^T in 32 x 32 tiles leaves a lane (row = lane % 32, half = lane / 32)
// keys 8 x + 4 half + {0..3}; two such quads are one operand of O^T += V^T P^T,
// and V is laid out in LDS in that order: weights never leave their lane.
// Bound: vector ALU (softmax) and matrix cores.
// ---------------------------------------------------------------------------
constexpr int TILE_ROWS_ATTN = 128;

template <int DT, int DC>
__global__ __launch_bounds__(256, DC == 4 ? 1 : 2) void k_attn_tile(const AttnArgs a, const AttnPlan pl)
{
    constexpr int NS = DT == DT_F32 ? 2 : 1;
    using WR = WeightRange<NS>;
    constexpr int DPAD = 64 * DC, KSTEPS = DPAD / 16, DT32 = DPAD / 32, UNITS = DC; // 16-byte units per thread
    constexpr int KBYTES = 64 * DPAD * 2, BUF = 2 * KBYTES + 512;
    // two buffers of K, V (binary16), K_scale, V_scale of a block
    __shared__ __attribute__((aligned(16))) uint8_t smem[2 * BUF];
    AttnJob j;
    if (!attn_job(a, pl, TILE_ROWS_ATTN, TILE_ROWS_ATTN, blockIdx.x + pl.wg0, j)) return;
    const int G = a.heads / a.c.heads, lane = lane_id(), wave = wave_id(), i = lane & 31, hf = lane >> 5;
    const int Dp = a.c.Dp, bpp = a.c.page_tokens / CACHE_BLOCK, tid = threadIdx.x;
    const int rho = 32 * wave + i;

    h8 q[NS][KSTEPS];
    float c;
    {
        const int rr = rho < j.rows ? j.row0 + rho : j.row0;
        const int64_t off = (j.tok0 + static_cast<int64_t>(rr / G)) * a.ldq_t + (j.kvh * G + rr % G) * a.ldq_h;
        float top = 0.0f;
        for (int d = 8 * hf; d < a.c.D; d += 16)
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(load_q<DT>(a, off, d + e)));
        top = max_across32(top);
        const int e2 = row_exponent(top);
        const float sgn = a.scale < 0.0f ? -1.0f : (a.scale > 0.0f ? 1.0f : 0.0f);
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = ldexpf(load_q<DT>(a, off, 16 * k + 8 * hf + e), e2) * sgn;
                const _Float16 hi = static_cast<_Float16>(x);
                q[0][k][e] = hi;
                if constexpr (NS == 2) q[1][k][e] = static_cast<_Float16>(x - static_cast<float>(hi));
            }
        c = row_factor(a.scale, e2);
    }
    const int lim = row_limit(j, G, rho);
    // a wave whose rows all lie past the tile multiplies nothing
    const bool wave_live = 32 * wave < j.rows;
    int lim_min = rho < j.rows ? lim : 0x7fffffff, lim_max = lim;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        lim_min = min(lim_min, __shfl_xor(lim_min, x));
        lim_max = max(lim_max, __shfl_xor(lim_max, x));
    }
    lim_min = __builtin_amdgcn_readfirstlane(lim_min);
    lim_max = __builtin_amdgcn_readfirstlane(lim_max);

    u4 kreg[UNITS], vreg[UNITS];
    float ksr = 0.0f, vsr = 0.0f;
    int page = -1;
    auto fetch = [&](int blk) {
        page = page_of(a, j, blk, bpp);
        const int64_t row = cache_row0(a.c, page < 0 ? 0 : page, j.kvh) + blk % bpp * CACHE_BLOCK;
        const int8_t *pk = a.c.K + row * Dp, *pv = a.c.V + row * Dp;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int id = tid + 256 * u, key = id / (4 * DC), col = 16 * (id % (4 * DC));
            kreg[u] = col < Dp ? *reinterpret_cast<const u4 *>(pk + key * Dp + col) : u4{0, 0, 0, 0};
            vreg[u] = id / 4 < Dp ? *reinterpret_cast<const u4 *>(pv + id * 16) : u4{0, 0, 0, 0};
        }
        const int key = blk * CACHE_BLOCK + lane;
        const bool seen = page >= 0 && key < j.keys;
        ksr = a.c.Ks[row + lane];
        vsr = a.c.Vs[row + lane];
        ksr = seen ? ksr : 0.0f;
        vsr = seen ? vsr : 0.0f;
    };
    float ref = 0.0f;
    // Writes the fetched block into a buffer; returns the factor its V_scale's
    // reference asks the sums to be multiplied with (the same in every wave).
    auto stage = [&](int buf) -> float {
        uint8_t *base = smem + buf * BUF;
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int id = tid + 256 * u, key = id / (4 * DC), cu = id % (4 * DC);
            // K: 16-byte unit (column / 8) * 64 + key, keys permuted by the unit pair so that
            // the eight units of a row fall into different banks
            h8 *pk = reinterpret_cast<h8 *>(base);
            pk[2 * cu * 64 + (key ^ (cu & 7))] = bytes_to_h8(kreg[u][0], kreg[u][1]);
            pk[(2 * cu + 1) * 64 + (key ^ (cu & 7))] = bytes_to_h8(kreg[u][2], kreg[u][3]);
            // V: unit (2 T + g % 2) * DPAD + d holds quads g and g + 2 of 16-key tile T
            const int d = id / 4, g = id % 4;
            uint2 *pv = reinterpret_cast<uint2 *>(base + KBYTES);
#pragma unroll
            for (int t = 0; t < 4; t += 2) {
                union {
                    h8 v;
                    uint2 w[2];
                } x;
                x.v = bytes_to_h8(vreg[u][t], vreg[u][t + 1]);
                pv[((2 * t + (g & 1)) * DPAD + d) * 2 + (g >> 1)] = x.w[0];
                pv[((2 * (t + 1) + (g & 1)) * DPAD + d) * 2 + (g >> 1)] = x.w[1];
            }
        }
        const float vtop = wave_max_nonneg(vsr);
        float f = 1.0f;
        if (vtop > ref) {
            const float ref2 = pow2_above(vtop);
            f = ref / ref2;
            ref = ref2;
        }
        if (wave == 0) {
            float *sc = reinterpret_cast<float *>(base + 2 * KBYTES);
            sc[lane] = ksr;
            sc[64 + lane] = ref > 0.0f ? vsr * (WR::PSCALE / ref) : 0.0f;
        }
        return f;
    };

    f16v o[DT32];
#pragma unroll
    for (int d = 0; d < DT32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
    float m = neg_inf(), l = 0.0f;
    if (j.blk0 < j.blk1) {
        fetch(j.blk0);
        (void)stage(0);
    }
    int cur_page = page;
    __syncthreads();
    for (int blk = j.blk0; blk < j.blk1; ++blk) {
        const int buf = (blk - j.blk0) & 1;
        const uint8_t *base = smem + buf * BUF;
        const int this_page = cur_page;
        if (blk + 1 < j.blk1) fetch(blk + 1);
        const int k0 = blk * CACHE_BLOCK;
        if (wave_live && this_page >= 0 && k0 < lim_max) {
            const h8 *pk = reinterpret_cast<const h8 *>(base), *pv = reinterpret_cast<const h8 *>(base + KBYTES);
            const f4 *sc = reinterpret_cast<const f4 *>(base + 2 * KBYTES);
            f16v s[2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const h8 kf = pk[(2 * k + hf) * 64 + ((32 * t + i) ^ (k & 7))];
#pragma unroll
                    for (int z = 0; z < NS; ++z) s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, q[z][k], s[t], 0, 0, 0);
                }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const f4 kq = sc[8 * t + 2 * x + hf];
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[t][4 * x + r] *= kq[r];
                }
            if (k0 + CACHE_BLOCK > lim_min) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int key = k0 + 32 * t + 8 * (r / 4) + 4 * hf + r % 4;
                        s[t][r] = key < lim ? s[t][r] : neg_inf();
                    }
            }
            float top = neg_inf();
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
            top = max_across32(top);
            const bool raise = top > neg_inf() && !((top - m) * c <= WR::SLACK);
            if (__any(raise)) {
                const float m2 = raise ? fmaxf(m, top) : m;
                const float f = raise ? __builtin_amdgcn_exp2f((m - m2) * c) : 1.0f;
                m = m2;
                l *= f;
#pragma unroll
                for (int d = 0; d < DT32; ++d) o[d] *= f;
            }
            const float mc = m > neg_inf() ? m * c : 0.0f;
            float w[4][8], least = WR::LEAST; // weights by 16-key tile
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const f4 vq = sc[16 + 4 * t + 2 * x + hf];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t / 2][8 * (t % 2) + 4 * x + r], c, -mc));
                        l += p;
                        w[t][4 * x + r] = p * vq[r];
                        least = fminf(least, w[t][4 * x + r]);
                    }
                }
            if (__any(least < WR::LEAST)) {
                // weights below LEAST: rounds of their own, each brought up by STEP
                float up = WR::STEP, down = 1.0f / WR::STEP;
                for (bool more = true; more; up *= WR::STEP, down *= 1.0f / WR::STEP) {
                    h8 p[4][NS];
                    more = false;
#pragma unroll
                    for (int t = 0; t < 4; ++t) more = round_weights<NS>(w[t], up, p[t]) || more;
                    more = __any(more);
#pragma unroll
                    for (int d = 0; d < DT32; ++d) {
                        f16v x;
#pragma unroll
                        for (int r = 0; r < 16; ++r) x[r] = 0.0f;
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const h8 vv = pv[(2 * t + hf) * DPAD + 32 * d + i];
#pragma unroll
                            for (int z = 0; z < NS; ++z) x = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, p[t][z], x, 0, 0, 0);
                        }
                        o[d] += x * down;
                        __builtin_amdgcn_sched_barrier(0); // one tile's registers at a time
                    }
                }
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[t][e] = w[t][e] >= WR::LEAST ? w[t][e] : 0.0f;
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                h8 p[NS];
                split_weights<NS>(w[t], p);
#pragma unroll
                for (int d = 0; d < DT32; ++d) {
                    const h8 vv = pv[(2 * t + hf) * DPAD + 32 * d + i];
#pragma unroll
                    for (int z = 0; z < NS; ++z) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, p[z], o[d], 0, 0, 0);
                }
            }
        }
        if (blk + 1 < j.blk1) {
            const float f = stage(buf ^ 1);
            if (f != 1.0f) {
#pragma unroll
                for (int d = 0; d < DT32; ++d) o[d] *= f;
            }
            cur_page = page;
        }
        __syncthreads();
    }
    l += __shfl_xor(l, 32);
    if (rho < j.rows) {
        const int rr = j.row0 + rho;
        const int64_t at = part_index(a, j.part, j.tok0 + rr / G, j.kvh * G + rr % G);
        f4 *po = reinterpret_cast<f4 *>(a.ws) + at * (Dp / 4);
        const float f = ref / WR::PSCALE;
#pragma unroll
        for (int d = 0; d < DT32; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int col = 32 * d + 8 * x + 4 * hf;
                if (col < Dp) po[col / 4] = f4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]} * f;
            }
        if (hf == 0)
            reinterpret_cast<float2 *>(a.ws + pl.ml_off)[at] = make_float2(m > neg_inf() ? m * c : neg_inf(), l);
    }
}

// Joins the parts of every row: a wave per (token, head), lanes the columns.
template <int DT>
__global__ __launch_bounds__(256) void k_attn_join(const AttnArgs a, const AttnPlan pl, int64_t rows)
{
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + wave_id();
    if (r >= rows) return;
    const int head = static_cast<int>(r % a.heads);
    const int64_t bi = r / a.heads;
    const int b = static_cast<int>(bi / a.max_q), i = static_cast<int>(bi % a.max_q), lane = lane_id();
    int first = b * a.max_q, n = a.max_q;
    if (a.q_start) {
        first = a.q_start[b];
        n = min(max(a.q_start[b + 1] - first, 0), a.max_q);
        if (first < 0 || first > a.tokens - n) return;
    }
    if (i >= n) return;
    const int64_t tok = static_cast<int64_t>(first) + i;
    const int parts = pl.splits_prefix + pl.splits_own, Dp = a.c.Dp;
    const float2 *pml = reinterpret_cast<const float2 *>(a.ws + pl.ml_off);
    float top = neg_inf();
    for (int p = 0; p < parts; ++p) top = fmaxf(top, pml[part_index(a, p, tok, head)].x);
    float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (top > neg_inf())
        for (int p = 0; p < parts; ++p) {
            const int64_t at = part_index(a, p, tok, head);
            const float2 x = pml[at];
            if (!(x.x > neg_inf())) continue;
            const float f = __builtin_amdgcn_exp2f(x.x - top);
            l += x.y * f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (lane + 64 * k < a.c.D) o[k] += a.ws[at * Dp + lane + 64 * k] * f;
        }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int d = lane + 64 * k;
        if (d >= a.c.D) continue;
        const int64_t at = tok * a.ldo_t + head * a.ldo_h + d;
        if constexpr (DT == DT_F32) static_cast<float *>(a.O)[at] = o[k] * inv;
        else static_cast<uint16_t *>(a.O)[at] = float_to_bf16_rne(o[k] * inv);
    }
    if (a.lse && lane == 0)
        a.lse[tok * a.heads + head] = l > 0.0f ? (top + log2f(l)) * ATTN_LN2 : neg_inf();
}

// ---- host -------------------------------------------------------------------
namespace {

int64_t div_up(int64_t x, int64_t y) { return (x + y - 1) / y; }

// Rows a workgroup takes: 16 with k_attn_stream, 128 with k_attn_tile.
int tile_rows(int64_t rows) { return rows <= 16 ? 16 : TILE_ROWS_ATTN; }

// Workgroups a launch should have: two for each of the 256 CUs.
constexpr int64_t kAttnWgs = 512;

AttnPlan attn_plan(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t seqs, int64_t max_q,
                   int64_t max_own, int64_t prefix)
{
    AttnPlan p;
    const int64_t G = heads / kv_heads, nbp = div_up(prefix, CACHE_BLOCK), nbo = div_up(max_own, CACHE_BLOCK);
    auto split = [](int64_t wgs, int64_t blocks, int64_t least, int *chunk, int *splits) {
        if (blocks == 0) {
            *chunk = *splits = 0;
            return;
        }
        int64_t s = kAttnWgs / wgs;
        const int64_t most = div_up(blocks, least);
        s = s < 1 ? 1 : (s > most ? most : s);
        *chunk = static_cast<int>(div_up(blocks, s));
        *splits = static_cast<int>(div_up(blocks, *chunk));
    };
    p.rows_prefix = tile_rows(tokens * G);
    p.rows_own = tile_rows(max_q * G);
    p.tiles_own = static_cast<int>(div_up(max_q * G, p.rows_own));
    const int64_t tp = div_up(tokens * G, p.rows_prefix);
    split(tp * kv_heads, nbp, 4, &p.chunk_prefix, &p.splits_prefix);
    split(seqs * p.tiles_own * kv_heads, nbo, 4, &p.chunk_own, &p.splits_own);
    p.wgs_prefix = static_cast<int>(tp * kv_heads * p.splits_prefix);
    p.wgs_own = static_cast<int>(seqs * p.tiles_own * kv_heads * p.splits_own);
    p.wg0 = 0;
    const int64_t parts = p.splits_prefix + p.splits_own, dp = div_up(head_dim, 16) * 16;
    p.ml_off = parts * tokens * heads * dp;
    return p;
}

template <int DT>
hipError_t launch_part(const AttnArgs &a, AttnPlan pl, int rows, int wg0, int wgs, hipStream_t st)
{
    if (wgs == 0) return hipSuccess;
    pl.wg0 = wg0;
    const int dc = a.c.Dp <= 64 ? 1 : a.c.Dp <= 128 ? 2 : 4;
    const dim3 grid(static_cast<unsigned>(wgs)), block(256);
#define BL_STREAM(DC) hipLaunchKernelGGL((k_attn_stream<DT, DC>), grid, block, 0, st, a, pl)
#define BL_TILE(DC) hipLaunchKernelGGL((k_attn_tile<DT, DC>), grid, block, 0, st, a, pl)
    if (rows == 16) {
        if (dc == 1) BL_STREAM(1);
        else if (dc == 2) BL_STREAM(2);
        else BL_STREAM(4);
    } else {
        if (dc == 1) BL_TILE(1);
        else if (dc == 2) BL_TILE(2);
        else BL_TILE(4);
    }
#undef BL_STREAM
#undef BL_TILE
    return hipGetLastError();
}

template <int DT>
hipError_t launch_attn(const AttnArgs &a, const AttnPlan &pl, hipStream_t st)
{
    hipError_t e = launch_part<DT>(a, pl, pl.rows_prefix, 0, pl.wgs_prefix, st);
    if (e == hipSuccess) e = launch_part<DT>(a, pl, pl.rows_own, pl.wgs_prefix, pl.wgs_own, st);
    if (e != hipSuccess) return e;
    const int64_t rows = static_cast<int64_t>(a.seqs) * a.max_q * a.heads;
    hipLaunchKernelGGL(k_attn_join<DT>, dim3(static_cast<unsigned>(div_up(rows, 4))), dim3(256), 0, st, a, pl, rows);
    return hipGetLastError();
}

} // namespace

int64_t attn_workspace_bytes(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t seqs,
                             int64_t max_q, int64_t max_own, int64_t prefix)
{
    const AttnPlan p = attn_plan(tokens, heads, kv_heads, head_dim, seqs, max_q, max_own, prefix);
    return (p.ml_off + 2 * (p.splits_prefix + p.splits_own) * tokens * heads) * 4;
}

hipError_t launch_attention(const AttnArgs &a, hipStream_t stream)
{
    const AttnPlan p = attn_plan(a.tokens, a.heads, a.c.heads, a.c.D, a.seqs, a.max_q, a.max_own, a.prefix);
    return a.dtype == DT_F32 ? launch_attn<DT_F32>(a, p, stream) : launch_attn<DT_BF16>(a, p, stream);
}

} // namespace bl
