// attn_masked.hip -- attention over the int8 cache for rows that do not see a
// sequence's first keys: a sliding window with a few first tokens, a tree of drafts.
// Few rows take k_attn_stream (attn_core.h), many k_attn_rows.
#include "attn_core.h"

#include <utility>

namespace bl {

// ---------------------------------------------------------------------------
// Many rows: k_attn_rows.  A workgroup of four waves takes 128 RT rows (a wave RT
// tiles of 32) and a chunk of keys, in halves of 32 keys of a block.  S^T = K Q^T in
// 32 x 32 tiles leaves a lane (row = lane % 32, hf = lane / 32) keys 8 x + 4 hf + {0..3},
// the operand order of O^T += V^T P^T: weights never leave their lane.
//
// A step is one half of a block.  Its products belong to the halves around it (values
// of the half before, scores of the half after), its vector instructions are the
// weights of its own, so that both have no need of each other and go out in turns: two
// weights behind every operand.  One barrier a step; K lies in LDS by halves, V by
// blocks, two of each.
//
// The first product is bf16 for bf16 queries, which takes the queries as they are (below a
// scale of SMALL_SCALE times 2^-64, as their products with the keys could pass binary32's range
// where their scores do not) and the bytes exactly, and binary16 in two terms for fp32 queries
// (brought into its range by a power of two per row).  Weights are w = 2^(x - M) V_scale, M a reference in base 2
// that a row gets with its first keys (the first 32 of which it sees some) and keeps until
// its weights outgrow it, so that few steps touch its sums:
//  - fp32 queries: three bf16 terms, 24 bits, in binary32's range; M is the largest
//    x of those keys.
//  - bf16 queries: one binary16 term, 11 bits.  M brings the largest weight so far to
//    2^FIRST_TOP: those that are 2^16 times smaller lose bits, all below 2^-27 of it are lost.
//    M so follows p V_scale, and is far below the scores where values are small or zero: down to
//    LEAST_BELOW of them, where a value's share of the row is at the end of binary32's range.
//    The sum of p is then held in units that are 2^LOW_BITS larger (low).
// A half's weights have outgrown M when their sum (times the block's largest V_scale for
// binary16) passes a bound that no weight of it can pass alone.  They are not in the sums
// yet: the row gets a new M, its sums are brought to it and the half's weights are formed
// again (raise).  So the time depends little on the scores: 4 x 200 tokens of 64 heads on up
// to 9000 keys at 1.6, 3, 6 and 13 nats of standard deviation: 192, 199, 225, 256 us.
//
// Bound: vector instructions.  A wave's block of 64 keys x 32 rows takes some 400 issue
// slots of four cycles (112 and 32 exponentials at a quarter of the rate for the weights, 90
// to convert and stage its share of K and V, the rest addresses, LDS and scalar work) beside
// 32 products of 33: 3200 of the 4370 cycles measured for two waves, in which matrix cores are
// busy for 48 %.  2 x 4096 tokens x 64 heads of 128 in a window of 1024: 385 us (448 in the first
// launches after an idle time), 55 % of a large matrix product's rate; counters over the whole
// kernel have matrix cores 35 % busy, since a job's start (queries, first blocks) takes 15 %.
// ---------------------------------------------------------------------------
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
constexpr float SMALL_SCALE = 0x1p-60f;
constexpr int SMALL_SCALE_E2 = -64;
// log2 of what a row's reference makes of the largest weight (one binary16 term); bounds of a half's sum of weights of
// one lane: with V_scale (binary16 ends at 2^16), and without
constexpr float FIRST_TOP = 2.0f, ROWS_WEIGHT_MAX = 0x1p15f, ROWS_SUM_MAX = 0x1p60f;
// log2 of the largest p of a row that needs the sum's larger units, of those units, and of the largest p there may be when
// a reference is set (16 of them and a few bits' growth stay in binary32)
constexpr float LOW_FROM = 40.0f, LOW_BITS = 70.0f, LEAST_BELOW = 110.0f, LOW_UNIT = 0x1p-70f;

// Eight int8 (two words) to bf16, exactly, by way of binary32.
__device__ __forceinline__ u4 bytes_to_b8(uint32_t a, uint32_t b)
{
    u4 r;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const uint32_t w = h < 2 ? a : b;
        const float lo = static_cast<float>(static_cast<int8_t>(w >> (16 * (h % 2))));
        const float hi = static_cast<float>(static_cast<int8_t>(w >> (16 * (h % 2) + 8)));
        r[h] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    }
    return r;
}

// Two weights as operands of the second product: one binary16 term, or three bf16 ones,
// the last rounded to nearest, those before cut (what is cut off is exact in binary32).
template <int DT, int NT>
__device__ __forceinline__ void weight_terms(float w0, float w1, uint32_t (&p)[NT])
{
    if constexpr (DT == DT_BF16) {
        const h2 r = {static_cast<_Float16>(w0), static_cast<_Float16>(w1)};
        p[0] = __builtin_bit_cast(uint32_t, r);
    } else {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int z = 0; z < NT; ++z) {
            if (z == NT - 1) {
                const b2 r = {static_cast<__bf16>(w0), static_cast<__bf16>(w1)};
                p[z] = __builtin_bit_cast(uint32_t, r);
            } else {
                p[z] = __builtin_amdgcn_perm(__float_as_uint(w1), __float_as_uint(w0), 0x07060302u);
                w0 -= __uint_as_float(__float_as_uint(w0) & 0xffff0000u);
                w1 -= __uint_as_float(__float_as_uint(w1) & 0xffff0000u);
            }
        }
    }
}

// Operand of the first product: bytes of K, and the queries.
template <int DT>
__device__ __forceinline__ u4 key_operand(uint32_t a, uint32_t b)
{
    if constexpr (DT == DT_BF16) return bytes_to_b8(a, b);
    else return __builtin_bit_cast(u4, bytes_to_h8(a, b));
}
template <int DT>
__device__ __forceinline__ f16v score_product(u4 k, u4 q, f16v s)
{
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, k), __builtin_bit_cast(b8, q), s, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, k), __builtin_bit_cast(h8, q), s, 0, 0, 0);
}

// The second product's: bytes of V, and the weights.
template <int DT>
__device__ __forceinline__ u4 value_operand(uint32_t a, uint32_t b)
{
    if constexpr (DT == DT_BF16) return __builtin_bit_cast(u4, bytes_to_h8(a, b));
    else return bytes_to_b8(a, b);
}
template <int DT>
__device__ __forceinline__ f16v value_product(u4 v, u4 p, f16v o)
{
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, v), __builtin_bit_cast(h8, p), o, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, v), __builtin_bit_cast(b8, p), o, 0, 0, 0);
}

// A value that the matrix instructions alone use, in accumulation registers; one that
// vector instructions use, in theirs (and formed here, not where it is used).
template <class T>
__device__ __forceinline__ void to_matrix(T &v)
{
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+a"(v));
#endif
}
template <class T>
__device__ __forceinline__ void to_vector(T &v)
{
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(v));
#endif
}

// x *= f for an x in an accumulation register, by way of one other (the compiler would find room for all of them).  Waits
// for a product that forms x, and before one that takes it.
__device__ __forceinline__ void scale_matrix(float &x, float f)
{
#if defined(__HIP_DEVICE_COMPILE__)
    float y;
    asm volatile("s_nop 15\n\ts_nop 7\n\tv_accvgpr_read_b32 %1, %0\n\ts_nop 1\n\tv_mul_f32 %1, %1, %2\n\ts_nop 1\n\t"
                 "v_accvgpr_write_b32 %0, %1\n\ts_nop 3" : "+a"(x), "=&v"(y) : "v"(f));
#endif
}

// f(0), f(1), .. f(N - 1) as constants.
template <class F, int... I>
__device__ __forceinline__ void in_turn(const F &f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>()), ...);
}
template <int N, class F>
__device__ __forceinline__ void in_turn(const F &f)
{
    in_turn(f, std::make_integer_sequence<int, N>());
}

// Waves of a SIMD: two where their registers (256 a lane) hold sums, scores, queries and weights.
constexpr int rows_waves(int dt, int dc, int rt) { return dt == DT_BF16 && dc * rt <= 2 ? 2 : 1; }

template <int DT, int DC, int RT, int MASK>
__global__ __launch_bounds__(256, rows_waves(DT, DC, RT)) void k_attn_rows(const AttnArgs a, const AttnPlan pl)
{
    constexpr int NS = DT == DT_F32 ? 2 : 1, NT = DT == DT_F32 ? 3 : 1; // terms of queries and of weights
    constexpr int DPAD = 64 * DC, KSTEPS = DPAD / 16, DT32 = DPAD / 32;
    // 16-byte units of half a block of K, and of a block of V, of a thread
    constexpr int KU = DC < 2 ? 1 : DC / 2, VU = DC;
    // K in LDS: 16-byte unit of 8 columns c8 of a key at ((c8 / 2 + KSTEPS (c8 % 2)) KROW + key), as in k_attn_tile
    constexpr int KROW = 33, KBYTES = 2 * KSTEPS * KROW * 16, VBYTES = 64 * DPAD * 2;
    // two blocks of K (four halves), of V and of scales
    __shared__ __attribute__((aligned(16))) uint8_t smem[4 * KBYTES + 2 * VBYTES + 2 * 512 + 16];
    // bytes of half a block of keys, a block of values and one of scales (K_scales, then V_scales) in it; last, the
    // largest V_scale of two blocks
    auto k_at = [](int n, int half) { return (2 * (n & 1) + half) * KBYTES; };
    auto v_at = [](int n) { return 4 * KBYTES + (n & 1) * VBYTES; };
    auto scales_at = [](int n) { return 4 * KBYTES + 2 * VBYTES + (n & 1) * 512; };
    auto top_at = [](int n) { return 4 * KBYTES + 2 * VBYTES + 2 * 512 + (n & 1) * 4; };
    auto lds4 = [&](uint32_t at) -> u4 & { return *reinterpret_cast<u4 *>(smem + at); };
    auto lds2 = [&](uint32_t at) -> uint2 & { return *reinterpret_cast<uint2 *>(smem + at); };
    auto lds1 = [&](uint32_t at) -> float & { return *reinterpret_cast<float *>(smem + at); };
    const int tid = threadIdx.x, G = a.heads / a.c.heads, Dp = a.c.Dp;
    AttnJob j;
    if (!attn_job<MASK>(a, pl, 128 * RT, blockIdx.x + pl.wg0, j)) return;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 31, hf = lane >> 5;
    const int nblk = j.blk1 - j.blk0;

    // this thread's bytes of a half of K and of a block of V; columns past Dp read the row's start (the queries
    // hold zeros there), V's rows past Dp its first rows (their sums are not stored)
    const bool k_mine = DC >= 2 || tid < 128; // (half a block of K is 128 units of 64 columns)
    u4 kreg[2][KU] = {};
    uint2 vreg[2][VU] = {}; // (a block's row of V has 8 bytes of either half in 16)
    uint32_t koff[KU], voff[VU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
        const int id = tid + 256 * u, col = 16 * (id % (4 * DC));
        koff[u] = (k_mine ? id / (4 * DC) : 0) * Dp + (col < Dp ? col : 0);
    }
#pragma unroll
    for (int u = 0; u < VU; ++u) {
        const int id = tid + 256 * u;
        voff[u] = (id / 4 < Dp ? id : id % 4) * 16;
    }
    // this lane's place in an operand of keys, of values and among the scales, this thread's in what it stages of keys
    // and of values; all else is a constant apart (values kept here, so that nothing they come from has to be)
    uint32_t kl = (KSTEPS * hf * KROW + i) * 16, vl = (hf * DPAD + i) * 16, sl = 16 * hf,
             kst = (tid % (4 * DC) * KROW + tid / (4 * DC)) * 16, vst = ((tid & 1) * DPAD + tid / 4) * 16 + (tid & 2) * 4;
    to_vector(kl);
    to_vector(vl);
    to_vector(sl);
    to_vector(kst);
    to_vector(vst);
    float ksr = 0.0f, vsr = 0.0f;
    auto fetch_k = [&](int half, int u, uint32_t unit) {
        kreg[half][u] = load_at<u4>(block_bytes(a.c.K, unit, Dp) + 32 * half * Dp, koff[u]);
    };
    auto fetch_v = [&](int half, int u, uint32_t unit) {
        vreg[half][u] = load_at<uint2>(block_bytes(a.c.V, unit, Dp) + 8 * half, voff[u]);
    };
    auto fetch_scales = [&](uint32_t unit) {
        ksr = load_at<float>(block_scales(a.c.Ks, unit), 4 * lane);
        vsr = load_at<float>(block_scales(a.c.Vs, unit), 4 * lane);
    };
    BlockTable table;
    uint32_t unit1 = 0, unit2 = 0, unit3 = 0; // places of the next three blocks (of some block, past the last)
    bool there0 = false, there1 = false, there2 = false, there3 = false;
    // the place of block n, which follows the ones before
    auto look_up = [&](int n, uint32_t &unit, bool &there) {
        there = false;
        if (n >= nblk) return;
        if (n % 64 == 0) table.load<MASK>(a, j, j.blk0 + n, 1);
        unit = table.at(n % 64);
        there = table.there(n % 64);
    };
    // block 0, and the first half of block 1's keys (in flight while the queries are read)
    u4 kfirst[KU] = {};
    if (nblk > 0) {
        uint32_t unit0 = 0;
        look_up(0, unit0, there0);
        unit1 = unit0;
        look_up(1, unit1, there1);
        unit2 = unit1;
        look_up(2, unit2, there2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int u = 0; u < KU; ++u) fetch_k(h, u, unit0);
#pragma unroll
            for (int u = 0; u < VU; ++u) fetch_v(h, u, unit0);
        }
        fetch_scales(unit0);
#pragma unroll
        for (int u = 0; u < KU; ++u) kfirst[u] = load_at<u4>(block_bytes(a.c.K, unit1, Dp), koff[u]);
    }

    // Queries: operands, and a row's factor from scores to base 2 (fp32: of its own power of two).
    u4 q[RT][KSTEPS][NS];
    float c[RT];
    RowSight<MASK> sight[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int rho = 32 * (RT * wave + t) + i, rr = j.row0 + (rho < j.rows ? rho : 0);
        const int64_t off = (j.tok0 + static_cast<int64_t>(rr / G)) * a.ldq_t + (j.kvh * G + rr % G) * a.ldq_h;
        sight[t].set(a, j, G, rho);
        float v[KSTEPS][8];
        load_queries<DT>(a, off, [&](int n) { return 16 * n + 8 * hf; }, v);
        if constexpr (DT == DT_BF16) {
            // (powers of two, so that the products are exact bf16 numbers)
            const int e2 = fabsf(a.scale) < SMALL_SCALE ? SMALL_SCALE_E2 : 0;
            const float by = a.scale == 0.0f ? 0.0f : __builtin_copysignf(e2 ? __builtin_ldexpf(1.0f, SMALL_SCALE_E2) : 1.0f, a.scale);
            c[t] = row_factor(a.scale, e2);
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    q[t][k][0][e] = __builtin_amdgcn_perm(__float_as_uint(v[k][2 * e + 1] * by), __float_as_uint(v[k][2 * e] * by),
                                                          0x07060302u);
        } else {
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) top = fmaxf(top, max_abs8(v[k]));
            top = max_across32(top);
            const int e2 = row_exponent(top < __builtin_inff() ? top : 0.0f);
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k) {
                h8 terms[NS];
                query_terms<NS>(v[k], e2, a.scale, terms);
#pragma unroll
                for (int z = 0; z < NS; ++z) q[t][k][z] = __builtin_bit_cast(u4, terms[z]);
            }
            c[t] = row_factor(a.scale, e2);
        }
    }

    // (the queries are operands only: in accumulation registers they leave the others to the vector instructions)
    if constexpr (rows_waves(DT, DC, RT) == 1) {
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
                for (int z = 0; z < NS; ++z) to_matrix(q[t][k][z]);
    }
    auto stage_k = [&](const u4 &from, int u, int part, int to) { // (a second unit: 256 / (4 DC) keys on)
        if (k_mine)
            lds4(kst + to + (KSTEPS * part * KROW + u * (64 / DC)) * 16) = key_operand<DT>(from[2 * part], from[2 * part + 1]);
    };
    // V: unit (2 T + g % 2) * DPAD + d holds quads g and g + 2 of 16-key tile T; a half is two tiles, the next unit of a
    // thread 64 rows on.
    auto stage_v = [&](int half, int u, int to) {
        const u4 x = value_operand<DT>(vreg[half][u].x, vreg[half][u].y);
        lds2(vst + to + (4 * half * DPAD + 64 * u) * 16) = make_uint2(x[0], x[1]);
        lds2(vst + to + ((4 * half + 2) * DPAD + 64 * u) * 16) = make_uint2(x[2], x[3]);
    };
    // (a hidden score is -inf: never times 0.  A V_scale that is not finite counts as the largest number of its sign:
    // its key's weight is 0 where it is hidden)
    auto stage_scales = [&](int n) {
        if (wave == 0) {
            const float v = fmaxf(fminf(vsr, 3.402823466e38f), -3.402823466e38f);
            lds1(4 * lane + scales_at(n)) = fmaxf(DT == DT_BF16 ? ksr * c[0] : ksr, 1.17549435e-38f);
            lds1(4 * lane + scales_at(n) + 256) = v;
            if constexpr (DT == DT_BF16) {
                const float top = wave_max_nonneg(fabsf(v));
                if (lane == 0) lds1(top_at(n)) = top;
            }
        }
    };

    f16v o[RT][DT32], s[2][RT]; // sums; scores of the two halves
    u4 p[2][RT][2][NT];         // weights of the two halves, by 16-key tile
    float M[RT], l[RT];
    bool set[RT], settled = false; // a row's reference, all of the wave's
    bool low[RT];                  // (bf16) l counts in units of 2^LOW_BITS
    uint64_t vis[RT];              // keys of the block the row sees
    bool hidden = false;           // the rows do not all see all of it
    // K_scales (V_scales) of keys 8 x + 4 hf .. of a half
    auto key_scales = [&](int n, int half, int x) { return __builtin_bit_cast(f4, lds4(sl + scales_at(n) + 128 * half + 32 * x)); };
    auto value_scales = [&](int n, int half, int x) {
        return __builtin_bit_cast(f4, lds4(sl + scales_at(n) + 256 + 128 * half + 32 * x));
    };
    // Which keys of block n the rows see.  A block that every row of the tile sees whole is told from the tile's bounds
    // alone.
    const TileSight<MASK> tile(a, j, G);
    auto look = [&](int n, bool there) {
        const int list = j.at<MASK>(j.blk0 + n);
        const bool pre = list < j.nbp;
        const int k0 = (pre ? list : list - j.nbp) * CACHE_BLOCK;
        hidden = !there || !tile.whole(a, j, pre, k0);
#pragma unroll
        for (int t = 0; t < RT; ++t) vis[t] = hidden ? sight[t].of(a, j, there, pre, k0) : ~uint64_t(0);
    };
    // The scores of a half that a row does not see.
    auto hide = [&](int half, f16v &sc, int t) {
        const uint32_t mine = static_cast<uint32_t>(vis[t] >> (32 * half)) >> (4 * hf);
#pragma unroll
        for (int r = 0; r < 16; ++r) sc[r] = mine >> (8 * (r / 4) + r % 4) & 1 ? sc[r] : neg_inf();
    };
    // The largest exponent x of a half's scores, and of x + log2 V_scale, that of the weights.
    auto meet = [&](int n, int half, const f16v &sc, int t, float &top, float &most) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const f4 kq = key_scales(n, half, x), vq = value_scales(n, half, x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = sc[4 * x + e], z = (DT == DT_BF16 ? y : y * c[t]) * kq[e];
                top = fmaxf(top, z);
                if constexpr (DT == DT_BF16) most = fmaxf(most, z + __builtin_log2f(vq[e])); // (-inf for a zero scale)
            }
        }
    };
    // The reference that a half's scores ask for.  The largest weight comes to 2^FIRST_TOP where it is binary16; a row whose
    // values are zero so far takes the least there is, which the first weight outgrows.  bf16 terms need no more than that of p.
    auto reference = [&](int n, int half, const f16v &sc, int t, float &top) {
        float most = neg_inf();
        top = neg_inf();
        meet(n, half, sc, t, top, most);
        top = max_across32(top);
        if constexpr (DT != DT_BF16) return top;
        most = max_across32(most);
        return fmaxf(most - FIRST_TOP, top - LEAST_BELOW);
    };
    // Before a half's weights: scores a row does not see, and the reference of a row whose first keys these are (its
    // sums are still zero).
    auto prepare = [&](auto half_c, int n) {
        constexpr int H = decltype(half_c)::value;
        if (hidden) {
#pragma unroll
            for (int t = 0; t < RT; ++t) hide(H, s[H][t], t);
        }
        if (settled) return;
        bool unset = false;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float top;
            const float m = reference(n, H, s[H][t], t, top);
            const bool now = !set[t] && top > neg_inf();
            M[t] = now ? m : M[t];
            if constexpr (DT == DT_BF16) low[t] = now ? top > m + LOW_FROM : low[t];
            set[t] = set[t] || now;
            unset |= !set[t] && l[t] == l[t]; // (one with a NaN query never gets any)
        }
        settled = !__any(unset);
    };

    auto sum_unit = [&](int t) { return DT == DT_BF16 && low[t] ? LOW_UNIT : 1.0f; };

    // Sums stay in accumulation registers and scores in the others; without a word the compiler carries them to and fro
    // (64 moves a step).
    auto place = [&](int half) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            to_vector(s[half][t]);
            if constexpr (rows_waves(DT, DC, RT) == 1) {
#pragma unroll
                for (int d = 0; d < DT32; ++d) to_matrix(o[t][d]);
            }
        }
    };

    // One block: for each half its weights, beside the products of the halves around it.  What a block stages is read
    // after its barrier: keys from the second half of the next block to the first of the one after, values up to the
    // first half of the next.  A register is loaded again as soon as it is staged, a block ahead of its use.
    constexpr int OPS = 4 * DC, PAIRS = 8 * RT, AHEAD = rows_waves(DT, DC, RT) == 2 ? 2 : 3; // operands of either product; pairs of weights
    constexpr int PER = RT * (NT + NS), PRODUCTS = OPS * PER, PARTS = 3 * PAIRS, STAGE = 4 * KU + 2 * VU + 1;
    u4 rk[AHEAD], rv[AHEAD];
    f4 kq[2], vq[2];
    float vtop = 0.0f; // the largest V_scale of the block
    auto read_ops = [&](int n, int y) { // operand y % OPS of half y / OPS
        if (y >= 2 * OPS) return;
        const int half = y / OPS, x = y % OPS;
        rv[y % AHEAD] = lds4(vl + v_at(half == 0 ? n - 1 : n) + (2 * (x / DT32 + 2 * (1 - half)) * DPAD + 32 * (x % DT32)) * 16);
        rk[y % AHEAD] = lds4(kl + (half == 0 ? k_at(n, 1) : k_at(n + 1, 0)) + x * KROW * 16);
    };
    auto read_scales = [&](int n, int x) { // quad x % 4 of half x / 4
        if (x >= 8) return;
        kq[x % 2] = key_scales(n, x / 4, x % 4);
        vq[x % 2] = value_scales(n, x / 4, x % 4);
    };
    auto stage = [&](int n, int x) {
        if (x < 4 * KU) { // second half of the next block's keys, first of the one after
            const int half = x < 2 * KU ? 1 : 0, u = x / 2 % KU, part = x % 2;
            stage_k(kreg[half][u], u, part, half ? k_at(n + 1, 1) : k_at(n + 2, 0));
            if (part == 1) fetch_k(half, u, half ? unit2 : unit3);
        } else if (x < 4 * KU + 2 * VU) { // second half of this block's values, first of the next
            const int half = x < 4 * KU + VU ? 1 : 0, u = (x - 4 * KU) % VU;
            stage_v(half, u, half ? v_at(n) : v_at(n + 1));
            fetch_v(half, u, half ? unit1 : unit2);
        } else {
            stage_scales(n + 1);
            fetch_scales(unit2);
        }
    };
    // A half whose weights outgrew a row's reference.
    auto raise = [&](auto half_c, int n, float (&sum)[RT][2]) {
        constexpr int H = decltype(half_c)::value;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            float top;
            const float m = fmaxf(M[t], reference(n, H, s[H][t], t, top)), f = __builtin_amdgcn_exp2f(M[t] - m);
            if constexpr (DT == DT_BF16) {
                // (the sum so far and this half's largest p say which units the sum takes from here on)
                const float by = M[t] - m + (low[t] ? LOW_BITS : 0.0f);
                low[t] = fmaxf(top - m, by + __builtin_log2f(sum_across32(l[t]))) > LOW_FROM;
                l[t] *= __builtin_amdgcn_exp2f(by - (low[t] ? LOW_BITS : 0.0f));
            } else {
                l[t] *= f;
            }
            M[t] = m;
#pragma unroll
            for (int d = 0; d < DT32; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    if constexpr (rows_waves(DT, DC, RT) == 1) {
                        float x = o[t][d][r];
                        scale_matrix(x, f);
                        o[t][d][r] = x;
                    } else {
                        o[t][d][r] *= f;
                    }
                }
            sum[t][0] = sum[t][1] = 0.0f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const f4 ks = key_scales(n, H, x), vs = value_scales(n, H, x);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    float g[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const float v = DT == DT_BF16 ? s[H][t][4 * x + e + z] : s[H][t][4 * x + e + z] * c[t];
                        g[z] = __builtin_amdgcn_exp2f(__builtin_fmaf(v, ks[e + z], -m));
                        sum[t][z] += g[z];
                    }
                    uint32_t terms[NT];
                    weight_terms<DT, NT>(g[0] * vs[e], g[1] * vs[e + 1], terms);
#pragma unroll
                    for (int z = 0; z < NT; ++z) p[H][t][x / 2][z][2 * (x % 2) + e / 2] = terms[z];
                }
            }
        }
    };
    auto half_block = [&](auto half_c, int n) {
        constexpr int H = decltype(half_c)::value;
        if (__builtin_expect_with_probability(hidden || !settled, 0, 0.9)) prepare(half_c, n);
        float sum[RT][2];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            to_vector(s[H][t]);
            sum[t][0] = sum[t][1] = 0.0f;
        }
        // the weights of a pair of keys in three parts; pairs by quads of keys
        float g[2];
        auto weights = [&](int y) {
            const int x = y / 3, part = y % 3, quad = x / (2 * RT), t = x / 2 % RT, e = 2 * (x % 2), r0 = 4 * quad + e;
            if (x % (2 * RT) == 0 && part == 0) read_scales(n, 4 * H + quad + 1);
            if (part < 2) {
                const float v = DT == DT_BF16 ? s[H][t][r0 + part] : s[H][t][r0 + part] * c[t];
                g[part] = __builtin_amdgcn_exp2f(__builtin_fmaf(v, kq[quad % 2][e + part], -M[t]));
                sum[t][part] += g[part];
                pin(sum[t][part]);
            } else {
                uint32_t terms[NT];
                weight_terms<DT, NT>(g[0] * vq[quad % 2][e], g[1] * vq[quad % 2][e + 1], terms);
#pragma unroll
                for (int z = 0; z < NT; ++z) {
                    to_vector(terms[z]);
                    p[H][t][r0 / 8][z][r0 / 2 % 4] = terms[z];
                }
            }
        };
        // Product m: operand x of both products in turn, value products (32 columns of 16 keys of the half before) and
        // score products (16 columns of the half after) one after the other, so that neither waits for its own last one.
        static_assert(NS <= NT, "scores have no more products than values");
        auto product = [&](int m) {
            const int x = m / PER, y = m % PER, ring = (OPS * H + x) % AHEAD;
            constexpr int BOTH = RT * NS;
            const bool score = y < 2 * BOTH && y % 2 == 1; // (v s v s .., then the rest of v)
            const int k = y < 2 * BOTH ? y / 2 : y - BOTH, t = k % RT, z = k / RT;
            if (!score) {
                o[t][x % DT32] = value_product<DT>(rv[ring], p[1 - H][t][x / DT32][z], o[t][x % DT32]);
            } else if (x == 0 && z == 0) {
                f16v zero;
#pragma unroll
                for (int r = 0; r < 16; ++r) zero[r] = 0.0f;
                s[1 - H][t] = score_product<DT>(rk[ring], q[t][x][z], zero);
            } else {
                s[1 - H][t] = score_product<DT>(rk[ring], q[t][x][z], s[1 - H][t]);
            }
        };
        // A wave issues in order: a second product right behind the first waits for it, and the vector instructions
        // behind both wait too.  So every product has its share of them right after it.
        __builtin_amdgcn_sched_barrier(0);
        weights(0);
        in_turn<PRODUCTS>([&](auto m_c) __attribute__((always_inline)) {
            constexpr int m = decltype(m_c)::value, all = H * PRODUCTS + m;
            __builtin_amdgcn_sched_barrier(0);
            product(m);
            if constexpr (m % PER == PER - 1) read_ops(n, OPS * H + m / PER + AHEAD);
            in_turn<(m + 1) * PARTS / PRODUCTS - m * PARTS / PRODUCTS>([&](auto y) __attribute__((always_inline)) {
                constexpr int part = m * PARTS / PRODUCTS + decltype(y)::value + 1;
                if constexpr (part < PARTS) weights(part);
            });
            in_turn<(all + 1) * STAGE / (2 * PRODUCTS) - all * STAGE / (2 * PRODUCTS)>([&](auto y) __attribute__((always_inline)) {
                stage(n, all * STAGE / (2 * PRODUCTS) + decltype(y)::value);
            });
        });
        __builtin_amdgcn_sched_barrier(0);
        bool outgrown = false;
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const float all = sum[t][0] + sum[t][1];
            if constexpr (DT == DT_BF16) outgrown |= all * sum_unit(t) > ROWS_SUM_MAX || all * vtop > ROWS_WEIGHT_MAX;
            else outgrown |= all > ROWS_SUM_MAX;
        }
        if (__builtin_expect_with_probability(__any(outgrown), 0, 0.95)) raise(half_c, n, sum);
#pragma unroll
        for (int t = 0; t < RT; ++t) l[t] += (sum[t][0] + sum[t][1]) * sum_unit(t);
        place(1 - H);
    };

#pragma unroll
    for (int t = 0; t < RT; ++t) {
        M[t] = l[t] = 0.0f;
        set[t] = low[t] = false;
        vis[t] = 0;
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int d = 0; d < DT32; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[t][d][r] = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[h][t][r] = 0.0f;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int z = 0; z < NT; ++z) p[0][t][x][z] = p[1][t][x][z] = u4{0, 0, 0, 0};
    }
    if (nblk > 0) {
#pragma unroll
        for (int x = 0; x < 4 * KU; ++x) stage_k(kreg[x / 2 / KU][x / 2 % KU], x / 2 % KU, x % 2, k_at(0, x / 2 / KU));
#pragma unroll
        for (int x = 0; x < 2 * KU; ++x) stage_k(kfirst[x / 2], x / 2, x % 2, k_at(1, 0));
#pragma unroll
        for (int u = 0; u < VU; ++u) stage_v(0, u, v_at(0));
        stage_scales(0);
        // (the first half adds zero weights of a block that is not there: its V must be finite)
        for (int x = tid; x < VBYTES / 32; x += 256) lds4(v_at(1) + VBYTES / 2 + 16 * x) = u4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            fetch_k(1, u, unit1);
            fetch_k(0, u, unit2);
        }
#pragma unroll
        for (int u = 0; u < VU; ++u) fetch_v(0, u, unit1); // (vreg[1] holds block 0's second half)
        fetch_scales(unit1);
        __syncthreads();
        // scores of the first half
#pragma unroll
        for (int x0 = 0; x0 < OPS; x0 += 4) { // (four operands at once: their reads take longer than a product)
            u4 k[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) k[x] = lds4(kl + k_at(0, 0) + (x0 + x) * KROW * 16);
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int z = 0; z < NS; ++z) s[0][t] = score_product<DT>(k[x], q[t][x0 + x][z], s[0][t]);
        }
        __syncthreads();
    }
    place(0);
    for (int n = 0; n < nblk; ++n) {
#pragma unroll
        for (int x = 0; x < AHEAD; ++x) read_ops(n, x);
        read_scales(n, 0);
        if constexpr (DT == DT_BF16) vtop = lds1(top_at(n));
        look(n, there0);
        unit3 = unit2;
        look_up(n + 3, unit3, there3);
        half_block(std::integral_constant<int, 0>(), n);
        half_block(std::integral_constant<int, 1>(), n);
        there0 = there1;
        there1 = there2;
        there2 = there3;
        unit1 = unit2;
        unit2 = unit3;
        __syncthreads();
    }
    if (nblk > 0) { // values of the last half
#pragma unroll
        for (int x0 = 0; x0 < OPS; x0 += 4) {
            u4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
                v[y] = lds4(vl + v_at(nblk - 1) + (2 * ((x0 + y) / DT32 + 2) * DPAD + 32 * ((x0 + y) % DT32)) * 16);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int x = x0 + y;
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int z = 0; z < NT; ++z) o[t][x % DT32] = value_product<DT>(v[y], p[1][t][x / DT32][z], o[t][x % DT32]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const float sum = sum_across32(l[t]);
        const int rho = 32 * (RT * wave + t) + i;
        if (rho >= j.rows) continue;
        const int rr = j.row0 + rho, head = j.kvh * G + rr % G;
        const int64_t tok = j.tok0 + rr / G, at = part_index(a, j.part, tok, head);
        f4 *po = reinterpret_cast<f4 *>(a.ws) + at * (Dp / 4);
        // (sums of values in the sum's units, and those units' reference)
        const float f = sum_unit(t) * (!pl.direct ? 1.0f : inverse_of(sum)), m = M[t] + (low[t] ? LOW_BITS : 0.0f);
#pragma unroll
        for (int d = 0; d < DT32; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int col = 32 * d + 8 * x + 4 * hf;
                const f4 v = f4{o[t][d][4 * x], o[t][d][4 * x + 1], o[t][d][4 * x + 2], o[t][d][4 * x + 3]} * f;
                if (pl.direct) store_result<DT>(a, tok, head, col, v);
                else if (col < Dp) po[col / 4] = v;
            }
        if (hf == 0) {
            if (!pl.direct) reinterpret_cast<float2 *>(a.ws + pl.ml_off)[at] = make_float2(part_reference(m, sum, set[t]), sum);
            else if (a.lse) a.lse[tok * a.heads + head] = lse_of(m, sum);
        }
    }
}

namespace {

template <int DT, int MASK>
hipError_t launch_piece(const AttnArgs &a, AttnPlan pl, int rows, int waves, int64_t first, int64_t wgs, hipStream_t st)
{
    if (rows == 16) return launch_attn_stream<DT, MASK>(a, pl, waves, first, wgs, st);
    pl.wg0 = static_cast<int>(first);
    const int dc = a.c.Dp <= 64 ? 1 : a.c.Dp <= 128 ? 2 : 4;
    const dim3 grid(static_cast<unsigned>(wgs));
#define BL_ROWS(DC, RT) hipLaunchKernelGGL((k_attn_rows<DT, DC, RT, MASK>), grid, dim3(256), 0, st, a, pl)
    if (rows == 256) {
        if constexpr (DT == DT_F32) BL_ROWS(1, 2);
    } else if (dc == 1) {
        BL_ROWS(1, 1);
    } else if (dc == 2) {
        BL_ROWS(2, 1);
    } else {
        BL_ROWS(4, 1);
    }
#undef BL_ROWS
    return hipGetLastError();
}

template <int DT, int MASK>
hipError_t launch_masked(const AttnArgs &a, const AttnPlan &pl, hipStream_t st)
{
    return launch_attn_parts(pl, [&](int rows, int waves, int64_t first, int64_t wgs) {
        return launch_piece<DT, MASK>(a, pl, rows, waves, first, wgs, st);
    });
}

} // namespace

hipError_t launch_attn_masked(const AttnArgs &a, const AttnPlan &pl, int mask, hipStream_t st)
{
    if (a.dtype == DT_F32)
        return mask == ATTN_TREE ? launch_masked<DT_F32, ATTN_TREE>(a, pl, st) : launch_masked<DT_F32, ATTN_WINDOW>(a, pl, st);
    return mask == ATTN_TREE ? launch_masked<DT_BF16, ATTN_TREE>(a, pl, st) : launch_masked<DT_BF16, ATTN_WINDOW>(a, pl, st);
}

} // namespace bl
