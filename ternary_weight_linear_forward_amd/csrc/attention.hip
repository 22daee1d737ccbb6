// attention.hip -- calls of attention over the int8 cache: the cut into parts, the
// causal kernels (attn_core.h) and the join of the parts.
#include "attn_core.h"

namespace bl {

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
    if (lane % PER < LPR) store_result<DT>(a, tok, head, col, o * inverse_of(l));
    if (a.lse && lane % PER == 0) a.lse[tok * a.heads + head] = lse_of(top, l);
}

// ---- host -------------------------------------------------------------------
namespace {

template <int DT>
hipError_t launch_causal(const AttnArgs &a, AttnPlan pl, int rows, int waves, int64_t first, int64_t wgs, hipStream_t st)
{
    if (rows == 16) return launch_attn_stream<DT, ATTN_CAUSAL>(a, pl, waves, first, wgs, st);
    pl.wg0 = static_cast<int>(first);
    const dim3 grid(static_cast<unsigned>(wgs)), block(64 * waves);
#define BL_TILE(DC, NW) hipLaunchKernelGGL((k_attn_tile<DT, DC, NW>), grid, block, 0, st, a, pl)
    if (a.c.Dp <= 64) {
        BL_TILE(1, 4);
    } else if constexpr (DT == DT_BF16) {
        if (rows == 128) BL_TILE(2, 4);
        else BL_TILE(2, 8);
    }
#undef BL_TILE
    return hipGetLastError();
}

template <int DT>
hipError_t launch_join(const AttnArgs &a, const AttnPlan &pl, hipStream_t st)
{
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

// How a call sees its keys: a window over every key there may be is none.
int mask_of(int64_t prefix, int64_t max_own, int64_t window, bool tree)
{
    return tree ? ATTN_TREE : window > 0 && window < prefix + max_own ? ATTN_WINDOW : ATTN_CAUSAL;
}

template <int DT>
hipError_t launch_attn(const AttnArgs &a, hipStream_t st)
{
    const int mask = mask_of(a.prefix, a.max_own, a.window, a.tree != nullptr);
    const AttnPlan pl = attn_plan(a.tokens, a.heads, a.c.heads, a.c.D, a.seqs, a.max_q, a.max_own, a.prefix, DT == DT_F32,
                                  mask != ATTN_CAUSAL, mask == ATTN_WINDOW ? a.window : 0, a.sinks);
    const hipError_t e = mask != ATTN_CAUSAL
                             ? launch_attn_masked(a, pl, mask, st)
                             : launch_attn_parts(pl, [&](int rows, int waves, int64_t first, int64_t wgs) {
                                   return launch_causal<DT>(a, pl, rows, waves, first, wgs, st);
                               });
    return e != hipSuccess || pl.direct ? e : launch_join<DT>(a, pl, st);
}

} // namespace

// Room for either type's plan.
int64_t attn_workspace_bytes(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t seqs,
                             int64_t max_q, int64_t max_own, int64_t prefix, int64_t window, int64_t sinks, bool tree)
{
    const int mask = mask_of(prefix, max_own, window, tree);
    int64_t most = 0;
    for (const int dtype : {DT_F32, DT_BF16}) {
        const AttnPlan p = attn_plan(tokens, heads, kv_heads, head_dim, seqs, max_q, max_own, prefix, dtype == DT_F32,
                                     mask != ATTN_CAUSAL, mask == ATTN_WINDOW ? window : 0, sinks);
        const int64_t need = p.direct ? 0 : (p.ml_off + 2 * (p.splits_prefix + p.splits_own) * tokens * heads) * 4;
        most = need > most ? need : most;
    }
    return most;
}

hipError_t launch_attention(const AttnArgs &a, hipStream_t stream)
{
    return a.dtype == DT_F32 ? launch_attn<DT_F32>(a, stream) : launch_attn<DT_BF16>(a, stream);
}

} // namespace bl
