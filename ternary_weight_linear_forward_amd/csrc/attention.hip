// attention.hip -- attention of a batch of sequences that share a prefix, over
// the int8 cache.  o = softmax(scale q k^T) v over the prefix's keys and the
// sequence's own, by one pass with a running maximum m and sum l:
//   m' = max(m, s),  l' = l e^(m - m') + e^(s - m'),  o' = o e^(m - m') + e^(s - m') v.
#include "cache_core.h"
#include "common.h"
#include "launch.h"

namespace bl {

constexpr float ATTN_LOG2E = 1.4426950408889634f, ATTN_LN2 = 0.6931471805599453f;

// Own keys query i of a sequence sees: own_len - n + i + 1, within [0, own_len].
__device__ __forceinline__ int attn_own_limit(int own_len, int n, int i)
{
    const int v = own_len - n + i + 1;
    return v < 0 ? 0 : (v > own_len ? own_len : v);
}

// One wave per (query, head).  A lane scores one key of 64 at a time, then the
// wave adds the 64 weighted values, a lane holding columns d = lane + 64 j.
template <int DT>
__global__ __launch_bounds__(64) void k_attn_rows(const AttnArgs a)
{
    __shared__ float q[256];
    const int b = blockIdx.x / a.max_q, i = blockIdx.x % a.max_q, head = blockIdx.y, lane = lane_id();
    int first = b * a.max_q, n = a.max_q;
    if (a.q_start) {
        first = a.q_start[b];
        n = min(max(a.q_start[b + 1] - first, 0), a.max_q);
    }
    const int64_t tok = static_cast<int64_t>(first) + i;
    if (i >= n || tok < 0 || tok >= a.tokens) return;
    const int kvh = head / (a.heads / a.c.heads), D = a.c.D;
    for (int d = lane; d < 256; d += 64)
        q[d] = d < D ? load_x<DT>(a.Q, tok * a.ldq_t + head * a.ldq_h + d) * (a.scale * ATTN_LOG2E) : 0.0f;
    __syncthreads();
    const int own = attn_own_limit(min(max(a.own_len[b], 0), a.max_own), n, i);
    float m = -__builtin_inff(), l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int part = 0; part < 2; ++part) {
        const int keys = part == 0 ? a.prefix : own;
        const int32_t *pages = part == 0 ? a.prefix_pages : a.own_pages + b * a.ld_pages;
        for (int k0 = 0; k0 < keys; k0 += CACHE_BLOCK) {
            const int page = pages[k0 / a.c.page_tokens];
            if (page < 0 || page >= a.c.pages) continue;
            const int64_t row = cache_row0(a.c, page, kvh) + k0 % a.c.page_tokens;
            const bool live = k0 + lane < keys;
            float s = 0.0f;
            const int8_t *kr = a.c.K + (row + lane) * a.c.Dp;
            for (int d = 0; d < D; ++d) s += q[d] * static_cast<float>(kr[d]);
            s = live ? s * a.c.Ks[row + lane] : -__builtin_inff();
            float top = s;
            for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
            const float m2 = fmaxf(m, top);
            const float p = live ? exp2f(s - m2) : 0.0f, f = exp2f(m - m2);
            float sum = p;
            for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x);
            l = l * f + sum;
            m = m2;
            const float pv = live ? p * a.c.Vs[row + lane] : 0.0f;
            for (int j = 0; j < 4; ++j) o[j] *= f;
            for (int t = 0; t < CACHE_BLOCK; ++t) {
                const float w = __shfl(pv, t);
                for (int j = 0; j < 4; ++j) {
                    const int d = lane + 64 * j;
                    if (d < D) o[j] += w * static_cast<float>(a.c.V[row * a.c.Dp + d * CACHE_BLOCK + cache_v_byte(t)]);
                }
            }
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    for (int j = 0; j < 4; ++j) {
        const int d = lane + 64 * j;
        if (d >= D) continue;
        const int64_t at = tok * a.ldo_t + head * a.ldo_h + d;
        if constexpr (DT == DT_F32) static_cast<float *>(a.O)[at] = o[j] * inv;
        else static_cast<uint16_t *>(a.O)[at] = float_to_bf16_rne(o[j] * inv);
    }
    if (a.lse && lane == 0)
        a.lse[tok * a.heads + head] = l > 0.0f ? (m + log2f(l)) * ATTN_LN2 : -__builtin_inff();
}

int64_t attn_workspace_bytes(int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t seqs,
                             int64_t max_q, int64_t max_own, int64_t prefix)
{
    (void)tokens, (void)heads, (void)kv_heads, (void)head_dim, (void)seqs, (void)max_q, (void)max_own, (void)prefix;
    return 0;
}

hipError_t launch_attention(const AttnArgs &a, hipStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(a.seqs) * static_cast<unsigned>(a.max_q), static_cast<unsigned>(a.heads)), block(64);
    if (a.dtype == DT_F32) hipLaunchKernelGGL(k_attn_rows<DT_F32>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(k_attn_rows<DT_BF16>, grid, block, 0, stream, a);
    return hipGetLastError();
}

} // namespace bl
