// cache.hip -- keys and values quantised to int8 as they are written into the
// paged cache, and read back.  Per token and head: scale = max|x| / 127, byte =
// rint(x (127 / max|x|)), the activation quantiser's rounding.
#include "cache_core.h"
#include "common.h"
#include "launch.h"

namespace bl {

// One wave per (token, head): blockIdx.x the token, blockIdx.y K or V, the
// waves of a workgroup the heads.
template <int DT>
__global__ __launch_bounds__(256) void k_cache_write(const CacheView c, const CacheRows r, const int64_t *slots)
{
    const int64_t m = blockIdx.x, slot = slots[m];
    if (slot < 0 || slot >= c.slots) return;
    const bool is_v = blockIdx.y != 0;
    const int64_t page = slot / c.page_tokens;
    const int t = static_cast<int>(slot % c.page_tokens);
    for (int head = wave_id(); head < c.heads; head += 4) {
        const void *src = is_v ? r.V : r.K;
        const int64_t off = m * (is_v ? r.ldv_t : r.ldk_t) + head * (is_v ? r.ldv_h : r.ldk_h);
        float top = 0.0f;
        for (int d = lane_id(); d < c.D; d += 64) top = fmaxf(top, fabsf(load_x<DT>(src, off + d)));
        top = wave_max_nonneg(top);
        const TokenQuant s = token_quant(top);
        const int64_t row0 = cache_row0(c, page, head);
        for (int d = lane_id(); d < c.Dp; d += 64) {
            const int8_t q = static_cast<int8_t>(d < c.D ? quant_one(load_x<DT>(src, off + d), s) : 0u);
            if (is_v) c.V[(row0 + t / CACHE_BLOCK * CACHE_BLOCK) * c.Dp + d * CACHE_BLOCK + cache_v_byte(t % CACHE_BLOCK)] = q;
            else c.K[(row0 + t) * c.Dp + d] = q;
        }
        if (lane_id() == 0) (is_v ? c.Vs : c.Ks)[row0 + t] = top / 127.0f;
    }
}

template <int DT>
__global__ __launch_bounds__(256) void k_cache_read(const CacheView c, const CacheRows r, const int64_t *slots)
{
    const int64_t m = blockIdx.x, slot = slots[m];
    const bool is_v = blockIdx.y != 0, ok = slot >= 0 && slot < c.slots;
    const int64_t page = ok ? slot / c.page_tokens : 0;
    const int t = ok ? static_cast<int>(slot % c.page_tokens) : 0;
    for (int head = wave_id(); head < c.heads; head += 4) {
        void *dst = is_v ? r.V : r.K;
        const int64_t off = m * (is_v ? r.ldv_t : r.ldk_t) + head * (is_v ? r.ldv_h : r.ldk_h);
        const int64_t row0 = cache_row0(c, page, head);
        const float s = ok ? (is_v ? c.Vs : c.Ks)[row0 + t] : 0.0f;
        for (int d = lane_id(); d < c.D; d += 64) {
            float v = 0.0f;
            if (ok) {
                const int8_t q = is_v ? c.V[(row0 + t / CACHE_BLOCK * CACHE_BLOCK) * c.Dp + d * CACHE_BLOCK +
                                            cache_v_byte(t % CACHE_BLOCK)]
                                      : c.K[(row0 + t) * c.Dp + d];
                v = static_cast<float>(q) * s;
            }
            if constexpr (DT == DT_F32) static_cast<float *>(dst)[off + d] = v;
            else static_cast<uint16_t *>(dst)[off + d] = float_to_bf16_rne(v);
        }
    }
}

hipError_t launch_cache_write(const CacheView &c, const CacheRows &r, int dtype, int64_t tokens, const int64_t *slots,
                              hipStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(tokens), 2), block(256);
    if (dtype == DT_F32) hipLaunchKernelGGL(k_cache_write<DT_F32>, grid, block, 0, stream, c, r, slots);
    else hipLaunchKernelGGL(k_cache_write<DT_BF16>, grid, block, 0, stream, c, r, slots);
    return hipGetLastError();
}

hipError_t launch_cache_read(const CacheView &c, const CacheRows &r, int dtype, int64_t tokens, const int64_t *slots,
                             hipStream_t stream)
{
    const dim3 grid(static_cast<unsigned>(tokens), 2), block(256);
    if (dtype == DT_F32) hipLaunchKernelGGL(k_cache_read<DT_F32>, grid, block, 0, stream, c, r, slots);
    else hipLaunchKernelGGL(k_cache_read<DT_BF16>, grid, block, 0, stream, c, r, slots);
    return hipGetLastError();
}

} // namespace bl
