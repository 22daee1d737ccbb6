// norm.hip -- RMS norm with the residual's addition and per-token int8 output,
// its gradient, and the values of int8 rows.
//
//   h = x + r,  rho = 1 / sqrt(mean h^2 + eps),  y = (h rho) w,
//   beta = max|y|,  q = rint(y 127 / beta)
// Activations of a BitLinear are 8-bit (LIT-380 record, dmarx anthology, Key
// takeaways, bullet 1); the norm before it can write them itself.
//
// Rows are read and written once: a workgroup holds its row in registers, eight
// consecutive elements (a "piece") per thread and slot.  Sums of squares are
// binary64: a term h^2 is exact there, so rho does not depend on the order of
// the sum to binary32's precision, and no h overflows it.
// Bound: HBM for many rows; for few, the chain load - sum - maximum - store.
// Measured (a copy of 1 GiB moves 4.78 TB/s, read and written): 8192 x 8192 bf16 with
// residual and kept sum, 470 MB: 102 us, 4.6 TB/s (tiled rows: 128, 16-byte pieces 1 KB
// apart); 176 x 8640 fp32: 7.1 us, a workgroup a row on 176 of 256 CUs; 1 x 3200: 3.9 us.
// The same passes as separate reads of the row took 3.6 times as long.
#include "common.h"
#include "launch.h"
#include "rows.h"

namespace bl {

// Sum over the wave in binary64, in every lane.
__device__ __forceinline__ double wave_sum64(double v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Sum over the workgroup (every lane active); red: one slot per wave, used once.
__device__ __forceinline__ double block_sum64(double v, double *red)
{
    v = wave_sum64(v);
    if (lane_id() == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double r = red[0];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 6); ++w) r += red[w];
    return r;
}

__device__ __forceinline__ float block_max_nn(float v, float *red)
{
    v = wave_max_nonneg(v);
    if (lane_id() == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float r = red[0];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 6); ++w) r = fmaxf(r, red[w]);
    return r;
}

// rho of a row from its sum of squares (binary64, rounded once; finite).
__device__ __forceinline__ float inv_rms(double ss, int64_t K, float eps)
{
    const double v = ss / static_cast<double>(K) + static_cast<double>(eps);
    if (!(v > 0.0)) return 0.0f;
    const float r = static_cast<float>(1.0 / sqrt(v));
    return r < 3.402823466e38f ? r : 3.402823466e38f;
}

// Byte of token m, column k (a multiple of 8) in the tiled activation layout (bitlinear.h).
__device__ __forceinline__ int64_t tiled_offset(int64_t m, int k, int layout, int nsteps)
{
    const int step_k = layout == LAYOUT_I2 ? 256 : (layout == LAYOUT_B3 ? 320 : 512), kblk = step_k / 4;
    const int nmf = layout == LAYOUT_I2 ? 4 : (layout == LAYOUT_B3 ? 5 : 8);
    const int st = k / step_k, r = k % step_k, g = r / kblk, d = (r % kblk) / 16;
    return (((m / 16 * nsteps + st) * nmf + d) * 64 + g * 16 + m % 16) * 16 + k % 16;
}

__device__ __forceinline__ void fill8(float (&v)[8], float x)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x;
}

// One workgroup per row, PPT pieces per thread.  'pieces' covers the row up to a
// multiple of 16 (tiled: the layout's padding): bytes past K are written with 0,
// and so are a wide stride's bytes past the pieces and whole rows past M (tiled
// layout).  A thread reads an element of x and r before it writes that
// element of H, so H may be either.
template <int XDT, int HDT, int PPT>
__global__ __launch_bounds__(1024) void k_norm_rows(const NormArgs a, int pieces, int nsteps)
{
    __shared__ double red64[16];
    __shared__ float red[16];
    const int64_t m = blockIdx.x;
    const int K = static_cast<int>(a.K);
    const bool live = m < a.M;
    float h[PPT][8], w[PPT][8];
#pragma unroll
    for (int j = 0; j < PPT; ++j) {
        const int k = 8 * static_cast<int>(threadIdx.x + j * blockDim.x);
        load8<XDT>(a.X, m * a.ldx + k, live ? K - k : 0, h[j]);
    }
    if (a.R) {
        float r[PPT][8];
#pragma unroll
        for (int j = 0; j < PPT; ++j) {
            const int k = 8 * static_cast<int>(threadIdx.x + j * blockDim.x);
            load8<HDT>(a.R, m * a.ldr + k, live ? K - k : 0, r[j]);
        }
#pragma unroll
        for (int j = 0; j < PPT; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[j][e] += r[j][e];
    }
#pragma unroll
    for (int j = 0; j < PPT; ++j) {
        const int k = 8 * static_cast<int>(threadIdx.x + j * blockDim.x);
        if (a.w) load8<DT_F32>(a.w, k, K - k, w[j]);
        else fill8(w[j], 1.0f);
    }
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < PPT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double x = h[j][e];
            ss = __builtin_fma(x, x, ss);
        }
    if (a.H && live) {
#pragma unroll
        for (int j = 0; j < PPT; ++j) {
            const int k = 8 * static_cast<int>(threadIdx.x + j * blockDim.x);
            store8<HDT>(a.H, m * a.ldh + k, K - k, h[j]);
        }
    }
    const float rho = inv_rms(block_sum64(ss, red64), a.K, a.eps);
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < PPT; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[j][e] = h[j][e] * rho * w[j][e];
            top = fmaxf(top, fabsf(h[j][e]));
        }
    const float b = block_max_nn(top, red);
    const TokenQuant s = token_quant(b);
#pragma unroll
    for (int j = 0; j < PPT; ++j) {
        const int p = static_cast<int>(threadIdx.x + j * blockDim.x);
        if (p >= pieces) continue;
        const uint2 q = make_uint2(quant4_bounded(h[j][0], h[j][1], h[j][2], h[j][3], s),
                                   quant4_bounded(h[j][4], h[j][5], h[j][6], h[j][7], s));
        *reinterpret_cast<uint2 *>(a.Xq + (a.layout >= 0 ? tiled_offset(m, 8 * p, a.layout, nsteps) : m * a.ldq + 8 * p)) = q;
    }
    // (int8 rows with a wide stride: the rest of the padding)
    if (a.layout < 0)
        for (int64_t k = 8 * (static_cast<int64_t>(pieces) + threadIdx.x); k < a.ldq; k += 8 * blockDim.x)
            *reinterpret_cast<uint2 *>(a.Xq + m * a.ldq + k) = make_uint2(0u, 0u);
    if (threadIdx.x == 0 && live) a.beta[m] = b;
}

// Rows too long for the registers: three passes over the row (sum of squares,
// maximum of |y|, output), a thread taking the same pieces in each.
template <int XDT, int HDT>
__global__ __launch_bounds__(1024) void k_norm_loop(const NormArgs a, int64_t width, int nsteps)
{
    __shared__ double red64[16];
    __shared__ float red[16];
    const int64_t m = blockIdx.x, K = m < a.M ? a.K : 0; // (tiled layout: rows past M are zeros)
    auto piece = [&](int64_t k, float (&h)[8], float (&w)[8]) {
        load8<XDT>(a.X, m * a.ldx + k, K - k, h);
        if (a.R) {
            float r[8];
            load8<HDT>(a.R, m * a.ldr + k, K - k, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] += r[e];
        }
        if (a.w) load8<DT_F32>(a.w, k, K - k, w);
        else fill8(w, 1.0f);
    };
    const int64_t step = 8 * static_cast<int64_t>(blockDim.x);
    float h[8], w[8];
    double ss = 0.0;
    for (int64_t k = 8 * threadIdx.x; k < K; k += step) {
        piece(k, h, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double x = h[e];
            ss = __builtin_fma(x, x, ss);
        }
    }
    const float rho = inv_rms(block_sum64(ss, red64), a.K, a.eps);
    float top = 0.0f;
    for (int64_t k = 8 * threadIdx.x; k < K; k += step) {
        piece(k, h, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(h[e] * rho * w[e]));
    }
    const float b = block_max_nn(top, red);
    const TokenQuant s = token_quant(b);
    for (int64_t k = 8 * threadIdx.x; k < width; k += step) {
        piece(k, h, w);
        if (a.H) store8<HDT>(a.H, m * a.ldh + k, K - k, h);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = h[e] * rho * w[e];
        *reinterpret_cast<uint2 *>(a.Xq + (a.layout >= 0 ? tiled_offset(m, static_cast<int>(k), a.layout, nsteps) : m * a.ldq + k)) =
            make_uint2(quant4_bounded(h[0], h[1], h[2], h[3], s), quant4_bounded(h[4], h[5], h[6], h[7], s));
    }
    if (threadIdx.x == 0 && m < a.M) a.beta[m] = b;
}

template <int XDT, int HDT>
static void launch_norm(const NormArgs &a, hipStream_t stream)
{
    const bool tiled = a.layout >= 0;
    const int nsteps = tiled ? static_cast<int>(tiled_nsteps(a.K, a.layout)) : 0;
    const int64_t width = tiled ? nsteps * tiled_step_k(a.layout) : a.ldq;
    const int64_t need = tiled ? width / 8 : (a.K + 15) / 16 * 2; // pieces of a row
    const dim3 grid(static_cast<unsigned>(tiled ? (a.M + 15) / 16 * 16 : a.M));
    // many rows: workgroups of four waves, so that rows in different phases share a CU;
    // few: one piece per thread as far as 1024 threads go, for the shorter chain
    const int64_t threads = a.M >= 1024 ? 256 : 1024;
    const int64_t ppt = need <= threads ? 1 : need <= 2 * threads ? 2 : need <= 4 * 1024 ? 4 : 0;
    const dim3 block(static_cast<unsigned>(ppt ? ((need + ppt - 1) / ppt + 63) / 64 * 64 : 1024));
    const int pieces = static_cast<int>(need);
    if (ppt == 1) hipLaunchKernelGGL((k_norm_rows<XDT, HDT, 1>), grid, block, 0, stream, a, pieces, nsteps);
    else if (ppt == 2) hipLaunchKernelGGL((k_norm_rows<XDT, HDT, 2>), grid, block, 0, stream, a, pieces, nsteps);
    else if (ppt == 4) hipLaunchKernelGGL((k_norm_rows<XDT, HDT, 4>), grid, block, 0, stream, a, pieces, nsteps);
    else hipLaunchKernelGGL((k_norm_loop<XDT, HDT>), grid, block, 0, stream, a, width, nsteps);
}

hipError_t launch_norm_quantize(const NormArgs &a, hipStream_t stream)
{
    if (a.x_dtype == DT_F32) {
        if (a.h_dtype == DT_F32) launch_norm<DT_F32, DT_F32>(a, stream);
        else launch_norm<DT_F32, DT_BF16>(a, stream);
    } else {
        if (a.h_dtype == DT_F32) launch_norm<DT_BF16, DT_F32>(a, stream);
        else launch_norm<DT_BF16, DT_BF16>(a, stream);
    }
    return hipGetLastError();
}

// V = q (beta / 127), a piece per thread, 'chunks' workgroups a row.  Bound: HBM
// (8192 x 8192 to bf16 behind the norm: 33 us, 6.0 TB/s, the bytes partly in cache).
template <int DT>
__global__ __launch_bounds__(256) void k_dequantize(const int8_t *Xq, int64_t ldq, const float *beta, int64_t K, void *V,
                                                    int64_t ldv, uint32_t chunks)
{
    const uint32_t m = blockIdx.x / chunks, k = (blockIdx.x % chunks * 256 + threadIdx.x) * 8;
    if (k >= K) return;
    const float r = beta[m] / 127.0f;
    const int8_t *src = Xq + m * ldq + k;
    uint32_t w[2] = {0, 0};
    if (K - k >= 8) {
        const u2_any u = *reinterpret_cast<const u2_any *>(src);
        w[0] = u[0];
        w[1] = u[1];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (k + e < K) w[e / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(src[e])) << (8 * (e % 4));
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(static_cast<int8_t>(w[e / 4] >> (8 * (e % 4)))) * r;
    store8<DT>(V, m * ldv + k, K - k, v);
}

hipError_t launch_dequantize_act(const int8_t *Xq, int64_t ldq, const float *beta, int64_t M, int64_t K, void *V,
                                 int v_dtype, int64_t ldv, hipStream_t stream)
{
    const uint32_t chunks = static_cast<uint32_t>((K + 2047) / 2048);
    const dim3 grid(static_cast<unsigned>(M) * chunks);
    if (v_dtype == DT_F32) hipLaunchKernelGGL(k_dequantize<DT_F32>, grid, dim3(256), 0, stream, Xq, ldq, beta, K, V, ldv, chunks);
    else hipLaunchKernelGGL(k_dequantize<DT_BF16>, grid, dim3(256), 0, stream, Xq, ldq, beta, K, V, ldv, chunks);
    return hipGetLastError();
}

// ---- gradient ---------------------------------------------------------------
// A workgroup takes rows p, p + parts, ... and keeps its share of dW, a row of K
// sums, in registers; k_norm_bwd_sum adds the workgroups' rows in a fixed order, so
// that no atomic's order reaches dW.  Bound: HBM.  2048 x 8640 bf16 with dH, 177 MB:
// 38 us, 4.6 TB/s, and 4.8 us for the sum; 100 x 3200 fp32: 5.2 and 3.2 us; rows past
// the registers (k_norm_bwd_loop), 2048 x 28672 bf16, 587 MB: 218 and 6.5 us.
int64_t norm_bwd_parts(int64_t M, int64_t K)
{
    const int64_t parts = K <= 4096 ? 512 : 256; // one or two for each CU
    return M < parts ? M : parts;
}

// The row's two sums, sum h^2 and sum g h, over the workgroup; red: two slots per wave.
__device__ __forceinline__ void block_sums64(double &a, double &b, double (*red)[2])
{
    a = wave_sum64(a);
    b = wave_sum64(b);
    if (lane_id() == 0) {
        red[threadIdx.x >> 6][0] = a;
        red[threadIdx.x >> 6][1] = b;
    }
    __syncthreads();
    a = red[0][0];
    b = red[0][1];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 6); ++w) {
        a += red[w][0];
        b += red[w][1];
    }
}

// c of dX = rho g - c h + dH.
__device__ __forceinline__ float bwd_factor(float rho, double gh, int64_t K)
{
    const double r = rho;
    return static_cast<float>(r * r * r * gh / static_cast<double>(K));
}

// Threads of a workgroup by its pieces per thread: what the registers of a row's
// dY, h, w, dX and dW allow.
constexpr int bwd_threads(int ppt) { return ppt == 1 ? 1024 : (ppt == 2 ? 640 : 512); }

template <int HDT, int PPT>
__global__ __launch_bounds__(bwd_threads(PPT)) void k_norm_bwd_rows(const NormBwdArgs a)
{
    __shared__ double red[2][16][2]; // alternating, so that one barrier a row is enough
    const int K = static_cast<int>(a.K);
    float w[PPT][8], acc[PPT][8], dy[PPT][8], h[PPT][8];
    auto at = [&](int j) { return 8 * static_cast<int>(threadIdx.x + j * blockDim.x); };
    auto fetch = [&](int64_t m) {
#pragma unroll
        for (int j = 0; j < PPT; ++j) load8<DT_F32>(a.dY, m * a.lddy + at(j), K - at(j), dy[j]);
#pragma unroll
        for (int j = 0; j < PPT; ++j) load8<HDT>(a.H, m * a.ldh + at(j), K - at(j), h[j]);
    };
    fetch(blockIdx.x);
#pragma unroll
    for (int j = 0; j < PPT; ++j) {
        if (a.w) load8<DT_F32>(a.w, at(j), K - at(j), w[j]);
        else fill8(w[j], 1.0f);
        fill8(acc[j], 0.0f);
    }
    int turn = 0;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
        double ss = 0.0, gh = 0.0;
        float dx[PPT][8];
#pragma unroll
        for (int j = 0; j < PPT; ++j) {
            if (a.dH) load8<HDT>(a.dH, m * a.lddh + at(j), K - at(j), dx[j]);
            else fill8(dx[j], 0.0f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double x = h[j][e];
                ss = __builtin_fma(x, x, ss);
                gh = __builtin_fma(x, static_cast<double>(dy[j][e] * w[j][e]), gh);
            }
        }
        block_sums64(ss, gh, red[turn]);
        const float rho = inv_rms(ss, a.K, a.eps), c = bwd_factor(rho, gh, a.K);
#pragma unroll
        for (int j = 0; j < PPT; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dx[j][e] = (rho * (dy[j][e] * w[j][e]) - c * h[j][e]) + dx[j][e];
                acc[j][e] += dy[j][e] * (h[j][e] * rho);
            }
            store8<HDT>(a.dX, m * a.lddx + at(j), K - at(j), dx[j]);
        }
        if (m + gridDim.x < a.M) fetch(m + gridDim.x);
    }
    if (a.dW)
#pragma unroll
        for (int j = 0; j < PPT; ++j) store8<DT_F32>(a.part, blockIdx.x * a.K + at(j), K - at(j), acc[j]);
}

// Rows too long for the registers: two passes over each row, the share of dW in
// the workgroup's row of the workspace.
template <int HDT>
__global__ __launch_bounds__(1024) void k_norm_bwd_loop(const NormBwdArgs a)
{
    __shared__ double red[2][16][2];
    const int64_t step = 8 * static_cast<int64_t>(blockDim.x);
    int turn = 0;
    float dy[8], h[8], w[8], t[8];
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
        auto piece = [&](int64_t k) {
            load8<DT_F32>(a.dY, m * a.lddy + k, a.K - k, dy);
            load8<HDT>(a.H, m * a.ldh + k, a.K - k, h);
            if (a.w) load8<DT_F32>(a.w, k, a.K - k, w);
            else fill8(w, 1.0f);
        };
        double ss = 0.0, gh = 0.0;
        for (int64_t k = 8 * threadIdx.x; k < a.K; k += step) {
            piece(k);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double x = h[e];
                ss = __builtin_fma(x, x, ss);
                gh = __builtin_fma(x, static_cast<double>(dy[e] * w[e]), gh);
            }
        }
        block_sums64(ss, gh, red[turn]);
        const float rho = inv_rms(ss, a.K, a.eps), c = bwd_factor(rho, gh, a.K);
        for (int64_t k = 8 * threadIdx.x; k < a.K; k += step) {
            piece(k);
            if (a.dH) load8<HDT>(a.dH, m * a.lddh + k, a.K - k, t);
            else fill8(t, 0.0f);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = (rho * (dy[e] * w[e]) - c * h[e]) + t[e];
            store8<HDT>(a.dX, m * a.lddx + k, a.K - k, t);
            if (a.dW) {
                const int64_t p = blockIdx.x * a.K + k;
                if (m == static_cast<int64_t>(blockIdx.x)) fill8(t, 0.0f);
                else load8<DT_F32>(a.part, p, a.K - k, t);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] += dy[e] * (h[e] * rho);
                store8<DT_F32>(a.part, p, a.K - k, t);
            }
        }
    }
}

// dW[k]: 32 columns a workgroup, 32 threads a column, each the sum of every 32nd
// partial row in order; then the 32 sums in order.
__global__ __launch_bounds__(1024) void k_norm_bwd_sum(const float *part, int parts, int64_t K, float *dW)
{
    __shared__ float red[32][33];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * 32 + c;
    float s = 0.0f;
    if (k < K)
#pragma unroll 8
        for (int p = g; p < parts; p += 32) s += part[p * K + k];
    red[g][c] = s;
    __syncthreads();
    if (g == 0 && k < K) {
#pragma unroll
        for (int x = 1; x < 32; ++x) s += red[x][c];
        dW[k] = s;
    }
}

template <int HDT>
static void launch_norm_bwd(const NormBwdArgs &a, unsigned parts, hipStream_t stream)
{
    const int64_t need = (a.K + 7) / 8;
    const dim3 grid(parts);
    const int64_t ppt = need <= bwd_threads(1) ? 1 : need <= 2 * bwd_threads(2) ? 2 : need <= 4 * bwd_threads(4) ? 4 : 0;
    const dim3 block(static_cast<unsigned>(ppt ? ((need + ppt - 1) / ppt + 63) / 64 * 64 : 1024));
    if (ppt == 1) hipLaunchKernelGGL((k_norm_bwd_rows<HDT, 1>), grid, block, 0, stream, a);
    else if (ppt == 2) hipLaunchKernelGGL((k_norm_bwd_rows<HDT, 2>), grid, block, 0, stream, a);
    else if (ppt == 4) hipLaunchKernelGGL((k_norm_bwd_rows<HDT, 4>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL(k_norm_bwd_loop<HDT>, grid, dim3(1024), 0, stream, a);
}

hipError_t launch_norm_backward(const NormBwdArgs &a, hipStream_t stream)
{
    const unsigned parts = static_cast<unsigned>(norm_bwd_parts(a.M, a.K));
    if (a.h_dtype == DT_F32) launch_norm_bwd<DT_F32>(a, parts, stream);
    else launch_norm_bwd<DT_BF16>(a, parts, stream);
    if (a.dW)
        hipLaunchKernelGGL(k_norm_bwd_sum, dim3(static_cast<unsigned>((a.K + 31) / 32)), dim3(1024), 0, stream, a.part,
                           static_cast<int>(parts), a.K, a.dW);
    return hipGetLastError();
}

} // namespace bl
