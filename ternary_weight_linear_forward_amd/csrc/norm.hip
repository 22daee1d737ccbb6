// norm.hip -- RMS norm with the residual's addition and per-token int8 output,
// its gradient, and the values of int8 rows.
//
//   h = x + r,  rho = 1 / sqrt(mean h^2 + eps),  y = (h rho) w,
//   beta = max|y|,  q = rint(y 127 / beta)
// Activations of a BitLinear are 8-bit (LIT-380 record, dmarx anthology, Key
// takeaways, bullet 1); the norm before it can write them itself.
#include "common.h"
#include "launch.h"

namespace bl {

__device__ __forceinline__ float load_f(const void *p, int dt, int64_t i)
{
    return dt == DT_F32 ? load_x<DT_F32>(p, i) : load_x<DT_BF16>(p, i);
}

__device__ __forceinline__ void store_f(void *p, int dt, int64_t i, float v)
{
    if (dt == DT_F32) static_cast<float *>(p)[i] = v;
    else static_cast<uint16_t *>(p)[i] = float_to_bf16_rne(v);
}

// Sum over the workgroup in binary64 (every lane active).
__device__ __forceinline__ double block_sum64(double v, double *red)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if (lane_id() == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double r = 0.0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) r += red[w];
    __syncthreads();
    return r;
}

__device__ __forceinline__ float block_max_nn(float v, float *red)
{
    v = wave_max_nonneg(v);
    if (lane_id() == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float r = red[0];
    for (int w = 1; w < static_cast<int>(blockDim.x >> 6); ++w) r = fmaxf(r, red[w]);
    __syncthreads();
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

// Byte of token m, column k in the tiled activation layout (bitlinear.h).
__device__ __forceinline__ int64_t tiled_offset(int64_t m, int64_t k, int layout, int64_t nsteps)
{
    const int64_t step_k = layout == LAYOUT_I2 ? 256 : (layout == LAYOUT_B3 ? 320 : 512), kblk = step_k / 4;
    const int64_t nmf = layout == LAYOUT_I2 ? 4 : (layout == LAYOUT_B3 ? 5 : 8);
    const int64_t st = k / step_k, r = k % step_k, g = r / kblk, d = (r % kblk) / 16;
    return (((m / 16 * nsteps + st) * nmf + d) * 64 + g * 16 + m % 16) * 16 + k % 16;
}

// One workgroup per row, three passes over it: sum of squares, maximum of |y|,
// output.  An element of H is written by the thread that reads it (H may be X
// or R).
__global__ __launch_bounds__(1024) void k_norm_loop(const NormArgs a, int64_t nsteps, int64_t width)
{
    __shared__ double red64[16];
    __shared__ float red[16];
    const int64_t m = blockIdx.x;
    const bool live = m < a.M;
    auto h_of = [&](int64_t k) {
        const float x = load_f(a.X, a.x_dtype, m * a.ldx + k);
        return a.R ? x + load_f(a.R, a.h_dtype, m * a.ldr + k) : x;
    };
    double ss = 0.0;
    if (live)
        for (int64_t k = threadIdx.x; k < a.K; k += blockDim.x) {
            const double h = h_of(k);
            ss += h * h;
        }
    const float rho = inv_rms(block_sum64(ss, red64), a.K, a.eps);
    float top = 0.0f;
    if (live)
        for (int64_t k = threadIdx.x; k < a.K; k += blockDim.x)
            top = fmaxf(top, fabsf(h_of(k) * rho * (a.w ? a.w[k] : 1.0f)));
    const float b = block_max_nn(top, red);
    const TokenQuant s = token_quant(b);
    for (int64_t k = threadIdx.x; k < width; k += blockDim.x) {
        uint32_t q = 0;
        if (live && k < a.K) {
            const float h = h_of(k);
            if (a.H) store_f(a.H, a.h_dtype, m * a.ldh + k, h);
            q = quant_one(h * rho * (a.w ? a.w[k] : 1.0f), s);
        }
        a.Xq[a.layout >= 0 ? tiled_offset(m, k, a.layout, nsteps) : m * a.ldq + k] = static_cast<int8_t>(q);
    }
    if (threadIdx.x == 0 && live) a.beta[m] = b;
}

hipError_t launch_norm_quantize(const NormArgs &a, hipStream_t stream)
{
    const bool tiled = a.layout >= 0;
    const int64_t nsteps = tiled ? tiled_nsteps(a.K, a.layout) : 0;
    const int64_t width = tiled ? nsteps * tiled_step_k(a.layout) : a.ldq;
    const int64_t rows = tiled ? (a.M + 15) / 16 * 16 : a.M;
    hipLaunchKernelGGL(k_norm_loop, dim3(static_cast<unsigned>(rows)), dim3(1024), 0, stream, a, nsteps, width);
    return hipGetLastError();
}

// V = q (beta / 127).
__global__ __launch_bounds__(256) void k_dequantize(const int8_t *Xq, int64_t ldq, const float *beta, int64_t K, void *V,
                                                    int v_dtype, int64_t ldv)
{
    const int64_t m = blockIdx.x;
    const float r = beta[m] / 127.0f;
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x)
        store_f(V, v_dtype, m * ldv + k, static_cast<float>(Xq[m * ldq + k]) * r);
}

hipError_t launch_dequantize_act(const int8_t *Xq, int64_t ldq, const float *beta, int64_t M, int64_t K, void *V,
                                 int v_dtype, int64_t ldv, hipStream_t stream)
{
    hipLaunchKernelGGL(k_dequantize, dim3(static_cast<unsigned>(M)), dim3(256), 0, stream, Xq, ldq, beta, K, V, v_dtype,
                       ldv);
    return hipGetLastError();
}

// ---- gradient ---------------------------------------------------------------
int64_t norm_bwd_parts(int64_t M, int64_t K)
{
    (void)K;
    return M < 256 ? M : 256;
}

// Workgroup p takes rows p, p + parts, ... : the row's sums, then dX, and the
// row's share of dW added to the workgroup's own row of partial sums.
__global__ __launch_bounds__(1024) void k_norm_bwd_loop(const NormBwdArgs a)
{
    __shared__ double red64[16];
    bool first = true;
    float *part = a.part + static_cast<int64_t>(blockIdx.x) * a.K;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        double ss = 0.0, gh = 0.0;
        for (int64_t k = threadIdx.x; k < a.K; k += blockDim.x) {
            const double h = load_f(a.H, a.h_dtype, m * a.ldh + k);
            const float g = a.dY[m * a.lddy + k] * (a.w ? a.w[k] : 1.0f);
            ss += h * h;
            gh += h * static_cast<double>(g);
        }
        const float rho = inv_rms(block_sum64(ss, red64), a.K, a.eps);
        const double r64 = rho;
        const float c = static_cast<float>(r64 * r64 * r64 * block_sum64(gh, red64) / static_cast<double>(a.K));
        for (int64_t k = threadIdx.x; k < a.K; k += blockDim.x) {
            const float h = load_f(a.H, a.h_dtype, m * a.ldh + k), dy = a.dY[m * a.lddy + k];
            const float g = dy * (a.w ? a.w[k] : 1.0f);
            float dx = rho * g - c * h;
            if (a.dH) dx += load_f(a.dH, a.h_dtype, m * a.lddh + k);
            store_f(a.dX, a.h_dtype, m * a.lddx + k, dx);
            if (a.dW) {
                const float t = dy * (h * rho);
                part[k] = first ? t : part[k] + t;
            }
        }
        first = false;
    }
}

// dW[k] = sum of the partial rows, in order.
__global__ __launch_bounds__(256) void k_norm_bwd_sum(const float *part, int64_t parts, int64_t K, float *dW)
{
    const int64_t k = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (k >= K) return;
    float s = 0.0f;
    for (int64_t p = 0; p < parts; ++p) s += part[p * K + k];
    dW[k] = s;
}

hipError_t launch_norm_backward(const NormBwdArgs &a, hipStream_t stream)
{
    const int64_t parts = norm_bwd_parts(a.M, a.K);
    hipLaunchKernelGGL(k_norm_bwd_loop, dim3(static_cast<unsigned>(parts)), dim3(1024), 0, stream, a);
    if (a.dW)
        hipLaunchKernelGGL(k_norm_bwd_sum, dim3(static_cast<unsigned>((a.K + 255) / 256)), dim3(256), 0, stream, a.part,
                           parts, a.K, a.dW);
    return hipGetLastError();
}

} // namespace bl
