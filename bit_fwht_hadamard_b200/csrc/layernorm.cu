// layernorm.cu -- layer norm of the rows of an M x D matrix, and its backward
// pass with the gradients of weight and bias.
//
// y = (x - mean) rstd gamma + beta, rstd = 1 / sqrt(var + eps).  With
// xhat = (x - mean) rstd and g = dy gamma:
//   dx = rstd (g - mean_d(g) - xhat mean_d(g xhat)),
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy.
#include "epilogue.cuh"

namespace qfp4 {

// Sums of a and b over the block, in every thread; red: 64 floats.
__device__ __forceinline__ float2 block_sum2(float a, float b, float *red)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) {
        red[warp] = a;
        red[32 + warp] = b;
    }
    __syncthreads();
    a = lane < nw ? red[lane] : 0.0f;
    b = lane < nw ? red[32 + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    return make_float2(a, b);
}

// A block a row; three reads of the row (the first from memory, the others
// from the caches).
template <int DT>
__global__ void __launch_bounds__(256) k_layernorm(const void *x, int64_t M, int64_t D, const void *gamma,
                                                    const void *beta, int w32, float eps, void *y, float *mean_out,
                                                    float *rstd_out)
{
    __shared__ float red[64];
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const int64_t r = m * D;
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < D; c += blockDim.x) s += ld_as_float(x, DT == QFP4_F32, r + c);
        const float mean = block_sum2(s, 0.0f, red).x / static_cast<float>(D);
        s = 0.0f;
        for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
            const float t = ld_as_float(x, DT == QFP4_F32, r + c) - mean;
            s += t * t;
        }
        const float rstd = 1.0f / sqrtf(block_sum2(s, 0.0f, red).x / static_cast<float>(D) + eps);
        for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
            float v = (ld_as_float(x, DT == QFP4_F32, r + c) - mean) * rstd;
            if (gamma) v *= ld_as_float(gamma, w32, c);
            if (beta) v += ld_as_float(beta, w32, c);
            if (DT == QFP4_F32) static_cast<float *>(y)[r + c] = v;
            else static_cast<__nv_bfloat16 *>(y)[r + c] = __float2bfloat16_rn(v);
        }
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[m] = mean;
            if (rstd_out) rstd_out[m] = rstd;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(256) k_layernorm_dx(const void *dy, const void *x, int64_t M, int64_t D,
                                                       const void *gamma, int w32, const float *mean_in,
                                                       const float *rstd_in, void *dx)
{
    __shared__ float red[64];
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const int64_t r = m * D;
        const float mean = mean_in[m], rstd = rstd_in[m];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
            float g = ld_as_float(dy, DT == QFP4_F32, r + c);
            if (gamma) g *= ld_as_float(gamma, w32, c);
            s1 += g;
            s2 += g * ((ld_as_float(x, DT == QFP4_F32, r + c) - mean) * rstd);
        }
        const float2 t = block_sum2(s1, s2, red);
        const float c1 = t.x / static_cast<float>(D), c2 = t.y / static_cast<float>(D);
        for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
            float g = ld_as_float(dy, DT == QFP4_F32, r + c);
            if (gamma) g *= ld_as_float(gamma, w32, c);
            const float xh = (ld_as_float(x, DT == QFP4_F32, r + c) - mean) * rstd;
            const float v = rstd * (g - c1 - xh * c2);
            if (DT == QFP4_F32) static_cast<float *>(dx)[r + c] = v;
            else static_cast<__nv_bfloat16 *>(dx)[r + c] = __float2bfloat16_rn(v);
        }
    }
}

// Column sums of a chunk of rows: partial[0][chunk][D] of dy xhat,
// partial[1][chunk][D] of dy.
template <int DT>
__global__ void __launch_bounds__(256) k_layernorm_dw(const void *dy, const void *x, int64_t M, int64_t D,
                                                       int64_t rows, const float *mean, const float *rstd,
                                                       float *partial)
{
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= D) return;
    const int64_t m0 = blockIdx.y * rows, m1 = imin(M, m0 + rows);
    float sg = 0.0f, sb = 0.0f;
    for (int64_t m = m0; m < m1; ++m) {
        const float d = ld_as_float(dy, DT == QFP4_F32, m * D + c);
        sg += d * ((ld_as_float(x, DT == QFP4_F32, m * D + c) - mean[m]) * rstd[m]);
        sb += d;
    }
    partial[blockIdx.y * D + c] = sg;
    partial[(gridDim.y + blockIdx.y) * D + c] = sb;
}

}  // namespace qfp4

using namespace qfp4;

static int layernorm_shape(int64_t M, int64_t D)
{
    return M < 0 || D < 0 || M > INT32_MAX / 2 || D > INT32_MAX / 2 || (D > 0 && M > (int64_t(1) << 38) / D)
               ? QFP4_ERR_SHAPE
               : QFP4_OK;
}

extern "C" int qfp4_layernorm_forward(const void *x, qfp4_dtype dt, int64_t M, int64_t D, const void *gamma,
                                      const void *beta, qfp4_dtype wdt, float eps, void *y, float *mean, float *rstd,
                                      qfp4_stream_t stream)
{
    if ((dt != QFP4_BF16 && dt != QFP4_F32) || (wdt != QFP4_BF16 && wdt != QFP4_F32)) return QFP4_ERR_ARG;
    if (!(eps >= 0.0f)) return QFP4_ERR_ARG;
    if (layernorm_shape(M, D) != QFP4_OK) return QFP4_ERR_SHAPE;
    if (M > 0 && D == 0) return QFP4_ERR_SHAPE;
    if (M > 0 && (!x || !y)) return QFP4_ERR_ARG;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(y) || !aligned16(mean) || !aligned16(rstd))
        return QFP4_ERR_ALIGN;
    if (M == 0) return QFP4_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int grid = static_cast<int>(imin<int64_t>(M, 64 * num_sms()));
    const int w32 = wdt == QFP4_F32;
    if (dt == QFP4_F32) k_layernorm<QFP4_F32><<<grid, 256, 0, s>>>(x, M, D, gamma, beta, w32, eps, y, mean, rstd);
    else k_layernorm<QFP4_BF16><<<grid, 256, 0, s>>>(x, M, D, gamma, beta, w32, eps, y, mean, rstd);
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

extern "C" size_t qfp4_layernorm_backward_workspace_bytes(int64_t M, int64_t D)
{
    if (M <= 0 || D <= 0 || layernorm_shape(M, D) != QFP4_OK) return 0;
    return 2 * sizeof(float) * epilogue_chunks(M, D) * D;
}

extern "C" int qfp4_layernorm_backward(const void *dy, const void *x, qfp4_dtype dt, int64_t M, int64_t D,
                                       const void *gamma, qfp4_dtype wdt, const float *mean, const float *rstd,
                                       void *dx, float *dgamma, float *dbeta, void *workspace, size_t workspace_bytes,
                                       qfp4_stream_t stream)
{
    if ((dt != QFP4_BF16 && dt != QFP4_F32) || (wdt != QFP4_BF16 && wdt != QFP4_F32)) return QFP4_ERR_ARG;
    if (layernorm_shape(M, D) != QFP4_OK) return QFP4_ERR_SHAPE;
    if (M > 0 && D == 0) return QFP4_ERR_SHAPE;
    if (!dx && !dgamma && !dbeta) return QFP4_ERR_ARG;
    if (M > 0 && (!dy || !x || !mean || !rstd)) return QFP4_ERR_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(gamma) || !aligned16(mean) || !aligned16(rstd) ||
        !aligned16(dx) || !aligned16(dgamma) || !aligned16(dbeta) || !aligned16(workspace))
        return QFP4_ERR_ALIGN;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) {
        if (dgamma && D > 0 && cudaMemsetAsync(dgamma, 0, D * sizeof(float), s) != cudaSuccess) return QFP4_ERR_CUDA;
        if (dbeta && D > 0 && cudaMemsetAsync(dbeta, 0, D * sizeof(float), s) != cudaSuccess) return QFP4_ERR_CUDA;
        return QFP4_OK;
    }
    const bool dw = dgamma || dbeta;
    if (dw && (!workspace || workspace_bytes < qfp4_layernorm_backward_workspace_bytes(M, D))) return QFP4_ERR_ARG;
    // dgamma and dbeta first: dx may overwrite dy
    if (dw) {
        const int64_t chunks = epilogue_chunks(M, D), rows = (M + chunks - 1) / chunks, used = (M + rows - 1) / rows;
        float *partial = static_cast<float *>(workspace);
        const dim3 grid(static_cast<unsigned>((D + 255) / 256), static_cast<unsigned>(used));
        if (dt == QFP4_F32) k_layernorm_dw<QFP4_F32><<<grid, 256, 0, s>>>(dy, x, M, D, rows, mean, rstd, partial);
        else k_layernorm_dw<QFP4_BF16><<<grid, 256, 0, s>>>(dy, x, M, D, rows, mean, rstd, partial);
        QFP4_LAUNCH_CHECK();
        const int st = column_sums(partial, used, D, dgamma, dbeta, true, s);
        if (st != QFP4_OK) return st;
    }
    const int w32 = wdt == QFP4_F32;
    if (dx) {
        const int grid = static_cast<int>(imin<int64_t>(M, 64 * num_sms()));
        if (dt == QFP4_F32) k_layernorm_dx<QFP4_F32><<<grid, 256, 0, s>>>(dy, x, M, D, gamma, w32, mean, rstd, dx);
        else k_layernorm_dx<QFP4_BF16><<<grid, 256, 0, s>>>(dy, x, M, D, gamma, w32, mean, rstd, dx);
        QFP4_LAUNCH_CHECK();
    }
    return QFP4_OK;
}
