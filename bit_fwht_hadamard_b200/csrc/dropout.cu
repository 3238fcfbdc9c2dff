// dropout.cu -- dropout from Philox words (no stored mask), optionally added
// to a residual, and the backward pass of the GEMM's epilogue (dropout,
// activation, bias).
#include "epilogue.cuh"

namespace qfp4 {

// Four consecutive elements as binary32, and back.
template <int DT>
__device__ __forceinline__ float4 ld4(const void *p, int64_t i)   // 4-element aligned
{
    if (DT == QFP4_F32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
    return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}
template <int DT>
__device__ __forceinline__ void st4(void *p, int64_t i, float4 v)
{
    if (DT == QFP4_F32) *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) =
            make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}
template <int DT>
__device__ __forceinline__ void st1(void *p, int64_t i, float v)
{
    if (DT == QFP4_F32) static_cast<float *>(p)[i] = v;
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// ------------------------------------------------------------------ dropout
template <int DT, bool RES>
__global__ void __launch_bounds__(256) k_dropout(const void *x, const void *res, int64_t n, DropParams d, void *out)
{
    const uint64_t step = drop_step(d);
    const int64_t nth = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t qd = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; qd < (n + 3) / 4; qd += nth) {
        uint4 w = make_uint4(~0u, ~0u, ~0u, ~0u);
        if (d.on) w = drop_words4(d, step, static_cast<uint64_t>(qd));
        const int64_t i = 4 * qd;
        if (i + 4 <= n) {
            float4 v = ld4<DT>(x, i);
            v = make_float4(drop1(d, v.x, w.x), drop1(d, v.y, w.y), drop1(d, v.z, w.z), drop1(d, v.w, w.w));
            if (RES) {
                const float4 r = ld4<DT>(res, i);
                v = make_float4(v.x + r.x, v.y + r.y, v.z + r.z, v.w + r.w);
            }
            st4<DT>(out, i, v);
        } else {
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            for (int t = 0; i + t < n; ++t) {
                float v = drop1(d, ld_as_float(x, DT == QFP4_F32, i + t), ww[t]);
                if (RES) v += ld_as_float(res, DT == QFP4_F32, i + t);
                st1<DT>(out, i + t, v);
            }
        }
    }
}

template <int DT>
static int launch_dropout(const void *x, const void *res, int64_t n, const DropParams &d, void *out, cudaStream_t s)
{
    const int grid = static_cast<int>(imin<int64_t>(((n + 3) / 4 + 255) / 256, 8 * num_sms()));
    if (res) k_dropout<DT, true><<<grid, 256, 0, s>>>(x, res, n, d, out);
    else k_dropout<DT, false><<<grid, 256, 0, s>>>(x, res, n, d, out);
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

// ------------------------------------------------------------------ epilogue backward
// One thread a column and row chunk: dz = drop(dy) act'(z), and the chunk's
// column sum into partial[chunk][N].
template <int DT>
__global__ void __launch_bounds__(256) k_epilogue_backward(const void *dy, const void *z, int64_t M, int64_t N,
                                                            int64_t rows, int act, DropParams d, void *dz,
                                                            float *partial)
{
    const uint64_t step = drop_step(d);
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= N) return;
    const int64_t m0 = blockIdx.y * rows, m1 = imin(M, m0 + rows);
    float sum = 0.0f;
    for (int64_t m = m0; m < m1; ++m) {
        const int64_t i = m * N + c;
        float v = ld_as_float(dy, DT == QFP4_F32, i);
        if (d.on) {
            const uint4 w = drop_words4(d, step, static_cast<uint64_t>(i) >> 2);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            v = drop1(d, v, ww[i & 3]);
        }
        if (act != QFP4_ACT_NONE) {
            const float zz = ld_as_float(z, DT == QFP4_F32, i);
            float vv[2] = {v, 0.0f}, zv[2] = {zz, 0.0f};
            act_backward<2>(vv, zv, act);
            v = vv[0];
        }
        sum += v;
        st1<DT>(dz, i, v);
    }
    if (partial) partial[blockIdx.y * N + c] = sum;
}

// out[c] = sum over the rows of partial (rows x N), in a fixed order: 32
// columns x 8 row lanes a block.  blockIdx.y selects one of up to two arrays.
__global__ void __launch_bounds__(256) k_column_sums(const float *partial, int64_t rows, int64_t N, float *out0,
                                                      float *out1)
{
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float *out = blockIdx.y ? out1 : out0;
    const float *src = partial + blockIdx.y * rows * N;
    float s = 0.0f;
    if (c < N)
        for (int64_t r = w; r < rows; r += 8) s += src[r * N + c];
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < N && out) {
        for (int k = 1; k < 8; ++k) s += red[k][lane];
        out[c] = s;
    }
}

static int column_sums(const float *partial, int64_t rows, int64_t N, float *out0, float *out1, bool two,
                       cudaStream_t s)
{
    k_column_sums<<<dim3(static_cast<unsigned>((N + 31) / 32), two ? 2 : 1), 256, 0, s>>>(partial, rows, N, out0, out1);
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

// Row chunks of the epilogue's backward pass: enough blocks for four waves
// of the device, at most 512 (the partial sums' rows).
static int64_t epilogue_chunks(int64_t M, int64_t N)
{
    const int64_t cols = (N + 255) / 256;
    return imax<int64_t>(1, imin<int64_t>(imin<int64_t>(M, 512), (8 * 148 + cols - 1) / cols));
}

}  // namespace qfp4

using namespace qfp4;

extern "C" int qfp4_dropout(const void *x, qfp4_dtype dt, int64_t n, double p, uint64_t seed, const uint64_t *step,
                            const void *residual, void *out, qfp4_stream_t stream)
{
    if (dt != QFP4_BF16 && dt != QFP4_F32) return QFP4_ERR_ARG;
    if (!dropout_ok(p)) return QFP4_ERR_ARG;
    if (n < 0 || n > (int64_t(1) << 38)) return QFP4_ERR_SHAPE;
    if (n > 0 && (!x || !out)) return QFP4_ERR_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(out) || !step_aligned(step))
        return QFP4_ERR_ALIGN;
    if (n == 0) return QFP4_OK;
    const DropParams d = drop_params(p, seed, step);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dt == QFP4_F32 ? launch_dropout<QFP4_F32>(x, residual, n, d, out, s)
                          : launch_dropout<QFP4_BF16>(x, residual, n, d, out, s);
}

extern "C" size_t qfp4_epilogue_backward_workspace_bytes(int64_t M, int64_t N)
{
    if (M <= 0 || N <= 0 || M > INT32_MAX / 2 || N > INT32_MAX / 2) return 0;
    return sizeof(float) * epilogue_chunks(M, N) * N;
}

extern "C" int qfp4_epilogue_backward(const void *dY, const void *Z, qfp4_dtype dt, int64_t M, int64_t N, qfp4_act act,
                                      double dropout_p, uint64_t seed, const uint64_t *step, void *dZ, float *dbias,
                                      void *workspace, size_t workspace_bytes, qfp4_stream_t stream)
{
    if (dt != QFP4_BF16 && dt != QFP4_F32) return QFP4_ERR_ARG;
    if (act < QFP4_ACT_NONE || act > QFP4_ACT_SILU || !dropout_ok(dropout_p)) return QFP4_ERR_ARG;
    if (M < 0 || N < 0 || M > INT32_MAX / 2 || N > INT32_MAX / 2) return QFP4_ERR_SHAPE;
    if (M * N > 0 && (!dY || !dZ || (act != QFP4_ACT_NONE && !Z))) return QFP4_ERR_ARG;
    if (!aligned16(dY) || !aligned16(Z) || !aligned16(dZ) || !aligned16(dbias) || !aligned16(workspace) ||
        !step_aligned(step))
        return QFP4_ERR_ALIGN;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M * N == 0) {
        if (dbias && N > 0 && cudaMemsetAsync(dbias, 0, N * sizeof(float), s) != cudaSuccess) return QFP4_ERR_CUDA;
        return QFP4_OK;
    }
    if (dbias && (!workspace || workspace_bytes < qfp4_epilogue_backward_workspace_bytes(M, N))) return QFP4_ERR_ARG;
    const int64_t chunks = epilogue_chunks(M, N), rows = (M + chunks - 1) / chunks;
    const int64_t used = (M + rows - 1) / rows;
    float *partial = dbias ? static_cast<float *>(workspace) : nullptr;
    const dim3 grid(static_cast<unsigned>((N + 255) / 256), static_cast<unsigned>(used));
    const DropParams d = drop_params(dropout_p, seed, step);
    if (dt == QFP4_F32) k_epilogue_backward<QFP4_F32><<<grid, 256, 0, s>>>(dY, Z, M, N, rows, act, d, dZ, partial);
    else k_epilogue_backward<QFP4_BF16><<<grid, 256, 0, s>>>(dY, Z, M, N, rows, act, d, dZ, partial);
    QFP4_LAUNCH_CHECK();
    return dbias ? column_sums(partial, used, N, dbias, nullptr, false, s) : QFP4_OK;
}
