// dropout.cu -- dropout from Philox words (no stored mask), optionally added
// to a residual, and the backward pass of the GEMM's epilogue (dropout,
// activation, bias).
#include "vec.cuh"

namespace qfp4 {

// ------------------------------------------------------------------ dropout
// A thread takes U vectors of 16 bytes, a block's width apart, with all their
// loads first.  Bound by memory and by the generator at once: its twenty wide
// multiplications a quad issue at a quarter of the rate, about 20 cycles an
// element and scheduler.  2^26 bf16 elements with a residual: 68 us alone, 77 in
// a sustained loop, 62 from memory alone (5.3 TB/s); one vector a thread 79.
constexpr int DROP_U = 4, DROP_BLOCKS = 4;
template <int DT, bool RES>
__global__ void __launch_bounds__(256, DROP_BLOCKS) k_dropout(const void *x, const void *res, int64_t n, DropParams d, void *out)
{
    constexpr int V = DT == QFP4_F32 ? 4 : 8;
    pdl_wait();
    pdl_trigger();
    const uint64_t step = drop_step(d);
    const int64_t vec0 = static_cast<int64_t>(blockIdx.x) * (256 * DROP_U) + threadIdx.x, nvec = n / V;
    Vec<DT, V> a[DROP_U], r[DROP_U];
#pragma unroll
    for (int u = 0; u < DROP_U; ++u)
        if (vec0 + 256 * u < nvec) {
            a[u].load(x, (vec0 + 256 * u) * V);
            if (RES) r[u].load(res, (vec0 + 256 * u) * V);
        }
#pragma unroll
    for (int u = 0; u < DROP_U; ++u) {
        const int64_t vec = vec0 + 256 * u, i = vec * V;
        float v[V], s[V];
        if (vec < nvec) {
            a[u].get(v);
            if (d.on) drop_values<V, true>(d, step, i, v);
            if (RES) {
                r[u].get(s);
#pragma unroll
                for (int t = 0; t < V; ++t) v[t] += s[t];
            }
            a[u].set(v);
            a[u].store(out, i);
        } else if (vec == nvec && i < n) {                  // the last, partial vector
            for (int t = 0; t < V; ++t) v[t] = i + t < n ? ld_as_float(x, DT == QFP4_F32, i + t) : 0.0f;
            if (d.on) drop_values<V, true>(d, step, i, v);
            for (int t = 0; t < V && i + t < n; ++t) {
                if (RES) v[t] += ld_as_float(res, DT == QFP4_F32, i + t);
                Vec<DT, 1> one;
                one.set(v + t);
                one.store(out, i + t);
            }
        }
    }
}

template <int DT>
static int launch_dropout(const void *x, const void *res, int64_t n, const DropParams &d, void *out, cudaStream_t s)
{
    const int64_t per = 256 * DROP_U * (DT == QFP4_F32 ? 4 : 8);
    const dim3 grid(static_cast<unsigned>((n + per - 1) / per));
    const cudaError_t e = res ? launch_pdl(k_dropout<DT, true>, grid, dim3(256), 0, s, x, res, n, d, out)
                              : launch_pdl(k_dropout<DT, false>, grid, dim3(256), 0, s, x, res, n, d, out);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return QFP4_ERR_CUDA;
    }
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

// ------------------------------------------------------------------ column sums of partial rows
// out[c] = sum over the rows r of partial[r][c] (in a fixed order): 32 columns
// x 32 row lanes a block.  A row of partial is `tiles` tiles of TW + V columns:
// slot V + j of tile t belongs to column t TW + j, j >= -V (V = 0: plain rows
// of TW = N columns).  blockIdx.y selects one of up to two outputs, whose
// partial rows follow one another.  Four rows a lane under way at once: all of
// 148 at once cost registers, and with them a second block an SM (layer norm
// backward 8192 x 4096 bf16 49 us, so 52).
__global__ void __launch_bounds__(1024) k_column_sums(const float *partial, int rows, int64_t N, int TW, int V, int tiles,
                                                       float *out0, float *out1)
{
    __shared__ float red[32][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float *out = blockIdx.y ? out1 : out0;
    if (!out) return;
    const int64_t stride = static_cast<int64_t>(tiles) * (TW + V);
    const float *src = partial + static_cast<int64_t>(blockIdx.y) * rows * stride;
    float s = 0.0f;
    if (c < N) {
        const int tile = static_cast<int>(c / TW), j = static_cast<int>(c - static_cast<int64_t>(tile) * TW);
        const float *p = src + static_cast<int64_t>(tile) * (TW + V) + V + j;
        const bool two = j >= TW - V && tile + 1 < tiles;       // the next tile's warps may hold this column too
#pragma unroll 4
        for (int r = w; r < rows; r += 32) {
            s += p[r * stride];
            if (two) s += p[r * stride + V];                     // slot j - TW + V of the next tile
        }
    }
    red[w][lane] = s;
    __syncthreads();
    const float t = warp_sum(red[lane][w]);                      // warp w: column w of the block
    const int64_t cw = static_cast<int64_t>(blockIdx.x) * 32 + w;
    if (lane == 0 && cw < N) out[cw] = t;
}

static int column_sums(const float *partial, int64_t rows, int64_t N, int TW, int V, int tiles, float *out0,
                       float *out1, bool two, cudaStream_t s)
{
    const dim3 grid(static_cast<unsigned>((N + 31) / 32), two ? 2 : 1);
    if (launch_pdl(k_column_sums, grid, dim3(1024), 0, s, partial, static_cast<int>(rows), N, TW, V, tiles, out0,
                   out1) != cudaSuccess) {
        (void)cudaGetLastError();
        return QFP4_ERR_CUDA;
    }
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

// ------------------------------------------------------------------ epilogue backward
// A warp takes one row at a time, eight rows apart, and a lane V = 16 bytes of
// columns, so that each lane keeps the sums of its own columns in registers.
// Vectors are aligned in memory, not in the row: a row of N columns starts
// off = (m N) mod V elements into a vector, the same for all rows that a warp
// takes (V divides 8), so its lanes' columns stay the same and any N runs on
// 16-byte accesses; the vectors that straddle a row's ends go element by
// element.  Reads dY and Z once, writes dZ once: bound by memory, with half of
// the issue slots taken by GELU's slope.  One wave of blocks, so that each
// keeps its columns' sums over many rows and few partial rows are left: 8192 x
// 11008 bf16 with GELU 98 us (83 from memory alone), some 20 more with several
// waves.
constexpr int EB_TILE = 32;                                   // vectors of a block's column tile
constexpr int EB_BLOCKS = 4, EB_WAVE = 4;

// Grid of the kernel: column tiles, row chunks (each a multiple of eight
// rows) for at most EB_WAVE blocks an SM, so that all run at once; several
// times as many where a lane would add more than SUM_TERMS rows one after the
// other (with terms of one sign the error of such a sum grows with its length:
// 16000 of them were 2e-4 off).
constexpr int SUM_TERMS = 2048;
struct EbGrid {
    int tiles, chunks;
    int64_t rows;
};
static EbGrid epilogue_backward_grid(int64_t M, int64_t N, int V)
{
    EbGrid g;
    const int64_t tw = EB_TILE * V;
    g.tiles = static_cast<int>((N % V ? N + V - 1 : N) / tw + ((N % V ? N + V - 1 : N) % tw != 0));
    const int64_t wave = imax<int64_t>(1, imin<int64_t>(EB_WAVE * SMS / g.tiles, 512));
    const int64_t waves = (M + wave * 8 * SUM_TERMS - 1) / (wave * 8 * SUM_TERMS);
    const int64_t want = imin<int64_t>(wave * waves, 65535 / wave * wave);      // blockIdx.y
    g.rows = ((M + want - 1) / want + 7) / 8 * 8;
    g.chunks = static_cast<int>((M + g.rows - 1) / g.rows);
    return g;
}

template <int DT, bool SHIFT>
__global__ void __launch_bounds__(256, EB_BLOCKS) k_epilogue_backward(const void *dy, const void *z, int64_t M,
                                                                       int64_t N, int64_t rows, int act, DropParams d,
                                                                       void *dz, float *partial)
{
    constexpr int V = DT == QFP4_F32 ? 4 : 8, TW = EB_TILE * V;
    __shared__ float red[8][TW + V];
    pdl_wait();
    pdl_trigger();
    const uint64_t step = drop_step(d);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int off = SHIFT ? static_cast<int>((w * (N & 7)) & (V - 1)) : 0;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * TW + lane * V - off;   // this lane's first column
    // without SHIFT a lane's columns are all in the row, or none
    const bool full = SHIFT ? c0 >= 0 && c0 + V <= N : c0 < N, some = SHIFT ? c0 + V > 0 && c0 < N : full;
    const int64_t m0 = blockIdx.y * rows, m1 = imin(M, m0 + rows);
    const bool use_z = act != QFP4_ACT_NONE;
    Fv<V> sums = Fv<V>::splat(0.0f);
    // rows m, m + 8, .. of this warp; the next one is loaded before the
    // present one is worked on
    Vec<DT, V> gn, an;
    auto load = [&](int64_t m) {
        const int64_t i = m * N + c0;
        if (full) {
            gn.load(dy, i);
            if (use_z) an.load(z, i);
        } else if constexpr (SHIFT) {
#pragma unroll
            for (int k = 0; k < 4; ++k) gn.r[k] = an.r[k] = 0u;
            if (some) {
#pragma unroll
                for (int t = 0; t < V; ++t)
                    if (c0 + t >= 0 && c0 + t < N) {
                        gn.load1(dy, i, t);
                        if (use_z) an.load1(z, i, t);
                    }
            }
        }
    };
    if (some && m0 + w < m1) load(m0 + w);
    if (some)
        for (int64_t m = m0 + w; m < m1; m += 8) {
            Vec<DT, V> g = gn;
            const Vec<DT, V> a = an;
            if (m + 8 < m1) load(m + 8);
            const int64_t i = m * N + c0;                       // a multiple of V
            float v[V], x[V];
            g.get(v);
            if (d.on) drop_values<V, true>(d, step, i, v);
            if (use_z) {
                a.get(x);
                act_backward<V>(v, x, act);
            }
            sums = sums + Fv<V>::of(v);                         // zero outside the row
            g.set(v);
            if (full) g.store(dz, i);
            else if constexpr (SHIFT) {
#pragma unroll
                for (int t = 0; t < V; ++t)
                    if (c0 + t >= 0 && c0 + t < N) g.store1(dz, i, t);
            }
        }
    if (!partial) return;
    // slot V + j of red: column blockIdx.x TW + j; a warp covers j = -off .. TW - off - 1
    for (int j = lane; j < V; j += 32) red[w][j] = red[w][TW + j] = 0.0f;
    __syncwarp();
    float sum[V];
    sums.to(sum);
#pragma unroll
    for (int t = 0; t < V; ++t) red[w][V + lane * V + t - off] = sum[t];
    __syncthreads();
    float *dst = partial + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * (TW + V);
    for (int j = threadIdx.x; j < TW + V; j += 256) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += red[k][j];
        dst[j] = s;
    }
}

template <int DT>
static int epilogue_backward(const void *dY, const void *Z, int64_t M, int64_t N, int act, const DropParams &d,
                             void *dZ, float *dbias, float *partial, cudaStream_t s)
{
    constexpr int V = DT == QFP4_F32 ? 4 : 8;
    const EbGrid g = epilogue_backward_grid(M, N, V);
    float *sums = dbias ? partial : nullptr;
    const dim3 grid(g.tiles, g.chunks);
    const cudaError_t e = N % V ? launch_pdl(k_epilogue_backward<DT, true>, grid, dim3(256), 0, s, dY, Z, M, N, g.rows,
                                             act, d, dZ, sums)
                                : launch_pdl(k_epilogue_backward<DT, false>, grid, dim3(256), 0, s, dY, Z, M, N, g.rows,
                                             act, d, dZ, sums);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return QFP4_ERR_CUDA;
    }
    QFP4_LAUNCH_CHECK();
    return dbias ? column_sums(partial, g.chunks, N, EB_TILE * V, V, g.tiles, dbias, nullptr, false, s) : QFP4_OK;
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
    if (!aligned16(x) || !aligned16(residual) || !aligned16(out) || !step_aligned(step)) return QFP4_ERR_ALIGN;
    if (n == 0) return QFP4_OK;
    const DropParams d = drop_params(p, seed, step);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dt == QFP4_F32 ? launch_dropout<QFP4_F32>(x, residual, n, d, out, s)
                          : launch_dropout<QFP4_BF16>(x, residual, n, d, out, s);
}

extern "C" size_t qfp4_epilogue_backward_workspace_bytes(int64_t M, int64_t N)
{
    if (M <= 0 || N <= 0 || M > INT32_MAX / 2 || N > INT32_MAX / 2) return 0;
    size_t most = 0;
    for (int V = 4; V <= 8; V += 4) {
        const EbGrid g = epilogue_backward_grid(M, N, V);
        most = imax(most, sizeof(float) * g.chunks * g.tiles * (EB_TILE * V + V));
    }
    return most;
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
    const DropParams d = drop_params(dropout_p, seed, step);
    float *partial = static_cast<float *>(workspace);
    return dt == QFP4_F32 ? epilogue_backward<QFP4_F32>(dY, Z, M, N, act, d, dZ, dbias, partial, s)
                          : epilogue_backward<QFP4_BF16>(dY, Z, M, N, act, d, dZ, dbias, partial, s);
}
