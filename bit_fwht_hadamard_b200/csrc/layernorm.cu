// layernorm.cu -- layer norm of the rows of an M x D matrix, and its backward
// pass with the gradients of weight and bias.
//
// y = (x - mean) rstd gamma + beta, rstd = 1 / sqrt(var + eps).  With
// xhat = (x - mean) rstd and g = dy gamma:
//   dx = rstd (g - mean_d(g) - xhat mean_d(g xhat)),
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy.
//
// Bound by memory: each call reads its matrices once and writes its result
// once.  A row lies in the registers of the group of threads that takes it
// (a warp, or a block of 64 to 1024), so the second pass of the variance (on x -
// mean, which keeps a large mean from cancelling) costs no second read: in
// vectors of 16 bytes where the rows start on 16 bytes; where they do not,
// element by element up to 4096 columns, beyond that in vectors aligned in memory
// (forward).  Longer rows are read again from the caches.
#include "vec.cuh"

namespace qfp4 {

template <int DT>
__host__ __device__ constexpr int ln_v()
{
    return DT == QFP4_F32 ? 4 : 8;
}

// ------------------------------------------------------------------ vectors at a row's ends
// A vector of elements i .. i + V - 1 of a matrix of n, columns c .. c + V - 1
// of a row of D: only the columns in [0, D) belong to the row; the others, a
// neighbouring row's, become zeros.  Only a vector past the matrix's end goes
// element by element.
template <int DT, int V>
__device__ __forceinline__ void ld_edge(Vec<DT, V> &v, const void *p, int64_t i, int64_t n, int c, int D)
{
    if (i + V <= n) {
        v.load(p, i);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool out = c + j < 0 || c + j >= D;
            if (DT == QFP4_F32) v.r[j % 4] = out ? 0u : v.r[j % 4];
            else if (out) v.r[j >> 1] &= j & 1 ? 0x0000FFFFu : 0xFFFF0000u;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v.r[k] = 0u;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (c + j >= 0 && c + j < D) v.load1(p, i, j);
}
template <int DT, int V>
__device__ __forceinline__ void st_edge(const Vec<DT, V> &v, void *p, int64_t i, int c, int D)
{
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (c + j >= 0 && c + j < D) v.store1(p, i, j);
}
template <int V>
__device__ __forceinline__ Fv<V> inside_row(const Fv<V> &f, int c, int D)
{
    float v[V];
    f.to(v);
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (c + j < 0 || c + j >= D) v[j] = 0.0f;
    return Fv<V>::of(v);
}
// Parameters of columns c .. c + V - 1 (0 outside the row), c any column with SHIFT.
template <int V, bool SHIFT>
__device__ __forceinline__ Fv<V> ld_columns(const void *p, int f32, int c, int D)
{
    if constexpr (!SHIFT) return ld_param<V>(p, f32, c);
    float v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = c + j >= 0 && c + j < D ? ld_as_float(p, f32, c + j) : 0.0f;
    return Fv<V>::of(v);
}

// ------------------------------------------------------------------ forward
// G threads take R rows at once, NV vectors of V elements of each.  The rows
// stay as they were loaded (unpacking them again for each of the three steps
// is cheap); R rows share the reads of gamma and beta, which for one row are
// as many bytes as the row itself and more, and the barriers.
//
// V = 1: rows that do not start on 16 bytes, element by element.  SHIFT: such
// rows, too long for that (a thread would hold too many elements, 4096 x 4098
// bf16 106 us against 38).  Vectors are then aligned in memory, not in the row:
// row m starts off = (m D) mod V elements into one, the same for rows V apart,
// which are the R rows that a group takes; the vectors that straddle a row's
// ends go element by element.
template <int DT, int V, int G, int NV, int R, bool SHIFT>
__global__ void __launch_bounds__(G == 32 ? 128 : G, V == 8 && R == 4 && (G == 128 || (G == 32 && NV == 4)) ? 5 : 0)
    k_layernorm(const void *x, int64_t M, int D, const void *gamma, const void *beta, int w32, float eps, void *y,
                float *mean_out, float *rstd_out)
{
    constexpr int STEP = SHIFT ? V : 1;
    __shared__ float red[2][R][G == 32 ? 1 : G / 32];
    pdl_wait();
    pdl_trigger();
    const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t gi = G == 32 ? blockIdx.x * 4ll + (threadIdx.x >> 5) : static_cast<int64_t>(blockIdx.x);
    const int64_t m = SHIFT ? gi / V * (V * R) + gi % V : gi * R;
    if (m >= M) return;                                       // a whole group
    const int off = SHIFT ? static_cast<int>(gi % V) * (D % V) % V : 0;
    const int nv = SHIFT ? (D + off + V - 1) / V : D / V;
    Vec<DT, V> raw[R][NV];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (t + k * G < nv && m + r * STEP < M) {
                const int c = (t + k * G) * V - off;
                const int64_t i = (m + r * STEP) * D + c;
                if (!SHIFT || (c >= 0 && c + V <= D)) raw[r][k].load(x, i);
                else if constexpr (SHIFT) ld_edge(raw[r][k], x, i, M * D, c, D);
            }
    const float inv = 1.0f / static_cast<float>(D);
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        Fv<V> s = Fv<V>::splat(0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (t + k * G < nv) s = s + raw[r][k].values();
        mean[r] = s.sum();
    }
    group_sums<G, R>(mean, red[0]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        mean[r] *= inv;
        const Fv<V> mean2 = Fv<V>::splat(mean[r]);
        Fv<V> s = Fv<V>::splat(0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (t + k * G < nv) {
                Fv<V> d = raw[r][k].values() - mean2;
                const int c = (t + k * G) * V - off;
                if constexpr (SHIFT)
                    if (c < 0 || c + V > D) d = inside_row(d, c, D);
                s = fma(d, d, s);
            }
        rstd[r] = s.sum();
    }
    group_sums<G, R>(rstd, red[1]);
#pragma unroll
    for (int r = 0; r < R; ++r) rstd[r] = 1.0f / sqrtf(fmaf(rstd[r], inv, eps));
#pragma unroll
    for (int k = 0; k < NV; ++k)
        if (t + k * G < nv) {
            const int c = (t + k * G) * V - off;
            const bool whole = !SHIFT || (c >= 0 && c + V <= D);
            const Fv<V> g = gamma ? ld_columns<V, SHIFT>(gamma, w32, c, D) : Fv<V>::splat(1.0f);
            const Fv<V> b = beta ? ld_columns<V, SHIFT>(beta, w32, c, D) : Fv<V>::splat(0.0f);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (m + r * STEP < M) {
                    const int64_t i = (m + r * STEP) * D + c;
                    raw[r][k].set(fma((raw[r][k].values() - Fv<V>::splat(mean[r])) * Fv<V>::splat(rstd[r]), g, b));
                    if (whole) raw[r][k].store(y, i);
                    else if constexpr (SHIFT) st_edge(raw[r][k], y, i, c, D);
                }
        }
    if (t == 0)
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (m + r * STEP < M) {
                if (mean_out) mean_out[m + r * STEP] = mean[r];
                if (rstd_out) rstd_out[m + r * STEP] = rstd[r];
            }
}

// Rows of any length: a block of 1024 a row, three reads of it.
template <int DT>
__global__ void __launch_bounds__(1024) k_layernorm_long(const void *x, int64_t M, int64_t D, const void *gamma,
                                                          const void *beta, int w32, float eps, void *y,
                                                          float *mean_out, float *rstd_out)
{
    __shared__ float red[2][32];
    pdl_wait();
    pdl_trigger();
    const float inv = 1.0f / static_cast<float>(D);
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const int64_t r = m * D;
        // four sums a thread: D / 4096 terms one after the other
        float s[4] = {};
        for (int64_t c = threadIdx.x; c < D; c += 4096)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + 1024 * j < D) s[j] += ld_as_float(x, DT == QFP4_F32, r + c + 1024 * j);
        const float mean = group_sum<1024>((s[0] + s[1]) + (s[2] + s[3]), red[0]) * inv;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = 0.0f;
        for (int64_t c = threadIdx.x; c < D; c += 4096)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + 1024 * j < D) {
                    const float t = ld_as_float(x, DT == QFP4_F32, r + c + 1024 * j) - mean;
                    s[j] = fmaf(t, t, s[j]);
                }
        const float rstd = 1.0f / sqrtf(group_sum<1024>((s[0] + s[1]) + (s[2] + s[3]), red[1]) * inv + eps);
        for (int64_t c = threadIdx.x; c < D; c += 1024) {
            float v = (ld_as_float(x, DT == QFP4_F32, r + c) - mean) * rstd;
            if (gamma) v *= ld_as_float(gamma, w32, c);
            if (beta) v += ld_as_float(beta, w32, c);
            Vec<DT, 1> o;
            o.set(&v);
            o.store(y, r + c);
        }
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[m] = mean;
            if (rstd_out) rstd_out[m] = rstd;
        }
    }
}

struct LnForward {
    const void *x;
    int64_t M, D;
    const void *gamma, *beta;
    int w32;
    float eps;
    void *y;
    float *mean, *rstd;
    cudaStream_t s;
};

template <int DT, int V, int G, int NV, int R, bool SHIFT>
static int launch_layernorm(const LnForward &a)
{
    const int64_t groups = SHIFT ? (a.M + V * R - 1) / (V * R) * V : (a.M + R - 1) / R;
    if (launch_pdl(k_layernorm<DT, V, G, NV, R, SHIFT>, dim3(static_cast<unsigned>(G == 32 ? (groups + 3) / 4 : groups)),
                   dim3(G == 32 ? 128 : G), 0, a.s, a.x, a.M, static_cast<int>(a.D), a.gamma, a.beta, a.w32, a.eps, a.y,
                   a.mean, a.rstd) != cudaSuccess) {
        (void)cudaGetLastError();
        return QFP4_ERR_CUDA;
    }
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

// The group of a row: a warp up to 128 vectors; else four vectors a thread,
// LN_ROWS rows at once, which keeps the most bytes in flight an SM (16384 x
// 4096 bf16: 44 us; one row at once 55, two 44; 256 threads and two vectors
// 50).  With so few rows that each has an SM to itself, as many threads as
// there are vectors: the row's own latency is then all there is.
constexpr int LN_ROWS = 4;
template <int DT>
static int layernorm_vectors(const LnForward &a)
{
    constexpr int V = ln_v<DT>();
    const int64_t nv = a.D / V;
    if (a.M <= 2 * SMS) {
        if (nv <= 32) return launch_layernorm<DT, V, 32, 1, 1, false>(a);
        if (nv <= 128) return launch_layernorm<DT, V, 128, 1, 1, false>(a);
        if (nv <= 512) return launch_layernorm<DT, V, 512, 1, 1, false>(a);
        if (nv <= 1024) return launch_layernorm<DT, V, 1024, 1, 1, false>(a);
        return launch_layernorm<DT, V, 1024, 4, 1, false>(a);
    }
    if (nv <= 32) return launch_layernorm<DT, V, 32, 1, LN_ROWS, false>(a);
    if (nv <= 64) return launch_layernorm<DT, V, 32, 2, LN_ROWS, false>(a);
    if (nv <= 128) return launch_layernorm<DT, V, 32, 4, LN_ROWS, false>(a);
    if (nv <= 256) return launch_layernorm<DT, V, 64, 4, LN_ROWS, false>(a);
    if (nv <= 512) return launch_layernorm<DT, V, 128, 4, LN_ROWS, false>(a);
    if (nv <= 1024) return launch_layernorm<DT, V, 256, 4, LN_ROWS, false>(a);
    if (nv <= 2048) return launch_layernorm<DT, V, 512, 4, LN_ROWS, false>(a);
    return launch_layernorm<DT, V, 1024, 4, 1, false>(a);
}

template <int DT>
static int layernorm_elements(const LnForward &a)
{
    if (a.M <= 2 * SMS) {
        if (a.D <= 1024) return launch_layernorm<DT, 1, 128, 8, 1, false>(a);
        return launch_layernorm<DT, 1, 1024, 4, 1, false>(a);
    }
    if (a.D <= 256) return launch_layernorm<DT, 1, 32, 8, 2, false>(a);
    if (a.D <= 1024) return launch_layernorm<DT, 1, 128, 8, 2, false>(a);
    if (a.D <= 2048) return launch_layernorm<DT, 1, 256, 8, 2, false>(a);
    return launch_layernorm<DT, 1, 512, 8, 2, false>(a);
}

template <int DT>
static int layernorm_forward(const LnForward &a)
{
    constexpr int V = ln_v<DT>();
    if (a.D % V == 0 && a.D / V <= 4096) return layernorm_vectors<DT>(a);
    if (a.D % V != 0 && a.D <= 4096) return layernorm_elements<DT>(a);
    const int64_t nv = (a.D + 2 * (V - 1)) / V;               // at most, whatever the row's offset
    if (a.D % V != 0 && nv <= 1024) return launch_layernorm<DT, V, 256, 4, LN_ROWS, true>(a);
    if (a.D % V != 0 && nv <= 2048) return launch_layernorm<DT, V, 512, 4, LN_ROWS, true>(a);
    const int grid = static_cast<int>(imin<int64_t>(a.M, 16 * num_sms()));
    if (launch_pdl(k_layernorm_long<DT>, dim3(grid), dim3(1024), 0, a.s, a.x, a.M, a.D, a.gamma, a.beta, a.w32, a.eps,
                   a.y, a.mean, a.rstd) != cudaSuccess) {
        (void)cudaGetLastError();
        return QFP4_ERR_CUDA;
    }
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

// ------------------------------------------------------------------ backward
// The column sums of a block's GR groups, one group after the other, added to
// the first's.  buf: G NV V floats.
template <int G, int NV, int GR, int V>
__device__ __forceinline__ void join_groups(Fv<V> *v, float *buf, int gi, int t)
{
#pragma unroll
    for (int from = 1; from < GR; ++from) {
        __syncthreads();
        if (gi == from) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float o[V];
                v[k].to(o);
#pragma unroll
                for (int j = 0; j < V; ++j) buf[(k * V + j) * G + t] = o[j];
            }
        }
        __syncthreads();
        if (gi == 0) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = buf[(k * V + j) * G + t];
                v[k] = v[k] + Fv<V>::of(o);
            }
        }
    }
}

// One pass: a group of G threads takes every groups-th row, NV vectors a
// thread; the next row's loads are issued before the row sums of the present
// one are joined.  A thread keeps the sums of dy xhat and dy of its own columns
// in registers over all its rows; at the end each block joins its GR groups'
// sums and writes them as one row of the partial sums.  V = 1: rows that do not
// start on 16 bytes, element by element.
template <int DT, int V, int G, int NV, int GR>
__global__ void __launch_bounds__(GR *G)
    k_layernorm_backward(const void *dy, const void *x, int64_t M, int D, const void *gamma, int w32,
                         const float *mean_in, const float *rstd_in, void *dx, float *partial)
{
    __shared__ float2 red[GR][2][G / 32];
    __shared__ float join[GR > 1 ? G * NV * V : 1];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x % G, gi = threadIdx.x / G;
    const int64_t groups = static_cast<int64_t>(gridDim.x) * GR;
    int64_t m = static_cast<int64_t>(gi) * gridDim.x + blockIdx.x;
    const int nv = D / V;
    const float inv = 1.0f / static_cast<float>(D);
    Fv<V> sg[NV], sb[NV], w[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        sg[k] = sb[k] = Fv<V>::splat(0.0f);
        w[k] = Fv<V>::splat(1.0f);
        if (gamma && t + k * G < nv) w[k] = ld_param<V>(gamma, w32, (t + k * G) * V);
    }
    Vec<DT, V> rd[NV], rx[NV];
    float mean = 0.0f, rstd = 0.0f;
    auto load = [&](int64_t row) {
        mean = mean_in[row];
        rstd = rstd_in[row];
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (t + k * G < nv) {
                const int64_t i = row * D + (t + k * G) * V;
                rd[k].load(dy, i);
                rx[k].load(x, i);
            }
    };
    if (m < M) load(m);
    for (int par = 0; m < M; m += groups, par ^= 1) {
        Fv<V> xh[NV], g[NV], s1 = Fv<V>::splat(0.0f), s2 = Fv<V>::splat(0.0f);
        const Fv<V> mean2 = Fv<V>::splat(mean), rstd2 = Fv<V>::splat(rstd);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (t + k * G < nv) {
                const Fv<V> d = rd[k].values();
                xh[k] = (rx[k].values() - mean2) * rstd2;
                sg[k] = fma(d, xh[k], sg[k]);
                sb[k] = sb[k] + d;
                g[k] = d * w[k];
                s1 = s1 + g[k];
                s2 = fma(g[k], xh[k], s2);
            }
        }
        if (m + groups < M) load(m + groups);
        if (!dx) continue;
        const float2 c = group_sum2<G>(s1.sum(), s2.sum(), red[gi][par], 1 + gi);
        const Fv<V> c1 = Fv<V>::splat(c.x * inv), c2 = Fv<V>::splat(c.y * inv);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (t + k * G < nv) {
                Vec<DT, V> o;
                o.set(rstd2 * (g[k] - fma(xh[k], c2, c1)));
                o.store(dx, m * D + (t + k * G) * V);
            }
    }
    if (!partial) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        Fv<V> *v = half ? sb : sg;
        join_groups<G, NV, GR, V>(v, join, gi, t);
        if (gi == 0) {
            float *dst = partial + (half * static_cast<int64_t>(gridDim.x) + blockIdx.x) * D;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (t + k * G < nv) {
                    float o[V];
                    v[k].to(o);
#pragma unroll
                    for (int j = 0; j < V; ++j) dst[(t + k * G) * V + j] = o[j];
                }
        }
    }
}

// Aligned rows of 65 to 2048 vectors (bf16 D in (512, 16384], binary32 D in
// (256, 8192]): the same pass with the rows of dy and x brought into shared
// memory by bulk copies, `stages` rows ahead, so that no register waits for
// memory, and gamma beside them (in L1 it gave way to dx: 8192 x 4096 bf16 52 us
// against 49, 31 from memory alone; binary32 79 against 71).  Bound by the latency
// of a row: shared memory, two sums over the group, 24 instructions an element
// (fetching the next row's values before those sums: 51 us).  One block an SM of GR groups of G threads, each group with rows, a
// ring and a named barrier of its own; a thread holds NV vectors' columns.
// The groups' sums are joined at the end, so there are no more partial rows
// than SMs.  KEEP: xhat and g stay in registers between the row sums and dx;
// else (1024 threads, 64 registers) they are formed again from shared memory.
template <int DT, int G, int NV, int GR, bool KEEP, bool GSM>
__global__ void __launch_bounds__(GR *G, 1)
    k_layernorm_backward_ring(const void *dy, const void *x, int64_t M, int D, const void *gamma, int w32,
                              const float *mean_in, const float *rstd_in, void *dx, float *partial, int stages)
{
    constexpr int V = ln_v<DT>(), ESZ = 16 / V, MAX_STAGES = 8;
    extern __shared__ __align__(128) uint8_t ln_smem[];
    __shared__ __align__(8) uint64_t full_sh[GR][MAX_STAGES];
    __shared__ float2 red_sh[GR][2][G / 32];
    const int t = threadIdx.x % G, gi = threadIdx.x / G, nv = D / V;
    const int row_bytes = D * ESZ;
    uint64_t *full = full_sh[gi];
    uint8_t *ring = ln_smem + static_cast<size_t>(gi) * stages * 2 * row_bytes;
    if (t == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();
    // gamma as binary32 behind the rings, read again for every row
    float *gsm = reinterpret_cast<float *>(ln_smem + static_cast<size_t>(GR) * stages * 2 * row_bytes);
    if constexpr (GSM)
        for (int c = threadIdx.x * V; c < D; c += GR * G * V) {
            float w[V];
            if (gamma) ld_param<V>(gamma, w32, c, w);
#pragma unroll
            for (int j = 0; j < V; j += 4)
                *reinterpret_cast<float4 *>(gsm + c + j) =
                    gamma ? make_float4(w[j], w[j + 1], w[j + 2], w[j + 3]) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
        }
    __syncthreads();
    const float inv = 1.0f / static_cast<float>(D);
    const int64_t groups = static_cast<int64_t>(gridDim.x) * GR, m0 = blockIdx.x * static_cast<int64_t>(GR) + gi;
    // a row into stage s
    auto issue = [&](int64_t row, int s) {
        if (row >= M) return;
        mbar_arrive_expect_tx(&full[s], 2 * row_bytes);
        bulk_g2s(ring + static_cast<size_t>(2 * s) * row_bytes, static_cast<const char *>(dy) + row * row_bytes, row_bytes,
                 &full[s]);
        bulk_g2s(ring + static_cast<size_t>(2 * s + 1) * row_bytes, static_cast<const char *>(x) + row * row_bytes, row_bytes,
                 &full[s]);
    };
    if (t == 0)
        for (int i = 0; i < stages - 1; ++i) issue(m0 + i * groups, i);
    Fv<V> sg[NV], sb[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) sg[k] = sb[k] = Fv<V>::splat(0.0f);
    float mean_next = 0.0f, rstd_next = 0.0f;
    if (m0 < M) {
        mean_next = mean_in[m0];
        rstd_next = rstd_in[m0];
    }
    bool ok = true;
    int s = 0, last = stages - 1;                             // this row's stage, and the row's before it
    uint32_t phase = 0, par = 0;
    for (int64_t m = m0; m < M; m += groups) {
        const float mean = mean_next, rstd = rstd_next;
        if (m + groups < M) {
            mean_next = mean_in[m + groups];
            rstd_next = rstd_in[m + groups];
        }
        // after a wait that gave up (the error is recorded) the rows go on
        // without waiting, so that every thread still meets the barriers
        ok = ok && mbar_wait(&full[s], phase);
        const uint8_t *pd = ring + static_cast<size_t>(2 * s) * row_bytes, *px = pd + row_bytes;
        Fv<V> xh[KEEP ? NV : 1], g[KEEP ? NV : 1], s1 = Fv<V>::splat(0.0f), s2 = Fv<V>::splat(0.0f);
        const Fv<V> mean2 = Fv<V>::splat(mean), rstd2 = Fv<V>::splat(rstd);
        auto row_terms = [&](int c, Fv<V> &d, Fv<V> &h, Fv<V> &w) {
            Vec<DT, V> a, b;
            a.load(pd, c);
            b.load(px, c);
            d = a.values();
            h = (b.values() - mean2) * rstd2;
            if constexpr (GSM) {
                float u[V];
#pragma unroll
                for (int j = 0; j < V; j += 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(gsm + c + j);
                    u[j] = q.x;
                    u[j + 1] = q.y;
                    u[j + 2] = q.z;
                    u[j + 3] = q.w;
                }
                w = d * Fv<V>::of(u);
            } else
                w = gamma ? d * ld_param<V>(gamma, w32, c) : d;
        };
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (t + k * G < nv) {
                Fv<V> d, &h = xh[KEEP ? k : 0], &w = g[KEEP ? k : 0];
                row_terms((t + k * G) * V, d, h, w);
                sg[k] = fma(d, h, sg[k]);
                sb[k] = sb[k] + d;
                s1 = s1 + w;
                s2 = fma(w, h, s2);
            }
        // this thread's reads of the stages so far come before the next bulk copy
        fence_proxy_async();
        const float2 c = group_sum2<G>(s1.sum(), s2.sum(), red_sh[gi][par], 1 + gi);
        // every thread of the group is done with the row before this one,
        // whose stage takes the row stages - 1 ahead
        if (t == 0) issue(m + (stages - 1) * groups, last);
        last = s;
        par ^= 1u;
        if (++s == stages) {
            s = 0;
            phase ^= 1u;
        }
        if (!dx) continue;
        const Fv<V> c1 = Fv<V>::splat(c.x * inv), c2 = Fv<V>::splat(c.y * inv);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (t + k * G < nv) {
                Fv<V> d, &h = xh[KEEP ? k : 0], &w = g[KEEP ? k : 0];
                if constexpr (!KEEP) row_terms((t + k * G) * V, d, h, w);
                Vec<DT, V> o;
                o.set(rstd2 * (w - fma(h, c2, c1)));
                o.store(dx, m * D + static_cast<int64_t>(t + k * G) * V);
            }
    }
    if (!ok) settle_ns(kSettleNs);                            // copies already issued may still be landing
    __syncthreads();
    if (!partial) return;
    // (no copy is under way now: the ring's memory is free)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        Fv<V> *v = half ? sb : sg;
        join_groups<G, NV, GR, V>(v, reinterpret_cast<float *>(ln_smem), gi, t);
        if (gi == 0) {
            float *dst = partial + (half * static_cast<int64_t>(gridDim.x) + blockIdx.x) * D;
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (t + k * G < nv) {
                    float o[V];
                    v[k].to(o);
#pragma unroll
                    for (int j = 0; j < V; j += 4)
                        *reinterpret_cast<float4 *>(dst + (t + k * G) * V + j) =
                            make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
        }
    }
}

// Rows too long for that: the column sums and dx in a kernel each.
template <int DT, int V>
__global__ void __launch_bounds__(1024) k_layernorm_dx_long(const void *dy, const void *x, int64_t M, int64_t D,
                                                             const void *gamma, int w32, const float *mean_in,
                                                             const float *rstd_in, void *dx)
{
    __shared__ float2 red[2][32];
    pdl_wait();
    pdl_trigger();
    const float inv = 1.0f / static_cast<float>(D);
    int par = 0;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x, par ^= 1) {
        const int64_t r = m * D;
        const Fv<V> mean = Fv<V>::splat(mean_in[m]), rstd = Fv<V>::splat(rstd_in[m]);
        auto terms = [&](int64_t c, Fv<V> &g, Fv<V> &h) {
            Vec<DT, V> a, b;
            a.load(dy, r + c);
            b.load(x, r + c);
            g = a.values();
            if (gamma) g = g * ld_param<V>(gamma, w32, c);
            h = (b.values() - mean) * rstd;
        };
        Fv<V> s1[2], s2[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) s1[j] = s2[j] = Fv<V>::splat(0.0f);
        for (int64_t c = threadIdx.x * V; c < D; c += 2048 * V)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (c + 1024 * V * j < D) {
                    Fv<V> g, h;
                    terms(c + 1024 * V * j, g, h);
                    s1[j] = s1[j] + g;
                    s2[j] = fma(g, h, s2[j]);
                }
        const float2 t = group_sum2<1024>((s1[0] + s1[1]).sum(), (s2[0] + s2[1]).sum(), red[par], 1);
        const Fv<V> c1 = Fv<V>::splat(t.x * inv), c2 = Fv<V>::splat(t.y * inv);
        for (int64_t c = threadIdx.x * V; c < D; c += 1024 * V) {
            Fv<V> g, h;
            terms(c, g, h);
            Vec<DT, V> o;
            o.set(rstd * (g - fma(h, c2, c1)));
            o.store(dx, r + c);
        }
    }
}

// Column sums of a chunk of rows: partial[0][chunk][D] of dy xhat,
// partial[1][chunk][D] of dy.
template <int DT>
__global__ void __launch_bounds__(256) k_layernorm_dw_long(const void *dy, const void *x, int64_t M, int64_t D,
                                                            int64_t rows, const float *mean, const float *rstd,
                                                            float *partial)
{
    pdl_wait();
    pdl_trigger();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= D) return;
    const int64_t m0 = blockIdx.y * rows, m1 = imin(M, m0 + rows);
    float sg = 0.0f, sb = 0.0f;
#pragma unroll 4
    for (int64_t m = m0; m < m1; ++m) {
        const float d = ld_as_float(dy, DT == QFP4_F32, m * D + c);
        sg = fmaf(d, (ld_as_float(x, DT == QFP4_F32, m * D + c) - mean[m]) * rstd[m], sg);
        sb += d;
    }
    partial[blockIdx.y * D + c] = sg;
    partial[(static_cast<int64_t>(gridDim.y) + blockIdx.y) * D + c] = sb;
}

// How the backward pass runs: threads a row G and vectors a thread NV of the
// one-pass kernels (G = 0: the kernels for long rows), `stages` of the ring
// (0: rows in registers), and the rows of partial sums that it writes.
struct LnPlan {
    int V, G, NV, GR, stages;
    bool gamma_sm;                                            // gamma too in shared memory: it fits beside three stages
    int64_t parts, rows;
};
constexpr int LNB_SMEM = 200 * 1024;                       // leaves L1 and the next kernel some

static LnPlan layernorm_backward_plan(int64_t M, int64_t D, bool f32)
{
    LnPlan p{};
    const int vec = f32 ? 4 : 8;
    p.V = D % vec ? 1 : vec;
    const int64_t nv = D / p.V;
    p.GR = 1;
    if (p.V == 1) {
        // eight elements a thread, for loads enough in flight (16384 x 1001
        // bf16: 39 us; one element a thread 232)
        p.NV = 8;
        if (nv <= 256) p.G = 32, p.GR = 4;
        else if (nv <= 1024) p.G = 128;
        else if (nv <= 2048) p.G = 256;
        else if (nv <= 4096) p.G = 512;
        else if (nv <= 8192) p.G = 1024;
    } else if (nv <= 32)
        p.G = 32, p.NV = 1, p.GR = 4;
    else if (nv <= 64)
        p.G = 32, p.NV = 2, p.GR = 4;
    else if (nv <= 2048) {
        // 512 threads an SM (1024 for the longest rows): one row of D = 4096
        // bf16 takes an SM's share of the memory rate about 1000 cycles, a
        // group's two passes over it about 700
        p.NV = 2;
        if (nv <= 128) p.G = 64, p.GR = 8;
        else if (nv <= 256) p.G = 128, p.GR = 4;
        else if (nv <= 512) p.G = 256, p.GR = 2;
        else if (nv <= 1024) p.G = 512;
        else p.G = 1024;
        const int64_t stage = p.GR * 2 * D * (f32 ? 4 : 2);
        p.gamma_sm = p.G < 1024 || (LNB_SMEM - 4 * D) / stage >= 3;
        p.stages = static_cast<int>(imin<int64_t>(8, (LNB_SMEM - (p.gamma_sm ? 4 * D : 0)) / stage));
    }
    if (p.G) {
        // one block an SM, or blocks for 1024 threads an SM, but no more than
        // there are rows; several waves of them where a group would add more
        // than SUM_TERMS rows one after the other
        const int64_t wave = p.stages ? SMS : SMS * (1024 / (p.G * p.GR));
        const int64_t waves = (M + wave * p.GR * SUM_TERMS - 1) / (wave * p.GR * SUM_TERMS);
        p.parts = imin<int64_t>((M + p.GR - 1) / p.GR, wave * waves);
    } else {
        const int64_t cols = (D + 255) / 256;
        // chunks for eight blocks an SM, and as many times more as keep a
        // chunk's running sum to SUM_TERMS rows
        const int64_t wave = imax<int64_t>(1, imin<int64_t>(imin<int64_t>(M, 512), (8 * SMS + cols - 1) / cols));
        const int64_t want = wave * ((M + wave * SUM_TERMS - 1) / (wave * SUM_TERMS));
        p.rows = (M + want - 1) / want;
        p.parts = (M + p.rows - 1) / p.rows;
    }
    return p;
}

struct LnBackward {
    const void *dy, *x;
    int64_t M, D;
    const void *gamma;
    int w32;
    const float *mean, *rstd;
    void *dx;
    float *partial;
    cudaStream_t s;
};

template <int DT, int V, int G, int NV, int GR>
static int launch_layernorm_backward(const LnBackward &a, const LnPlan &p)
{
    if (launch_pdl(k_layernorm_backward<DT, V, G, NV, GR>, dim3(static_cast<unsigned>(p.parts)), dim3(GR * G), 0,
                   a.s, a.dy, a.x, a.M, static_cast<int>(a.D), a.gamma, a.w32, a.mean, a.rstd, a.dx,
                   a.partial) != cudaSuccess) {
        (void)cudaGetLastError();
        return QFP4_ERR_CUDA;
    }
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

template <int DT, int G, int NV, int GR, bool KEEP = true, bool GSM = true>
static int launch_layernorm_ring(const LnBackward &a, const LnPlan &p)
{
    const int smem = static_cast<int>(a.D) * (GR * p.stages * 2 * (DT == QFP4_F32 ? 4 : 2) + (GSM ? 4 : 0));
    if (ensure_dyn_smem<k_layernorm_backward_ring<DT, G, NV, GR, KEEP, GSM>>(LNB_SMEM) != QFP4_OK) return QFP4_ERR_CUDA;
    if (launch_pdl(k_layernorm_backward_ring<DT, G, NV, GR, KEEP, GSM>, dim3(static_cast<unsigned>(p.parts)), dim3(GR * G),
                   smem, a.s, a.dy, a.x, a.M, static_cast<int>(a.D), a.gamma, a.w32, a.mean, a.rstd, a.dx, a.partial,
                   p.stages) != cudaSuccess) {
        (void)cudaGetLastError();
        return QFP4_ERR_CUDA;
    }
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

template <int DT>
static int layernorm_backward_by_size(const LnBackward &a, const LnPlan &p)
{
    if (p.V == 1) {
        if (p.G == 32) return launch_layernorm_backward<DT, 1, 32, 8, 4>(a, p);
        if (p.G == 128) return launch_layernorm_backward<DT, 1, 128, 8, 1>(a, p);
        if (p.G == 256) return launch_layernorm_backward<DT, 1, 256, 8, 1>(a, p);
        if (p.G == 512) return launch_layernorm_backward<DT, 1, 512, 8, 1>(a, p);
        return launch_layernorm_backward<DT, 1, 1024, 8, 1>(a, p);
    }
    if (p.G == 32)
        return p.NV == 1 ? launch_layernorm_backward<DT, ln_v<DT>(), 32, 1, 4>(a, p)
                         : launch_layernorm_backward<DT, ln_v<DT>(), 32, 2, 4>(a, p);
    if (p.G == 64) return launch_layernorm_ring<DT, 64, 2, 8>(a, p);
    if (p.G == 128) return launch_layernorm_ring<DT, 128, 2, 4>(a, p);
    if (p.G == 256) return launch_layernorm_ring<DT, 256, 2, 2>(a, p);
    if (p.G == 512) return launch_layernorm_ring<DT, 512, 2, 1>(a, p);
    return p.gamma_sm ? launch_layernorm_ring<DT, 1024, 2, 1, false, true>(a, p)
                      : launch_layernorm_ring<DT, 1024, 2, 1, false, false>(a, p);
}

template <int DT>
static int layernorm_backward(const LnBackward &a, const LnPlan &p, float *dgamma, float *dbeta)
{
    if (p.G) {
        const int st = layernorm_backward_by_size<DT>(a, p);
        if (st != QFP4_OK || !a.partial) return st;
        return column_sums(a.partial, p.parts, a.D, static_cast<int>(a.D), 0, 1, dgamma, dbeta, true, a.s);
    }
    if (a.partial) {                                          // first: dx may overwrite dy
        const dim3 grid(static_cast<unsigned>((a.D + 255) / 256), static_cast<unsigned>(p.parts));
        if (launch_pdl(k_layernorm_dw_long<DT>, grid, dim3(256), 0, a.s, a.dy, a.x, a.M, a.D, p.rows, a.mean, a.rstd,
                       a.partial) != cudaSuccess) {
            (void)cudaGetLastError();
            return QFP4_ERR_CUDA;
        }
        QFP4_LAUNCH_CHECK();
        const int st = column_sums(a.partial, p.parts, a.D, static_cast<int>(a.D), 0, 1, dgamma, dbeta, true, a.s);
        if (st != QFP4_OK) return st;
    }
    if (!a.dx) return QFP4_OK;
    const int grid = static_cast<int>(imin<int64_t>(a.M, 16 * num_sms()));
    const bool vectors = a.D % ln_v<DT>() == 0;
    const cudaError_t e =
        vectors ? launch_pdl(k_layernorm_dx_long<DT, ln_v<DT>()>, dim3(grid), dim3(1024), 0, a.s, a.dy, a.x, a.M, a.D,
                             a.gamma, a.w32, a.mean, a.rstd, a.dx)
                : launch_pdl(k_layernorm_dx_long<DT, 1>, dim3(grid), dim3(1024), 0, a.s, a.dy, a.x, a.M, a.D, a.gamma,
                             a.w32, a.mean, a.rstd, a.dx);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return QFP4_ERR_CUDA;
    }
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
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
    const LnForward a{x, M, D, gamma, beta, wdt == QFP4_F32, eps, y, mean, rstd, s};
    return dt == QFP4_F32 ? layernorm_forward<QFP4_F32>(a) : layernorm_forward<QFP4_BF16>(a);
}

extern "C" size_t qfp4_layernorm_backward_workspace_bytes(int64_t M, int64_t D)
{
    if (M <= 0 || D <= 0 || layernorm_shape(M, D) != QFP4_OK) return 0;
    // of either type
    const int64_t parts = imax(layernorm_backward_plan(M, D, false).parts, layernorm_backward_plan(M, D, true).parts);
    return 2 * sizeof(float) * parts * D;
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
    const LnBackward a{dy, x, M, D, gamma, wdt == QFP4_F32, mean, rstd, dx,
                       dw ? static_cast<float *>(workspace) : nullptr, s};
    const LnPlan p = layernorm_backward_plan(M, D, dt == QFP4_F32);
    return dt == QFP4_F32 ? layernorm_backward<QFP4_F32>(a, p, dgamma, dbeta)
                          : layernorm_backward<QFP4_BF16>(a, p, dgamma, dbeta);
}
