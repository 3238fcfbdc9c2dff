// epilogue.cuh -- device numerics of the operators around a linear layer:
// activations and their derivatives, and dropout from Philox4x32-10 words.
#pragma once

#include "qfp4_common.cuh"

namespace qfp4 {

// ------------------------------------------------------------------ dropout
// Element e stays iff word e mod 4 of Philox4x32-10, keyed on the 64-bit seed
// at counter (e / 4, 2^63 + step), is >= threshold = floor(p 2^32); it is then
// multiplied by scale = fl(1 / (1 - p)).  The stochastic rounding of the
// quantize calls uses counters (e / 4, 0), so bit 63 keeps the two sets of
// words apart under one seed.  The mask is never stored: the backward pass
// forms the same words again.
struct DropParams {
    uint64_t seed = 0;
    const uint64_t *step = nullptr;   // device counter (a captured graph's replays read its current value), or NULL: 0
    uint32_t threshold = 0;
    float scale = 1.0f;
    int on = 0;                        // 0: p == 0, nothing is drawn
};

inline bool dropout_ok(double p) { return p >= 0.0 && p < 1.0; }   // false for a NaN
inline bool step_aligned(const uint64_t *step) { return (reinterpret_cast<uintptr_t>(step) & 7u) == 0; }

// p has passed dropout_ok.
inline DropParams drop_params(double p, uint64_t seed, const uint64_t *step)
{
    DropParams d;
    d.seed = seed;
    d.step = step;
    d.threshold = static_cast<uint32_t>(p * 4294967296.0);
    d.scale = static_cast<float>(1.0 / (1.0 - p));
    d.on = p > 0.0;
    return d;
}

__device__ __forceinline__ uint64_t drop_step(const DropParams &d) { return d.on && d.step ? *d.step : 0ull; }

// The four words of elements 4q .. 4q + 3.
__device__ __forceinline__ uint4 drop_words4(const DropParams &d, uint64_t step, uint64_t q)
{
    uint32_t c0 = static_cast<uint32_t>(q), c1 = static_cast<uint32_t>(q >> 32);
    uint32_t c2 = static_cast<uint32_t>(step), c3 = static_cast<uint32_t>(step >> 32) | 0x80000000u;
    uint32_t k0 = static_cast<uint32_t>(d.seed), k1 = static_cast<uint32_t>(d.seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0, p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
        c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
        c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
        c1 = static_cast<uint32_t>(p1);
        c3 = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ float drop1(const DropParams &d, float v, uint32_t word)
{
    return word >= d.threshold ? __fmul_rn(v, d.scale) : 0.0f;
}

// ------------------------------------------------------------------ activations
// All in binary32 on the unrounded sum z.  A NaN stays a NaN in each of them.
__device__ __forceinline__ float act_forward(float z, int act)
{
    switch (act) {
    case QFP4_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case QFP4_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case QFP4_ACT_GELU_TANH: {
        // 1/2 (1 + tanh u) = 1 / (1 + e^-2u)
        const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
        return __fdividef(z, 1.0f + __expf(-u2));
    }
    case QFP4_ACT_SILU: return __fdividef(z, 1.0f + __expf(-z));
    default: return z;
    }
}

// Beyond |z| = 80 every slope is 0 or 1 to binary32; the clamp keeps z^2, z^3
// and the exponentials' products finite there.
__device__ __forceinline__ float act_slope(float z, int act)
{
    z = z > 80.0f ? 80.0f : z < -80.0f ? -80.0f : z;
    switch (act) {
    case QFP4_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case QFP4_ACT_GELU:
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * 0.39894228040143268f * __expf(-0.5f * z * z);
    case QFP4_ACT_GELU_TANH: {
        const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
        const float f = __fdividef(1.0f, 1.0f + __expf(-u2));
        return f + z * f * (1.0f - f) * (1.5957691216057308f * (1.0f + 0.134145f * z * z));
    }
    case QFP4_ACT_SILU: {
        const float f = __fdividef(1.0f, 1.0f + __expf(-z));
        return f * (1.0f + z * (1.0f - f));
    }
    default: return 1.0f;
    }
}

// ------------------------------------------------------------------ element access
__device__ __forceinline__ float ld_as_float(const void *p, int f32, int64_t i)
{
    return f32 ? static_cast<const float *>(p)[i]
               : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
}
__device__ __forceinline__ float2 ld2_as_float(const void *p, int f32, int64_t i)   // i even
{
    if (f32) return *reinterpret_cast<const float2 *>(static_cast<const float *>(p) + i);
    const uint32_t w = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p) + i);
    return make_float2(bf16lo(w), bf16hi(w));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

// ------------------------------------------------------------------ GEMM epilogue
struct EpParams {
    const void *bias;          // N values, or NULL
    const void *residual;      // M x N, or NULL
    void *preact;              // M x N of the output type, or NULL
    int bias_f32, residual_f32, act;
    int wide;                  // rows of out, preact and residual all start on 32 bytes
    DropParams drop;
};

// 32 bytes a thread: a row's thread fills whole sectors of its own.
__device__ __forceinline__ void ld_v8(const void *p, uint32_t *r)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}
__device__ __forceinline__ void st_v8(void *p, const uint32_t *r)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Sixteen consecutive values of one row, as loaded: binary32 in r[0 .. 15],
// bf16 pairs in r[0 .. 7].  nc < 16 (a multiple of 4): the row's last ones.
struct Row16 {
    uint32_t r[16];
};
__device__ __forceinline__ void row16_load(Row16 &v, const void *p, int f32, int64_t i, int nc, int wide)
{
    if (f32) {
        const float *s = static_cast<const float *>(p) + i;
        if (wide && nc == 16) {
            ld_v8(s, v.r);
            ld_v8(s + 8, v.r + 8);
        } else {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (4 * g < nc) *reinterpret_cast<uint4 *>(v.r + 4 * g) = *reinterpret_cast<const uint4 *>(s + 4 * g);
        }
    } else {
        const uint16_t *s = static_cast<const uint16_t *>(p) + i;
        if (wide && nc == 16) ld_v8(s, v.r);
        else {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (4 * g < nc) *reinterpret_cast<uint2 *>(v.r + 2 * g) = *reinterpret_cast<const uint2 *>(s + 4 * g);
        }
    }
}
__device__ __forceinline__ float row16_get(const Row16 &v, int f32, int t)
{
    if (f32) return __uint_as_float(v.r[t]);
    return t & 1 ? bf16hi(v.r[t >> 1]) : bf16lo(v.r[t >> 1]);
}
template <int OUT>
__device__ __forceinline__ void row16_store(void *p, int64_t i, const float *v, int nc, int wide)
{
    if (OUT == QFP4_F32) {
        float *d = static_cast<float *>(p) + i;
        if (wide && nc == 16) {
            st_v8(d, reinterpret_cast<const uint32_t *>(v));
            st_v8(d + 8, reinterpret_cast<const uint32_t *>(v + 8));
        } else {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (4 * g < nc)
                    *reinterpret_cast<float4 *>(d + 4 * g) = make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
        }
    } else {
        uint16_t *d = static_cast<uint16_t *>(p) + i;
        uint32_t w[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) w[t] = pack_bf16(v[2 * t], v[2 * t + 1]);
        if (wide && nc == 16) st_v8(d, w);
        else {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (4 * g < nc) *reinterpret_cast<uint2 *>(d + 4 * g) = make_uint2(w[2 * g], w[2 * g + 1]);
        }
    }
}

// Four bias values from column col on (the same for every row: the loads are
// broadcasts, and read-only, so they may be issued ahead of the stores).
__device__ __forceinline__ float4 bias4_load(const EpParams &ep, int col)
{
    if (ep.bias_f32) return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(ep.bias) + col));
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(ep.bias) + col));
    return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

template <int ACT>
__device__ __forceinline__ void act16(float *v)
{
#pragma unroll
    for (int t = 0; t < 16; ++t) v[t] = act_forward(v[t], ACT);
}

// The last step of qfp4_gemm_epilogue on the accumulators acc[0 .. 15] of one
// row's columns col .. col + 15 (the first nc of them exist; nc and col are
// multiples of 4), i = row * N + col: z = alpha acc + bias, the optional copy
// of z, the activation, dropout, the residual, one rounding to the output
// type.  The residual's loads are issued first and used last.
template <int OUT>
__device__ __forceinline__ void ep_chunk16(const EpParams &ep, void *out, int64_t i, int col, int nc, float alpha,
                                           uint64_t step, const uint32_t *acc)
{
    Row16 res;
    if (ep.residual) row16_load(res, ep.residual, ep.residual_f32, i, nc, ep.wide);
    float v[16];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (ep.bias && 4 * g < nc) b = bias4_load(ep, col + 4 * g);
        v[4 * g] = fmaf(__uint_as_float(acc[4 * g]), alpha, b.x);
        v[4 * g + 1] = fmaf(__uint_as_float(acc[4 * g + 1]), alpha, b.y);
        v[4 * g + 2] = fmaf(__uint_as_float(acc[4 * g + 2]), alpha, b.z);
        v[4 * g + 3] = fmaf(__uint_as_float(acc[4 * g + 3]), alpha, b.w);
    }
    if (ep.preact) row16_store<OUT>(ep.preact, i, v, nc, ep.wide);
    switch (ep.act) {                                   // the same for every thread
    case QFP4_ACT_RELU: act16<QFP4_ACT_RELU>(v); break;
    case QFP4_ACT_GELU: act16<QFP4_ACT_GELU>(v); break;
    case QFP4_ACT_GELU_TANH: act16<QFP4_ACT_GELU_TANH>(v); break;
    case QFP4_ACT_SILU: act16<QFP4_ACT_SILU>(v); break;
    default: break;
    }
    if (ep.drop.on) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const uint4 w = drop_words4(ep.drop, step, (static_cast<uint64_t>(i) >> 2) + g);   // i % 4 == 0
            v[4 * g] = drop1(ep.drop, v[4 * g], w.x);
            v[4 * g + 1] = drop1(ep.drop, v[4 * g + 1], w.y);
            v[4 * g + 2] = drop1(ep.drop, v[4 * g + 2], w.z);
            v[4 * g + 3] = drop1(ep.drop, v[4 * g + 3], w.w);
        }
    }
    if (ep.residual) {
        if (ep.residual_f32) {
#pragma unroll
            for (int t = 0; t < 16; ++t) v[t] += row16_get(res, 1, t);
        } else {
#pragma unroll
            for (int t = 0; t < 16; ++t) v[t] += row16_get(res, 0, t);
        }
    }
    row16_store<OUT>(out, i, v, nc, ep.wide);
}

// Asks L2 for the residual of one thread's 128 columns before the
// accumulators are there.  row < M only.
__device__ __forceinline__ void ep_prefetch128(const EpParams &ep, int N, int row, int col0)
{
    const int esz = ep.residual_f32 ? 4 : 2;
    const char *p = static_cast<const char *>(ep.residual) + (static_cast<int64_t>(row) * N + col0) * esz;
    const int bytes = imin(128, N - col0) * esz;
    for (int o = 0; o < bytes; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + o));
}

// One thread's row: the epilogue of the accumulators r[0 .. 127] of columns
// col0 .. col0 + 127, sixteen at a time.  row < M only.
template <int OUT>
__device__ __forceinline__ void ep_row128(const EpParams &ep, void *out, int N, int row, int col0, float alpha,
                                          uint64_t step, const uint32_t *r)
{
    const int64_t i0 = static_cast<int64_t>(row) * N + col0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int col = col0 + 16 * c, nc = imin(16, N - col);
        if (nc > 0) ep_chunk16<OUT>(ep, out, i0 + 16 * c, col, nc, alpha, step, r + 16 * c);
    }
}

}  // namespace qfp4
