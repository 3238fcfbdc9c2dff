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
    DropParams drop;
};

}  // namespace qfp4
