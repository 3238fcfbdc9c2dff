// epilogue.cuh -- device numerics of the operators around a linear layer:
// activations and their derivatives, and dropout from Philox4x32-10 words.
#pragma once

#include "qfp4_common.cuh"

namespace qfp4 {

// SMs that grids and workspaces are sized for.  A constant, where num_sms() asks
// the device: a workspace query needs no device, and its call must agree with it.
constexpr int SMS = 148;

// ------------------------------------------------------------------ dropout
// Element e stays iff word e mod 4 of Philox4x32-10, keyed on the 64-bit seed
// at counter (e / 4, 2^63 + step), is >= threshold = floor(p 2^32); it is then
// multiplied by scale = fl(1 / (1 - p)).  The stochastic rounding of the
// quantize calls uses counters (e / 4, 0), so bit 63 keeps the two sets of
// words apart under one seed.  The mask is never stored: the backward pass
// forms the same words again.
struct DropParams {
    uint32_t k0[10] = {}, k1[10] = {};   // the seed's key of each round (read as constants by the rounds)
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
    for (int r = 0; r < 10; ++r) {
        d.k0[r] = static_cast<uint32_t>(seed) + static_cast<uint32_t>(r) * 0x9E3779B9u;
        d.k1[r] = static_cast<uint32_t>(seed >> 32) + static_cast<uint32_t>(r) * 0xBB67AE85u;
    }
    d.step = step;
    d.threshold = static_cast<uint32_t>(p * 4294967296.0);
    d.scale = static_cast<float>(1.0 / (1.0 - p));
    d.on = p > 0.0;
    return d;
}

__device__ __forceinline__ uint64_t drop_step(const DropParams &d) { return d.on && d.step ? *d.step : 0ull; }

// The four words of elements 4q .. 4q + 3, q = hi 2^32 + lo.  Where a thread
// takes several quads under one hi, their first product and (from hi and the
// step alone) one of the second round's are the same, which the compiler sees.
__device__ __forceinline__ uint4 drop_words4(const DropParams &d, uint64_t step, uint32_t lo, uint32_t hi)
{
    uint32_t c0 = lo, c1 = hi;
    uint32_t c2 = static_cast<uint32_t>(step), c3 = static_cast<uint32_t>(step >> 32) | 0x80000000u;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0, p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
        c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ d.k0[r];
        c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ d.k1[r];
        c1 = static_cast<uint32_t>(p1);
        c3 = static_cast<uint32_t>(p0);
    }
    return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ float drop1(const DropParams &d, float v, uint32_t word)
{
    return word >= d.threshold ? __fmul_rn(v, d.scale) : 0.0f;
}

// Dropout of V values whose first one is element i, in place (i and V are
// multiples of 4).  ALIGNED: i is a multiple of V too, so that the quads
// share the counter's high word.
template <int V, bool ALIGNED>
__device__ __forceinline__ void drop_values(const DropParams &d, uint64_t step, int64_t i, float *v)
{
    const uint64_t q = static_cast<uint64_t>(i) >> 2;
#pragma unroll
    for (int g = 0; g < V / 4; ++g) {
        const uint4 w = drop_words4(d, step, static_cast<uint32_t>(q) + g,
                                    static_cast<uint32_t>((ALIGNED ? q : q + g) >> 32));
        v[4 * g] = drop1(d, v[4 * g], w.x);
        v[4 * g + 1] = drop1(d, v[4 * g + 1], w.y);
        v[4 * g + 2] = drop1(d, v[4 * g + 2], w.z);
        v[4 * g + 3] = drop1(d, v[4 * g + 3], w.w);
    }
}

// ------------------------------------------------------------------ activations
// All in binary32 on the unrounded sum z.  A NaN stays a NaN in each of them.
//
// GELU on pairs of values, from the normal distribution function of the
// negative half line, so that nothing cancels there: with a = |z| and
// E = e^(-a^2/2),
//   Phi(-a) = E m(a),   GELU(z) = max(z, 0) - a Phi(-a).
// m (Mills' ratio over sqrt(2 pi)) falls like 1 / a: a quotient of polynomials
// of degree 3 and 4 keeps its digits on the whole half line.  All their terms
// are positive; they were fitted on [0, 13.4] by least squares of the relative
// error over 1.5 + 0.6 a^2, the weights raised towards the largest (u = 2^-24:
// within (1.1 + 0.43 a^2) u; a rounding a step, the coefficients', the reciprocal
// and the product at most 12 u more).  E is within (4 + 1.05 a^2) u (its rounded
// exponent), so GELU(z) for z < 0 is within (19 + 1.5 z^2) u of itself, down to
// 2^-126 where E ends; on a dense grid it was within (12 + 1.25 z^2) u.  Two
// special-function instructions a value, nine packed multiply-adds a pair.  A
// polynomial in a of degree 10, weighted by E, took as long (8192 x 11008 x 4096
// NVFP4 with bias, GELU and z kept 212 us, this one 210) but was accurate in
// absolute terms only: 23 % off at -5, eleven times too large at -6.  1 / (1 +
// 0.34 a) times a polynomial of degree 8 in it is as accurate as the quotient,
// with a longer chain (backward pass 102 us, the quotient 98).  A NaN stays one.
__device__ __forceinline__ float abs_upto(float x, float most)
{
    float r;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %1;\n\tmin.NaN.f32 %0, t, %2;\n\t}" : "=f"(r) : "f"(x), "f"(most));
    return r;
}
__device__ __forceinline__ float max0_nan(float x)
{
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// E of a pair
__device__ __forceinline__ uint64_t gauss2(uint64_t a)
{
    float x, y;
    f2unpack(f2mul(f2mul(a, f2pack(-0.721347520f, -0.721347520f)), a), x, y);   // -a^2 / 2 log2 e
    return f2pack(exp2_fast(x), exp2_fast(y));
}
// m of a pair, a >= 0
__device__ __forceinline__ uint64_t mills2(uint64_t a)
{
    uint64_t n = f2pack(0.0144826053f, 0.0144826053f);
    n = f2fma(n, a, f2pack(0.108570509f, 0.108570509f));
    n = f2fma(n, a, f2pack(0.342697442f, 0.342697442f));
    n = f2fma(n, a, f2pack(0.49999997f, 0.49999997f));
    uint64_t d = f2pack(0.0363141261f, 0.0363141261f);
    d = f2fma(d, a, f2pack(0.271760285f, 0.271760285f));
    d = f2fma(d, a, f2pack(0.900663376f, 0.900663376f));
    d = f2fma(d, a, f2pack(1.48327541f, 1.48327541f));
    d = f2fma(d, a, f2pack(1.0f, 1.0f));
    float x, y;
    f2unpack(d, x, y);
    return f2mul(n, f2pack(rcp_fast(x), rcp_fast(y)));
}
__device__ __forceinline__ uint64_t gelu2(float z0, float z1)
{
    const uint64_t a = f2pack(abs_upto(z0, 16.0f), abs_upto(z1, 16.0f));
    const uint64_t na = f2mul(a, f2pack(-1.0f, -1.0f));
    return f2fma(f2mul(na, gauss2(a)), mills2(a), f2pack(max0_nan(z0), max0_nan(z1)));
}
// The slope from the same m: Phi(-a) - a phi(a) = E t, t = m - a / sqrt(2 pi),
// is the slope at -a, and 1 - E t the one at a, so that the negative side
// keeps its digits here too (E t within (19 + 1.5 a^2) u of its two terms' sum;
// a polynomial for t weighted by E, and 1/2 + sign(z) (1/2 - E t), was within
// 1.2e-7 whatever the slope, and took as long).
__device__ __forceinline__ uint64_t gelu_slope2(float z0, float z1)
{
    const uint64_t a = f2pack(abs_upto(z0, 16.0f), abs_upto(z1, 16.0f));
    const uint64_t t = f2fma(a, f2pack(-0.39894228f, -0.39894228f), mills2(a));
    const uint64_t up = f2pack(z0 >= 0.0f ? 1.0f : 0.0f, z1 >= 0.0f ? 1.0f : 0.0f);
    const uint64_t sign = f2fma(up, f2pack(-2.0f, -2.0f), f2pack(1.0f, 1.0f));
    return f2fma(f2mul(gauss2(a), t), sign, up);
}

// x within [-most, most]; a NaN stays one.
__device__ __forceinline__ float clamp_nan(float x, float most)
{
    float r;
    asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, %2;\n\tmax.NaN.f32 %0, t, %3;\n\t}"
        : "=f"(r)
        : "f"(x), "f"(most), "f"(-most));
    return r;
}

// The sigmoid f of a pair of x and g = 1 - f, from E = e^-|x| <= 1 and r = 1 /
// (1 + E): r and E r are the two, so neither loses digits where it is small
// (1 / (1 + e^-x) from the fast exponential was 95 u off at x = -80, and 1 - f had
// no digit left beyond x = 17), and no divisor is ever large.
struct Sigmoid2 {
    uint64_t E, r;

    __device__ __forceinline__ void finish()
    {
        float x, y;
        f2unpack(f2add(E, f2pack(1.0f, 1.0f)), x, y);
        r = f2pack(rcp_fast(x), rcp_fast(y));
    }
    // f of the pair whose signs are z0's and z1's
    __device__ __forceinline__ uint64_t f(float z0, float z1) const
    {
        float x, y;
        f2unpack(E, x, y);
        return f2mul(f2pack(z0 >= 0.0f ? 1.0f : x, z1 >= 0.0f ? 1.0f : y), r);
    }
    // z f g
    __device__ __forceinline__ uint64_t zfg(uint64_t z) const { return f2mul(f2mul(z, r), f2mul(E, r)); }
};
// E from both words of |x| log2 e: the rounding of the first, up to 2^-18 of E,
// comes back as 1 - ln 2 times it.
__device__ __forceinline__ Sigmoid2 sigmoid2(float x0, float x1)
{
    const uint64_t a = f2pack(abs_upto(x0, 128.0f), abs_upto(x1, 128.0f));
    const uint64_t n = f2mul(a, f2pack(-1.44269502f, -1.44269502f));
    const uint64_t over =
        f2fma(a, f2pack(1.92596303e-08f, 1.92596303e-08f), f2fma(a, f2pack(1.44269502f, 1.44269502f), n));
    float x, y;
    f2unpack(n, x, y);
    Sigmoid2 s;
    s.E = f2mul(f2pack(exp2_fast(x), exp2_fast(y)),
                f2fma(over, f2pack(-0.693147182f, -0.693147182f), f2pack(1.0f, 1.0f)));
    s.finish();
    return s;
}
// GELU's tanh form: 1/2 (1 + tanh t) is the sigmoid of x = 2 t = 2 sqrt(2/pi) (z
// + 0.044715 z^3), here times log2 e.  (x is rounded already: no second word.)
__device__ __forceinline__ Sigmoid2 sigmoid_tanh2(float z0, float z1)
{
    const uint64_t z = f2pack(z0, z1);
    float x, y;
    f2unpack(f2mul(z, f2fma(f2mul(z, f2pack(0.102943234f, 0.102943234f)), z, f2pack(2.30220819f, 2.30220819f))), x, y);
    Sigmoid2 s;
    s.E = f2pack(exp2_fast(-fabsf(x)), exp2_fast(-fabsf(y)));
    s.finish();
    return s;
}

// In place on an even number of values; act is the same for every thread.
template <int N>
__device__ __forceinline__ void act_forward(float *v, int act)
{
    switch (act) {
    case QFP4_ACT_RELU:
#pragma unroll
        for (int t = 0; t < N; ++t) v[t] = v[t] < 0.0f ? 0.0f : v[t];
        break;
    case QFP4_ACT_GELU:
#pragma unroll
        for (int t = 0; t < N; t += 2) f2unpack(gelu2(v[t], v[t + 1]), v[t], v[t + 1]);
        break;
    case QFP4_ACT_GELU_TANH:
#pragma unroll
        for (int t = 0; t < N; t += 2)
            f2unpack(f2mul(f2pack(v[t], v[t + 1]), sigmoid_tanh2(v[t], v[t + 1]).f(v[t], v[t + 1])), v[t], v[t + 1]);
        break;
    case QFP4_ACT_SILU:
#pragma unroll
        for (int t = 0; t < N; t += 2)
            f2unpack(f2mul(f2pack(v[t], v[t + 1]), sigmoid2(v[t], v[t + 1]).f(v[t], v[t + 1])), v[t], v[t + 1]);
        break;
    default: break;
    }
}

// d[t] *= act'(z[t]) on N values (N even).  (ReLU's slope at a NaN is 0.)
template <int N>
__device__ __forceinline__ void act_backward(float *d, const float *z, int act)
{
    switch (act) {
    case QFP4_ACT_RELU:
#pragma unroll
        for (int t = 0; t < N; ++t) d[t] = z[t] > 0.0f ? d[t] : 0.0f;
        break;
    case QFP4_ACT_GELU:
#pragma unroll
        for (int t = 0; t < N; t += 2)
            f2unpack(f2mul(f2pack(d[t], d[t + 1]), gelu_slope2(z[t], z[t + 1])), d[t], d[t + 1]);
        break;
    case QFP4_ACT_GELU_TANH:
        // f + x f g 2 sqrt(2/pi) (1 + 3 0.044715 x^2); beyond |z| = 80 the slope is
        // 0 or 1 to binary32: the clamp keeps z^3 and the products finite
#pragma unroll
        for (int t = 0; t < N; t += 2) {
            const float x0 = clamp_nan(z[t], 80.0f), x1 = clamp_nan(z[t + 1], 80.0f);
            const Sigmoid2 s = sigmoid_tanh2(x0, x1);
            const uint64_t x = f2pack(x0, x1);
            const uint64_t k = f2fma(f2mul(x, f2pack(0.214064449f, 0.214064449f)), x, f2pack(1.59576917f, 1.59576917f));
            f2unpack(f2mul(f2pack(d[t], d[t + 1]), f2fma(s.zfg(x), k, s.f(x0, x1))), d[t], d[t + 1]);
        }
        break;
    case QFP4_ACT_SILU:
        // f + z f g
#pragma unroll
        for (int t = 0; t < N; t += 2) {
            const Sigmoid2 s = sigmoid2(z[t], z[t + 1]);
            const uint64_t k = f2add(s.zfg(f2pack(z[t], z[t + 1])), s.f(z[t], z[t + 1]));
            f2unpack(f2mul(f2pack(d[t], d[t + 1]), k), d[t], d[t + 1]);
        }
        break;
    default: break;
    }
}

// ------------------------------------------------------------------ element access
__device__ __forceinline__ float ld_as_float(const void *p, int f32, int64_t i)
{
    return f32 ? static_cast<const float *>(p)[i]
               : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
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
struct alignas(16) Row16 {
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

// Four bias values from column col on, as binary32; zeros without a bias or
// beyond the nc columns that exist (nc a multiple of 4).
__device__ __forceinline__ float4 bias4_load(const EpParams &ep, int col, int nc)
{
    if (!ep.bias || nc <= 0) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (ep.bias_f32) return __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(ep.bias) + col));
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(ep.bias) + col));
    return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

// A lane has a row and works on sixteen columns at a time, whole 32-byte
// sectors: 8192 x 11008 x 4096 NVFP4 with bias, GELU and z kept took 693 us on
// the plain product's fragments (two columns a lane, one element at a time),
// 322 a lane a row (with erff), 215 with GELU as above and the bias staged (255 in
// a sustained loop, under the power cap; with the bias alone 182).
//
// The last step of qfp4_gemm_epilogue on the accumulators acc[0 .. 15] of one
// row's columns col .. col + 15 (the first nc of them exist; nc and col are
// multiples of 4), i = row * N + col: z = alpha acc + bias, the optional copy
// of z, the activation, dropout, the residual, one rounding to the output
// type.  bias: the sixteen values, in shared memory (every thread of a warp
// reads the same ones) or registers.  The residual's loads are issued first
// and used last.
template <int OUT>
__device__ __forceinline__ void ep_chunk16(const EpParams &ep, void *out, int64_t i, int nc, float alpha, uint64_t step,
                                           const uint32_t *acc, const float4 *bias)
{
    Row16 res;
    if (ep.residual) row16_load(res, ep.residual, ep.residual_f32, i, nc, ep.wide);
    float v[16];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const float4 b = bias[g];
        v[4 * g] = fmaf(__uint_as_float(acc[4 * g]), alpha, b.x);
        v[4 * g + 1] = fmaf(__uint_as_float(acc[4 * g + 1]), alpha, b.y);
        v[4 * g + 2] = fmaf(__uint_as_float(acc[4 * g + 2]), alpha, b.z);
        v[4 * g + 3] = fmaf(__uint_as_float(acc[4 * g + 3]), alpha, b.w);
    }
    if (ep.preact) row16_store<OUT>(ep.preact, i, v, nc, ep.wide);
    act_forward<16>(v, ep.act);
    if (ep.drop.on) {
        drop_values<16, false>(ep.drop, step, i, v);
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
// col0 .. col0 + 127, sixteen at a time.  bias: those columns' values in
// shared memory.  row < M only.
template <int OUT>
__device__ __forceinline__ void ep_row128(const EpParams &ep, void *out, int N, int row, int col0, float alpha,
                                          uint64_t step, const uint32_t *r, const float4 *bias)
{
    const int64_t i0 = static_cast<int64_t>(row) * N + col0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int col = col0 + 16 * c, nc = imin(16, N - col);
        if (nc > 0) ep_chunk16<OUT>(ep, out, i0 + 16 * c, nc, alpha, step, r + 16 * c, bias + 4 * c);
    }
}

}  // namespace qfp4
