// vec.cuh -- sixteen-byte vectors of bf16 or binary32 values, and reductions,
// for the elementwise and row kernels (dropout, epilogue backward, layer norm).
#pragma once

#include "epilogue.cuh"

namespace qfp4 {

// V binary32 values as packed pairs (V = 1: one value), so that sums and
// products take one instruction for two of them.
template <int V>
struct Fv {
    uint64_t p[V / 2];

    static __device__ __forceinline__ Fv splat(float s)
    {
        Fv o;
#pragma unroll
        for (int k = 0; k < V / 2; ++k) o.p[k] = f2pack(s, s);
        return o;
    }
    static __device__ __forceinline__ Fv of(const float *v)
    {
        Fv o;
#pragma unroll
        for (int k = 0; k < V / 2; ++k)
            o.p[k] = static_cast<uint64_t>(__float_as_uint(v[2 * k + 1])) << 32 | __float_as_uint(v[2 * k]);
        return o;
    }
    __device__ __forceinline__ void to(float *v) const
    {
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            v[2 * k] = __uint_as_float(static_cast<uint32_t>(p[k]));
            v[2 * k + 1] = __uint_as_float(static_cast<uint32_t>(p[k] >> 32));
        }
    }
    __device__ __forceinline__ float sum() const
    {
        uint64_t a = p[0];
#pragma unroll
        for (int k = 1; k < V / 2; ++k) a = f2add(a, p[k]);
        float x, y;
        f2unpack(a, x, y);
        return x + y;
    }
};
template <>
struct Fv<1> {
    float p[1];
    static __device__ __forceinline__ Fv splat(float s) { return Fv{{s}}; }
    static __device__ __forceinline__ Fv of(const float *v) { return Fv{{v[0]}}; }
    __device__ __forceinline__ void to(float *v) const { v[0] = p[0]; }
    __device__ __forceinline__ float sum() const { return p[0]; }
};
__device__ __forceinline__ float f2add(float a, float b) { return a + b; }
__device__ __forceinline__ float f2sub(float a, float b) { return a - b; }
__device__ __forceinline__ float f2mul(float a, float b) { return a * b; }
__device__ __forceinline__ float f2fma(float a, float b, float c) { return fmaf(a, b, c); }
#define QFP4_FV(expr)                                      \
    Fv<V> o;                                               \
    _Pragma("unroll") for (int k = 0; k < (V + 1) / 2; ++k) o.p[k] = expr; \
    return o
template <int V>
__device__ __forceinline__ Fv<V> operator+(const Fv<V> &a, const Fv<V> &b)
{
    QFP4_FV(f2add(a.p[k], b.p[k]));
}
template <int V>
__device__ __forceinline__ Fv<V> operator-(const Fv<V> &a, const Fv<V> &b)
{
    QFP4_FV(f2sub(a.p[k], b.p[k]));
}
template <int V>
__device__ __forceinline__ Fv<V> operator*(const Fv<V> &a, const Fv<V> &b)
{
    QFP4_FV(f2mul(a.p[k], b.p[k]));
}
template <int V>
__device__ __forceinline__ Fv<V> fma(const Fv<V> &a, const Fv<V> &b, const Fv<V> &c)
{
    QFP4_FV(f2fma(a.p[k], b.p[k], c.p[k]));
}
#undef QFP4_FV

// V values of type DT at element i: 16 bytes (V = 8 bf16 or 4 binary32; i a
// multiple of V), or one value (V = 1).  Raw holds them as loaded.
template <int DT, int V>
struct Vec {
    static constexpr int W = V * (DT == QFP4_F32 ? 4 : 2) / 4;   // 32-bit words
    static_assert(V == 1 || W == 4, "16 bytes or one value");
    uint32_t r[V == 1 ? 1 : 4];

    __device__ __forceinline__ void load(const void *p, int64_t i)
    {
        if constexpr (V > 1) {
            const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + i * (DT == QFP4_F32 ? 4 : 2));
            r[0] = u.x;
            r[1] = u.y;
            r[2] = u.z;
            r[3] = u.w;
        } else if constexpr (DT == QFP4_F32)
            r[0] = static_cast<const uint32_t *>(p)[i];
        else
            r[0] = static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]);
    }
    __device__ __forceinline__ void get(float *v) const
    {
#pragma unroll
        for (int t = 0; t < V; ++t) {
            if constexpr (DT == QFP4_F32) v[t] = __uint_as_float(r[t]);
            else v[t] = t & 1 ? bf16hi(r[t >> 1]) : bf16lo(r[t >> 1]);
        }
    }
    __device__ __forceinline__ Fv<V> values() const
    {
        float v[V];
        get(v);
        return Fv<V>::of(v);
    }
    __device__ __forceinline__ void set(const Fv<V> &f)
    {
        float v[V];
        f.to(v);
        set(v);
    }
    // one rounding to DT
    __device__ __forceinline__ void set(const float *v)
    {
        if constexpr (DT == QFP4_F32) {
#pragma unroll
            for (int t = 0; t < V; ++t) r[t] = __float_as_uint(v[t]);
        } else if constexpr (V == 1)
            r[0] = pack_bf16(v[0], 0.0f);
        else {
#pragma unroll
            for (int t = 0; t < V; t += 2) r[t >> 1] = pack_bf16(v[t], v[t + 1]);
        }
    }
    __device__ __forceinline__ void store(void *p, int64_t i) const
    {
        if constexpr (V > 1)
            *reinterpret_cast<uint4 *>(static_cast<char *>(p) + i * (DT == QFP4_F32 ? 4 : 2)) =
                make_uint4(r[0], r[1], r[2], r[3]);
        else if constexpr (DT == QFP4_F32)
            static_cast<uint32_t *>(p)[i] = r[0];
        else
            static_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(r[0]);
    }
    // element t alone (of the vector that starts at element i of p)
    __device__ __forceinline__ void load1(const void *p, int64_t i, int t)
    {
        if constexpr (DT == QFP4_F32) r[t] = static_cast<const uint32_t *>(p)[i + t];
        else {
            const uint32_t h = static_cast<const uint16_t *>(p)[i + t];
            r[t >> 1] = t & 1 ? (r[t >> 1] & 0xFFFFu) | (h << 16) : (r[t >> 1] & 0xFFFF0000u) | h;
        }
    }
    __device__ __forceinline__ void store1(void *p, int64_t i, int t) const
    {
        if constexpr (DT == QFP4_F32) static_cast<uint32_t *>(p)[i + t] = r[t];
        else static_cast<uint16_t *>(p)[i + t] = static_cast<uint16_t>(t & 1 ? r[t >> 1] >> 16 : r[t >> 1]);
    }
};

// V parameter values (gamma, beta) from column c on (c a multiple of V), of
// either type.
template <int V>
__device__ __forceinline__ void ld_param(const void *p, int f32, int64_t c, float *v)
{
    if constexpr (V == 1) v[0] = ld_as_float(p, f32, c);
    else if (f32) {
#pragma unroll
        for (int t = 0; t < V; t += 4) {
            const float4 u = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + c + t));
            v[t] = u.x;
            v[t + 1] = u.y;
            v[t + 2] = u.z;
            v[t + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int t = 0; t < V; t += 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + c + t));
            v[t] = bf16lo(u.x);
            v[t + 1] = bf16hi(u.x);
            v[t + 2] = bf16lo(u.y);
            v[t + 3] = bf16hi(u.y);
        }
    }
}

template <int V>
__device__ __forceinline__ Fv<V> ld_param(const void *p, int f32, int64_t c)
{
    float v[V];
    ld_param<V>(p, f32, c, v);
    return Fv<V>::of(v);
}

__device__ __forceinline__ float warp_sum(float a)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    return a;
}

// Sum of G threads' values in each of them (G = 32: the warp; else the whole
// block of G), in a fixed order.  red: G / 32 floats that nothing else uses
// until the block's next barrier after this one.
template <int G>
__device__ __forceinline__ float group_sum(float a, float *red)
{
    a = warp_sum(a);
    if constexpr (G > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
        __syncthreads();
        a = 0.0f;
#pragma unroll
        for (int w = 0; w < G / 32; ++w) a += red[w];
    }
    return a;
}
// The same of R values each, with one barrier.
template <int G, int R>
__device__ __forceinline__ void group_sums(float *a, float (*red)[G == 32 ? 1 : G / 32])
{
#pragma unroll
    for (int r = 0; r < R; ++r) a[r] = warp_sum(a[r]);
    if constexpr (G > 32) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) red[r][threadIdx.x >> 5] = a[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            a[r] = 0.0f;
#pragma unroll
            for (int w = 0; w < G / 32; ++w) a[r] += red[r][w];
        }
    }
}
// The same of two values; `bar` is the named barrier of the G threads (their
// block may hold several groups), which all of them pass once.
template <int G>
__device__ __forceinline__ float2 group_sum2(float a, float b, float2 *red, int bar)
{
    a = warp_sum(a);
    b = warp_sum(b);
    if constexpr (G > 32) {
        if ((threadIdx.x & 31) == 0) red[(threadIdx.x % G) >> 5] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(G) : "memory");
        uint64_t s = 0ull;                                    // (0, 0)
#pragma unroll
        for (int w = 0; w < G / 32; ++w) s = f2add(s, *reinterpret_cast<const uint64_t *>(red + w));
        f2unpack(s, a, b);
    }
    return make_float2(a, b);
}

}  // namespace qfp4
