// quad.cuh -- four columns of one row in the two storage types, and the
// activations of the convolution and the selective scan, on float32 pairs.
#pragma once

#include "f32x2.cuh"
#include "sse_internal.cuh"

namespace sse {

template <typename T> struct Quad;
template <> struct Quad<__nv_bfloat16> {
    using Raw = uint2;
    static __device__ __forceinline__ void unpack(Raw u, F2 (&f)[2]) {
        f[0] = f2_bits(u.x << 16, u.x & 0xffff0000u);
        f[1] = f2_bits(u.y << 16, u.y & 0xffff0000u);
    }
    static __device__ __forceinline__ uint32_t two(F2 v) {
        const float2 f = f2_get(v);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
    static __device__ __forceinline__ Raw pack(const F2 (&f)[2]) { return make_uint2(two(f[0]), two(f[1])); }
    static __device__ __forceinline__ Raw zero() { return make_uint2(0, 0); }
};
template <> struct Quad<float> {
    using Raw = uint4;
    static __device__ __forceinline__ void unpack(Raw u, F2 (&f)[2]) {
        f[0] = f2_bits(u.x, u.y);
        f[1] = f2_bits(u.z, u.w);
    }
    static __device__ __forceinline__ Raw pack(const F2 (&f)[2]) {
        const float2 a = f2_get(f[0]), b = f2_get(f[1]);
        return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
    static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
};

// One column of two rows, as a pair over the rows.
template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> {
    using Raw = uint16_t;
    static __device__ __forceinline__ F2 unpack(Raw a, Raw b) { return f2_bits((uint32_t)a << 16, (uint32_t)b << 16); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *a, __nv_bfloat16 *b, F2 v, bool first, bool second) {
        const uint32_t w = Quad<__nv_bfloat16>::two(v);
        if (first) *reinterpret_cast<uint16_t *>(a) = (uint16_t)w;
        if (second) *reinterpret_cast<uint16_t *>(b) = (uint16_t)(w >> 16);
    }
};
template <> struct Two<float> {
    using Raw = uint32_t;
    static __device__ __forceinline__ F2 unpack(Raw a, Raw b) { return f2_bits(a, b); }
    static __device__ __forceinline__ void store(float *a, float *b, F2 v, bool first, bool second) {
        const float2 f = f2_get(v);
        if (first) *a = f.x;
        if (second) *b = f.y;
    }
};

__device__ __forceinline__ F2 both(float x) { return f2(x, x); }
__device__ __forceinline__ float fold(F2 v) {
    const float2 f = f2_get(v);
    return f.x + f.y;
}
// Two pairs as one 16-byte word.
__device__ __forceinline__ void write_quad(float *to, const F2 (&f)[2]) {
    const float2 u = f2_get(f[0]), v = f2_get(f[1]);
    *reinterpret_cast<float4 *>(to) = make_float4(u.x, u.y, v.x, v.y);
}
__device__ __forceinline__ void read_quad(const float *from, F2 (&f)[2]) {
    const float4 v = *reinterpret_cast<const float4 *>(from);
    f[0] = f2(v.x, v.y);
    f[1] = f2(v.z, v.w);
}
__device__ __forceinline__ float ex2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ F2 ex2_ftz(F2 x) {
    const float2 v = f2_get(x);
    return f2(ex2_ftz(v.x), ex2_ftz(v.y));
}
__device__ __forceinline__ F2 rcp_ftz(F2 x) {
    const float2 v = f2_get(x);
    return f2(rcp_ftz(v.x), rcp_ftz(v.y));
}

// 1 / (1 + exp(-u)).  For bf16 rows from the approximate exponential: the product's rounding is |u| 2^-24 of exp(-u), next to
// the rows' own steps of 2^-8 nothing.  In float32 exp is expf.  The reciprocal is one unit in the last place off.
template <typename T> __device__ __forceinline__ F2 sigmoid2(F2 u) {
    if constexpr (sizeof(T) == 4) {
        const float2 v = f2_get(u);
        return rcp_ftz(f2(1.f + expf(-v.x), 1.f + expf(-v.y)));
    } else {
        return rcp_ftz(add2(ex2_ftz(mul2(u, both(-1.44269504f))), both(1.f)));
    }
}

__device__ __forceinline__ int clamp_token(int t, int T) { return t < 0 ? 0 : t > T ? T : t; }

// Largest s in [0, S) with cu[s] <= t (0 if none): the sequence of token t, and for a token past the last one the last sequence.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int S, int t) {
    int lo = 0, hi = S;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// f(q) for the empty ones among the sequences first, first + stride, ...: a warp's lanes 0 to n - 1 look at n of them at a
// time (one after the other 400 sequences of a call without other work took 170 us).  All of those lanes call it.
template <typename F>
__device__ __forceinline__ void each_empty(const int32_t *cu, int S, int first, int stride, int lane, int n, F f) {
    const uint32_t lanes = n < 32 ? (1u << n) - 1 : 0xffffffffu;
    for (int64_t q0 = first; q0 < S; q0 += (int64_t)n * stride) {
        const int64_t q = q0 + (int64_t)lane * stride;
        uint32_t m = __ballot_sync(lanes, q < S && __ldg(cu + (q < S ? q : 0)) >= __ldg(cu + (q < S ? q : 0) + 1));
        for (; m; m &= m - 1) f((int)(q0 + (int64_t)(__ffs(m) - 1) * stride));
    }
}

// N words of 16 bytes, every STEP-th, from `from` (zeros without) to `to`, loads ahead of the stores.
template <int N, int STEP> __device__ __forceinline__ void copy_words(float *to, const float *from) {
    constexpr int B = N < 4 ? N : 4;
    static_assert(N % B == 0, "whole batches");
#pragma unroll
    for (int i = 0; i < N; i += B) {
        float4 v[B];
#pragma unroll
        for (int k = 0; k < B; ++k)
            v[k] = from ? *reinterpret_cast<const float4 *>(from + (i + k) * STEP * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < B; ++k) *reinterpret_cast<float4 *>(to + (i + k) * STEP * 4) = v[k];
    }
}

}  // namespace sse
