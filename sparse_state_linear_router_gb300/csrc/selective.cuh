// selective.cuh -- what the forward and the backward of the selective scan share:
// ranges of the packed token axis, the steps and their decays, tiles of 16 tokens and
// their staging.
#pragma once

#include "quad.cuh"

namespace sse {

constexpr int kTile = 16;        // tokens of a tile, aligned in the packed token axis
constexpr int kMaxRanges = 128;  // of the token axis
static_assert(kTile == kSelectiveCheckpoint, "a checkpoint is the state before a tile");

struct SelectiveShape {
    int width, groups, per, tiles;  // channels; groups; channels and tiles of a group
    int ranges;                     // of the token axis, at most: CTAs along it
    int fill;                       // ranges that fill the GPU
    bool alone;                     // sequences that fill it by themselves, if they are even
};

// Ranges of the token axis for `ctas` along the channels, of which the GPU holds `slots`.  A range that begins inside a
// sequence costs a pass of its own over the range before it and the last wave of CTAs is as long as the others, so ranges
// make whole waves: as many of `waves` (most first) as leave a range `tokens` of each.  One sequence of 32768 x 2048: forward
// with 1, 2 and 3 waves of three warps per SM quarter 519, 515 and 538 us, between two of them 523 to 538; backward with 2
// and 4 1562 and 1567, between them 1598 and 1635.  8192 x 512: forward with two warps per quarter 58, with one 60, with
// three 69; backward with 1 and 2 waves 125 and 134.
struct Waves {
    double waves;
    int tokens;
};
template <int M> inline int ranges_that_fill(int64_t ctas, int slots, const Waves (&choices)[M], int64_t T) {
    const int64_t most = T / (4 * kTile) < kMaxRanges ? T / (4 * kTile) : kMaxRanges;
    int64_t r = 0;
    for (const Waves &w : choices) {
        r = (int64_t)(w.waves * slots / ctas);
        if (r <= kMaxRanges && r * w.tokens <= T) break;
    }
    r = r < most ? r : most;
    return r < 1 ? 1 : (int)r;
}

inline SelectiveShape selective_shape(const sse_selective_config_t &c, int cols) {
    SelectiveShape s{c.width, c.groups, c.width / c.groups, 0, 1, 1, false};
    s.tiles = (s.per + cols - 1) / cols;
    return s;
}
// Sequences that make `enough` warps by themselves have a range each where the kernels find them even: no range then needs a
// pass of its own.  Measured at a range each against ranges that fill the GPU, 8 x 2048 tokens in bf16 with 8, 16 and 32
// states: forward with 512 warps 289, 391, 644 against 207, 273, 509 us, 832 warps 291, 396, 668 against 322, 437, 836, 1024
// warps 293, 398, 692 against 377, 525, 997; backward with 512 warps 566, 767, 1690 against 320, 429, 938, 1024 warps 572,
// 780, 1718 against 617, 824, 1775, 1664 warps 964, 1261, 2934 against 994, 1331, 2870, 2048 warps 1127, 1526, 3394 against
// 1189, 1588, 3391.  The one limit of 1000 is on the right side of these but for the forward's 832 warps; between two whole
// waves it is not: backward with 1280 warps 957, 1237, 2835 against 777, 1030, 2234.  float32 and 64 states go the same way.
inline void set_ranges(SelectiveShape &s, int fill, int enough, int32_t S) {
    s.fill = fill;
    s.alone = S > 1 && S <= kMaxRanges && (int64_t)S * s.tiles * s.groups >= enough;
    s.ranges = s.alone && S > fill ? S : fill;
}

// log2 e and what float32 leaves of it.
constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596303e-8f;

// A step's decay, 2^(d A log2 e).  The approximate exponential is low by 6e-9 to 2e-8 of the decay on average for exponents
// from -0.1 to 0, and a state with a long memory has that a thousand times over; 1.5e-8 put on the exponent leaves a third.
// (Relative error of the gradient of A, 8 x 4096 x 2048: 1.8e-6 without, 8e-7 with; the states' own steps are above it for
// exponents beyond -0.3.)
__device__ __forceinline__ F2 decay2(F2 d, F2 A) { return ex2_ftz(fma2(d, A, both(2.1e-8f))); }

// -150 at least (exp of it is 0), so that an infinity makes no NaN; a NaN stays one.
__device__ __forceinline__ float above(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(-150.f));
    return y;
}

// softplus(v) = max(v, 0) + log1p(exp(-|v|)), log1p(u) = 2 atanh(u / (2 + u)): the odd series of atanh on [0, 1/3] as a
// polynomial of degree 4 in the square (relative error 8e-9 by its coefficients).  The exponent's rounding is put back to
// first order: small steps are proportional to exp(v), and a step's relative error goes into a state's whole memory.
// With SLOPE its derivative 1 / (1 + exp(-v)) from the same exponential.
template <bool SLOPE> __device__ __forceinline__ F2 softplus2(F2 v, F2 &slope) {
    const float2 f = f2_get(v);
    const F2 m = f2(above(-fabsf(f.x)), above(-fabsf(f.y)));
    const F2 t = mul2(m, both(kLog2e));
    const F2 r = fma2(m, both(kLog2eRest), fma2(m, both(kLog2e), mul2(t, both(-1.f))));
    F2 u = ex2_ftz(t);
    u = fma2(u, mul2(r, both(0.693147181f)), u);
    const F2 s = mul2(u, rcp_ftz(add2(u, both(2.f)))), z = mul2(s, s);
    F2 p = both(0.28178346f);
    p = fma2(p, z, both(0.2796061f));
    p = fma2(p, z, both(0.4002491f));
    p = fma2(p, z, both(0.66666317f));
    p = fma2(p, z, both(2.f));
    if constexpr (SLOPE) {
        const F2 q = rcp_ftz(add2(u, both(1.f)));
        const float2 hi = f2_get(q), lo = f2_get(mul2(u, q));
        slope = f2(f.x < 0.f ? lo.x : hi.x, f.y < 0.f ? lo.y : hi.y);
    }
    // a NaN stays one: exp(-|v|) has it
    return fma2(s, p, f2(fmaxf(f.x, 0.f), fmaxf(f.y, 0.f)));
}

// ---------------------------------------------------------------------------
// Ranges of the token axis, of 64 tokens and more.  Range r of n begins at the
// start of a sequence that is no further than a quarter of a range from the
// r-th n-th of the tokens, or at the multiple of 16 below that; one that begins
// inside a sequence takes the state that the ranges before it hand on.  Starts
// are in order: from their places, 64 tokens apart, they are a quarter of that off,
// or 15 to the left.  Even sequences, a sixteenth off at most, have a range each.
// ---------------------------------------------------------------------------
// Whether every sequence starts a sixteenth of a sequence at most from its place; all lanes of a warp ask.
__device__ __forceinline__ bool even_sequences(const int32_t *cu, int S, int end) {
    bool even = true;
    for (int q = threadIdx.x & 31; q < S; q += 32) {
        const int64_t off = (int64_t)__ldg(cu + q) * S - (int64_t)end * q;
        even = even && off * 16 <= end && off * 16 >= -end;
    }
    return __all_sync(0xffffffffu, even);
}

struct Ranges {
    const int32_t *cu;
    int S, end, n;  // sequences, their last token's successor, ranges with tokens
    // All lanes of a warp, with the same arguments; `even` is even_sequences.
    template <typename Even>
    __device__ __forceinline__ Ranges(const SelectiveArgs &a, const SelectiveShape &sh, Even even) : cu(a.cu_seqlens), S(a.num_seqs) {
        end = clamp_token(__ldg(cu + S), a.total_tokens);
        n = max(1, min(sh.fill, end / (4 * kTile)));  // of 64 tokens and more: starts are in order
        if (sh.alone && end / S >= 4 * kTile && even(cu, S, end)) n = S;
    }
    __device__ __forceinline__ int start(int r) const {
        if (r <= 0) return 0;
        if (r >= n) return end;
        const int t = (int)((int64_t)end * r / n), near = end / (4 * n);
        const int s = sequence_of(cu, S, t), lo = clamp_token(__ldg(cu + s), end), hi = clamp_token(__ldg(cu + s + 1), end);
        const int to = t - lo <= hi - t ? lo : hi;
        return abs(t - to) <= near ? to : t & ~(kTile - 1);
    }
    // The first token of the sequence that token t continues; t itself where t begins one, or is the end.
    __device__ __forceinline__ int origin(int t) const {
        return t >= end ? t : clamp_token(__ldg(cu + sequence_of(cu, S, t)), t);
    }
};

// Where sequences begin and end among the 16 tokens of a tile; tokens outside [t0, t1) have no bits.
struct Edges {
    uint32_t starts, ends;  // bit i: token i is the first / last of its sequence
    int seq;                // lane i: the sequence of token i
    int lo, hi;             // tokens of the last sequence looked up
    __device__ __forceinline__ Edges() : starts(0), ends(0), seq(0), lo(1), hi(0) {}
    __device__ __forceinline__ void find(const Ranges &rg, int row0, int t0, int t1, int lane) {
        if (row0 > lo && row0 + kTile < hi) {  // inside the sequence of the tile before
            starts = ends = 0;
            return;
        }
        const int t = row0 + (lane < kTile ? lane : kTile - 1);
        int b = 0, e = 0;
        seq = -1;
        if (t >= t0 && t < t1) {
            seq = sequence_of(rg.cu, rg.S, t);
            b = __ldg(rg.cu + seq);
            e = __ldg(rg.cu + seq + 1);
        }
        const bool mine = lane < kTile && seq >= 0;
        starts = __ballot_sync(0xffffffffu, mine && b == t);
        ends = __ballot_sync(0xffffffffu, mine && e == t + 1);
        lo = __shfl_sync(0xffffffffu, b, kTile - 1);
        hi = __shfl_sync(0xffffffffu, e, kTile - 1);
    }
};

// A warp's channels: COLS of one group, or what is left of it.
struct Columns {
    int g, c0, left;  // group, first channel, channels
    __device__ __forceinline__ Columns(const SelectiveShape &s, int tile, int cols) {
        g = tile / s.tiles;
        const int i = (tile - g * s.tiles) * cols;
        c0 = g * s.per + i;
        left = min(cols, s.per - i);
    }
};

// ---------------------------------------------------------------------------
// Staging: rows of a tile to shared memory by asynchronous copies of 16 bytes.
// Rows outside [t0, t1) and channels past the group's end are filled with zeros.
// ---------------------------------------------------------------------------
// `bytes` of each of the 16 rows, of which `live` exist (whole words).
template <int BYTES>
__device__ __forceinline__ void copy_rows(uint32_t dst, const char *src, int64_t stride, int live, int row0, int t0, int t1,
                                          const void *safe, int lane) {
    constexpr int W = BYTES / 16;
#pragma unroll
    for (int k = 0; k < kTile * W; k += 32) {
        const int id = k + lane, row = id / W, w = id % W;
        if (kTile * W < 32 && id >= kTile * W) break;
        const int t = row0 + row;
        const bool ok = t >= t0 && t < t1 && w * 16 < live;
        const void *from = ok ? static_cast<const void *>(src + (int64_t)t * stride + w * 16) : safe;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + id * 16), "l"(from), "r"(ok ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's groups are in flight; then the whole warp's words are there.
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncwarp();
}

// Four channels' float32 parameters; zeros where there are none.
__device__ __forceinline__ void load_quad(const float *p, int c, bool live, F2 (&f)[2]) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p && live) v = __ldg(reinterpret_cast<const float4 *>(p + c));
    f[0] = f2(v.x, v.y);
    f[1] = f2(v.z, v.w);
}

// 2 P floats in a row as P pairs.
template <int P> __device__ __forceinline__ void read_pairs(const float *p, F2 (&f)[P]) {
    static_assert(P % 2 == 0, "whole 16-byte words");
#pragma unroll
    for (int k = 0; k < P; k += 2) {
        const float4 v = *reinterpret_cast<const float4 *>(p + 2 * k);
        f[k] = f2(v.x, v.y);
        f[k + 1] = f2(v.z, v.w);
    }
}
template <int P> __device__ __forceinline__ void write_pairs(float *p, const F2 (&f)[P]) {
#pragma unroll
    for (int k = 0; k < P; k += 2) {
        const float2 u = f2_get(f[k]), v = f2_get(f[k + 1]);
        *reinterpret_cast<float4 *>(p + 2 * k) = make_float4(u.x, u.y, v.x, v.y);
    }
}

// States of a pair of channels, as pairs over the channels: NT in a row in each of two rows `stride` apart.  swap: the
// second two come first.
template <int NT> __device__ __forceinline__ void read_states(const float *p, int64_t stride, int swap, F2 (&f)[NT]) {
#pragma unroll
    for (int k = 0; k < NT; k += 2) {
        const int at = k ^ (swap << 1);
        const float2 u = *reinterpret_cast<const float2 *>(p + at), v = *reinterpret_cast<const float2 *>(p + stride + at);
        f[k] = f2(u.x, v.x);
        f[k + 1] = f2(u.y, v.y);
    }
}
template <int NT> __device__ __forceinline__ void write_states(float *p, int64_t stride, int swap, const F2 (&f)[NT]) {
#pragma unroll
    for (int k = 0; k < NT; k += 2) {
        const int at = k ^ (swap << 1);
        const float2 u = f2_get(f[k]), v = f2_get(f[k + 1]);
        *reinterpret_cast<float2 *>(p + at) = make_float2(u.x, v.x);
        *reinterpret_cast<float2 *>(p + stride + at) = make_float2(u.y, v.y);
    }
}
template <int NT> __device__ __forceinline__ void no_states(F2 (&f)[NT]) {
#pragma unroll
    for (int k = 0; k < NT; ++k) f[k] = both(0.f);
}
// Four values of B or C to shared memory, each twice: a pair of channels takes one as it is.
template <typename T> __device__ __forceinline__ void leave_twice(float4 *to, typename Quad<T>::Raw from) {
    F2 f[2];
    Quad<T>::unpack(from, f);
    const float2 u = f2_get(f[0]), v = f2_get(f[1]);
    to[0] = make_float4(u.x, u.x, u.y, u.y);
    to[1] = make_float4(v.x, v.x, v.y, v.y);
}
// NT values of a token, each twice, at `p`; swap as above.
template <int NT> __device__ __forceinline__ void read_twice(const float *p, int swap, F2 (&f)[NT]) {
#pragma unroll
    for (int k = 0; k < NT; k += 2) {
        const float4 v = *reinterpret_cast<const float4 *>(p + 2 * (k ^ (swap << 1)));
        f[k] = f2(v.x, v.y);
        f[k + 1] = f2(v.z, v.w);
    }
}

}  // namespace sse
