// scan.cu -- the gated linear recurrence h_t = a_t h_{t-1} + s(a_t) x_t, one
// state per channel: forward, backward and one step.
//
// A run of steps composes to h -> P h + q (P the product of its decays, q what
// it makes of a zero state), and runs compose in order.  So a long sequence is
// split over warps and CTAs: each makes its rows' (P, q), the runs ahead are
// composed to the state the rows start from, and the rows are gone through
// again from that state.  Rows stay in shared memory between the two, so HBM is
// read once and written once.
//
//  - A lane has 4 bytes of a row (two bf16 channels as a float32 pair, or one
//    float32), a warp ("worker") one 128-byte line of each of 16 (backward: 8)
//    consecutive rows, a CTA eight workers' rows: its tile.
//  - The CTAs of a cluster take consecutive tiles of the same 128-byte column,
//    hand their (P, q) to each other through distributed shared memory and move
//    on by the cluster's size.  The workers make the next tile's run while a
//    ninth warp (the conductor) composes and exchanges this one's.  Nothing
//    waits on global memory, there is no workspace, and the order of every
//    product and sum is fixed.
//  - The batch's packed token axis is one axis: a sequence's first row starts
//    from its own initial state (a reset), its last one writes the final state,
//    so uneven lengths cost nothing.  A reset is a select and no product with
//    zero: a NaN of one sequence does not reach the next.
//  - Rows come by asynchronous copies up to three tiles ahead, in 16-byte
//    words, and leave in 16-byte words from the place of the inputs they replace.
//  - Where a cluster's sequences fall evenly into a part for each of its CTAs,
//    each CTA goes through its own part alone.
//
// Measured on a GB300 (72000 tokens x 2048 channels in bf16; HBM floor at 6.77
// TB/s: forward 131 us, backward 218 us).  One sequence: forward 160 us with s = 1,
// 212 with s = 1 - a and 217 with s = sqrt(1 - a^2), backward 293, 362 and 398 us.
// 16 even sequences: 164, 157 and 159, 223, 288 and 319 us.  What is left is a
// cluster's exchange (the difference between the two) and, with a costly input
// factor, the arithmetic.  Gates below -1/2 take the general form of the factor:
// with log-gates 16 times as strong 222 and 224, 369 and 414 us, in even sequences
// 165 and 171, 302 and 336.  A column of one sequence has 8 CTAs at most, so narrow
// rows are bound by its steps: 512 channels 97 to 126 us forward, 211 to 221
// backward.  The first form, in
// which every warp composed for itself between two cluster barriers, took 413 us
// forward (s = 1, one sequence).  Exchange by asynchronous remote stores that an
// mbarrier counts, instead of the cluster's barrier: 196 against 179 us.
#include <atomic>
#include <type_traits>

#include <cooperative_groups.h>

#include "f32x2.cuh"
#include "sse_internal.cuh"

namespace sse {
namespace {

namespace cg = cooperative_groups;

constexpr int kWorkers = 8;                   // warps that go through rows
constexpr int kThreads = (kWorkers + 1) * 32;  // and the conductor
constexpr int kRowsFwd = 16, kRowsBwd = 8;    // rows of a worker in one tile
constexpr int kMaxCluster = 8;                // the portable cluster size
constexpr int kSolo = 6, kShare = 5;          // CTAs go alone if the largest part is at most 6/5 of its share
static_assert(kWorkers * kRowsBwd % kScanCheckpoint == 0 && kScanCheckpoint % kRowsFwd == 0,
              "checkpoints lie at workers' first rows, and the backward's tiles at checkpoints");

// ---------------------------------------------------------------------------
// A lane's channels of one row: two bf16 (computed as a float32 pair) or one
// float32.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }

template <typename F> __device__ __forceinline__ F2 each(F2 x, F f) {
    const float2 v = f2_get(x);
    return f2(f(v.x), f(v.y));
}
template <typename F> __device__ __forceinline__ float each(float x, F f) { return f(x); }
template <typename F> __device__ __forceinline__ F2 each(F2 x, F2 y, F2 z, F f) {
    const float2 v = f2_get(x), w = f2_get(y), u = f2_get(z);
    return f2(f(v.x, w.x, u.x), f(v.y, w.y, u.y));
}
template <typename F> __device__ __forceinline__ float each(float x, float y, float z, F f) { return f(x, y, z); }

template <typename T> struct Lane;
template <> struct Lane<__nv_bfloat16> {
    using V = F2;
    static constexpr int kCols = 2;
    static __device__ __forceinline__ V splat(float x) { return f2(x, x); }
    static __device__ __forceinline__ V unpack(uint32_t u) { return f2_bits(u << 16, u & 0xffff0000u); }
    static __device__ __forceinline__ uint32_t pack(V v) {
        const float2 f = f2_get(v);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
    static __device__ __forceinline__ V load_state(const float *p) {
        const float2 f = *reinterpret_cast<const float2 *>(p);
        return f2(f.x, f.y);
    }
    static __device__ __forceinline__ void store_state(float *p, V v) { *reinterpret_cast<float2 *>(p) = f2_get(v); }
};
template <> struct Lane<float> {
    using V = float;
    static constexpr int kCols = 1;
    static __device__ __forceinline__ V splat(float x) { return x; }
    static __device__ __forceinline__ V unpack(uint32_t u) { return __uint_as_float(u); }
    static __device__ __forceinline__ uint32_t pack(V v) { return __float_as_uint(v); }
    static __device__ __forceinline__ V load_state(const float *p) { return *p; }
    static __device__ __forceinline__ void store_state(float *p, V v) { *p = v; }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN stays NaN
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The root and its reciprocal, for float32 channels too: 2^-23 and 2^-22.9 off at most, once per row and channel, against
// 1e-7 of the series below them.
__device__ __forceinline__ float rsqrt_ftz(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sqrt_ftz(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a = exp(la) = 2^(la log2 e).  The product's rounding error is |la| 2^-24 of
// the result: next to the bf16 gates' own steps nothing.  For float32 gates it is
// put back to first order, 2^(t + r) = 2^t (1 + r ln 2); -infinity stops at
// e^-150 (the least float32 is e^-103), where the result is 0.
template <typename T> __device__ __forceinline__ typename Lane<T>::V decay(typename Lane<T>::V la) {
    using L = Lane<T>;
    if constexpr (sizeof(T) == 4) {
        la = max_nan(la, -150.f);
        const float t = la * 1.44269504f;
        const float r = fmaf(la, 1.92596303e-8f, fmaf(la, 1.44269504f, -t));  // log2 e - 1.44269504f
        const float a = ex2(t);
        return fmaf(a, r * 0.693147181f, a);
    } else {
        return each(mul2(la, L::splat(1.44269504f)), [](float x) { return ex2(x); });
    }
}

// 1 - exp(u) for -1/2 <= u <= 0: -u times the Chebyshev interpolation of (exp(u) -
// 1) / u on that interval.  Relative errors: for float32 gates, degree 5, 3.2e-9,
// 1e-7 with float32 roundings (the last product alone rounds by 6e-8); for bf16
// gates degree 4, 1.05e-7 and 1.9e-7, against the 2^-8 that a gate and its row are
// rounded by (and 3 to 5 % of the time with s = sqrt(1 - a^2)).  1 - exp(u) formed
// from exp(u) would cancel here.
template <typename T> __device__ __forceinline__ typename Lane<T>::V one_minus_exp_near0(typename Lane<T>::V u) {
    using L = Lane<T>;
    if constexpr (sizeof(T) == 2) {
        auto p = L::splat(-0.00678286f);
        p = fma2(p, u, L::splat(-0.04101321f));
        p = fma2(p, u, L::splat(-0.16655193f));
        p = fma2(p, u, L::splat(-0.49999288f));
        p = fma2(p, u, L::splat(-0.99999994f));
        return mul2(p, u);
    }
    auto p = L::splat(-0.0011234042f);
    p = fma2(p, u, L::splat(-0.008189614f));
    p = fma2(p, u, L::splat(-0.041630074f));
    p = fma2(p, u, L::splat(-0.16666242f));
    p = fma2(p, u, L::splat(-0.49999982f));
    p = fma2(p, u, L::splat(-1.f));
    return mul2(p, u);
}

// A row's decay a, input factor s(a) and, with GRAD, ds/dla.  NEAR0: every
// log-gate of the warp's rows is in [-1/2, 0], where one series gives 1 - a and
// with it a, without an exponential or a select.
template <typename T, int MODE, bool NEAR0, bool GRAD = false>
__device__ __forceinline__ void factors(typename Lane<T>::V la, typename Lane<T>::V &a, typename Lane<T>::V &s,
                                        typename Lane<T>::V *slope = nullptr) {
    using L = Lane<T>;
    const auto one = L::splat(1.f), minus = L::splat(-1.f);
    if constexpr (MODE == SSE_INPUT_PLAIN) {
        a = decay<T>(la);
    } else if constexpr (MODE == SSE_INPUT_COMPLEMENT) {
        if constexpr (NEAR0) {
            s = one_minus_exp_near0<T>(la);
            a = fma2(s, minus, one);
        } else {
            a = decay<T>(la);
            s = each(la, one_minus_exp_near0<T>(la), a, [](float x, float near0, float e) { return x > -0.5f ? near0 : 1.f - e; });
        }
        if constexpr (GRAD) *slope = mul2(a, minus);
    } else {
        typename L::V s2;  // 1 - a^2
        if constexpr (NEAR0) {
            const auto c = one_minus_exp_near0<T>(la);
            a = fma2(c, minus, one);
            s2 = fma2(c, a, c);
        } else {
            a = decay<T>(la);
            const auto u = add2(la, la);
            s2 = each(u, one_minus_exp_near0<T>(u), mul2(a, a), [](float x, float near0, float e) { return x > -0.5f ? near0 : 1.f - e; });
        }
        // r = 1 / s, 0 where no input enters (1 - a^2 below the least normal number, as the forward's root takes it):
        // the slope is 0 there.  A NaN stays.  The slope has one reciprocal root's error, 2^-22.9.
        if constexpr (GRAD) {
            const auto r = each(s2, [](float v) { return fabsf(v) < 1.17549435e-38f ? 0.f : rsqrt_ftz(v); });
            s = mul2(s2, r);
            *slope = mul2(mul2(a, a), mul2(r, minus));
        } else {
            s = each(s2, [](float v) { return sqrt_ftz(v); });
        }
    }
}

// A word's largest log-gate magnitude so far, as bits: larger bits of a negative
// number are further from 0.
__device__ __forceinline__ uint32_t further(uint32_t x, uint32_t y, uint32_t z, __nv_bfloat16) { return __vimax3_u16x2(x, y, z); }
__device__ __forceinline__ uint32_t further(uint32_t x, uint32_t y, uint32_t z, float) { return __vimax3_u32(x, y, z); }
// Whether all are in [-1/2, 0].
__device__ __forceinline__ bool near0(uint32_t bits, __nv_bfloat16) {
    return (bits & 0xffffu) <= 0xbf00u && (bits >> 16) <= 0xbf00u;
}
__device__ __forceinline__ bool near0(uint32_t bits, float) { return bits <= 0xbf000000u; }

// A run's composition.
template <typename V> struct Run {
    V P, q;
};

__device__ __forceinline__ int clamp_token(int t, int T) { return t < 0 ? 0 : t > T ? T : t; }

// Largest s with cu[s] <= t (-1 if none); S if t >= cu[S].
__device__ __forceinline__ int sequence_of(const int32_t *cu, int S, int t) {
    int lo = -1, hi = S + 1;  // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The packed tokens of one cluster: from the sequence start nearest to the
// range's share of the tokens to that of the next range.
__device__ __forceinline__ int range_start(const ScanArgs &p, int r, int ranges) {
    const int T = p.total_tokens, S = p.num_seqs;
    if (r >= ranges) return clamp_token(__ldg(p.cu_seqlens + S), T);
    if (r == 0) return clamp_token(__ldg(p.cu_seqlens), T);
    const int t = (int)((int64_t)T * r / ranges);
    const int s = sequence_of(p.cu_seqlens, S, t);
    const int lo = __ldg(p.cu_seqlens + (s < 0 ? 0 : s)), hi = __ldg(p.cu_seqlens + (s < S ? s + 1 : S));
    return clamp_token(t - lo <= hi - t ? lo : hi, T);
}

// Where sequences begin and end among the rows of a warp.
template <int ROWS> struct Edges {
    uint32_t starts, ends;  // bit i: row i is the first / last token of its sequence
    int seq;                // lane i: the sequence of row i
    int lo, hi;             // tokens of the last sequence looked up
    // Rows [row0, row0 + ROWS) within [t0, t1); rows outside have no bits.
    __device__ __forceinline__ void find(const ScanArgs &p, int row0, int t0, int t1, int lane) {
        if (row0 > lo && row0 + ROWS < hi) {  // inside the sequence of the rows before
            starts = ends = 0;
            return;
        }
        const int t = row0 + (lane < ROWS ? lane : ROWS - 1);
        int b = 0, e = 0;
        seq = -1;
        if (t >= t0 && t < t1) {
            seq = p.num_seqs == 1 ? 0 : sequence_of(p.cu_seqlens, p.num_seqs, t);
            seq = seq < 0 ? 0 : seq < p.num_seqs ? seq : p.num_seqs - 1;  // within bounds whatever cu_seqlens holds
            b = __ldg(p.cu_seqlens + seq);
            e = __ldg(p.cu_seqlens + seq + 1);
        }
        const bool mine = lane < ROWS && seq >= 0;
        starts = __ballot_sync(0xffffffffu, mine && b == t);
        ends = __ballot_sync(0xffffffffu, mine && e == t + 1);
        lo = __shfl_sync(0xffffffffu, b, ROWS - 1);
        hi = __shfl_sync(0xffffffffu, e, ROWS - 1);
    }
};

// ---------------------------------------------------------------------------
// Staging of rows: each warp copies its own rows to shared memory a few tiles
// ahead (16 bytes per lane, four rows per instruction) and waits for nobody
// else.  Rows outside [t0, t1) are filled with zeros, which change nothing:
// decay 1, input 0.
// ---------------------------------------------------------------------------
// row0: the tile's first row; whole: all its rows are within [t0, t1).  Lanes
// past the row's end copy nothing: their words start as zeros, and zeros are
// what rows of zeros leave in them.  (Addresses are formed anew for each tile:
// running pointers for every tensor took 30 registers.)
template <int ROWS>
__device__ __forceinline__ void copy_rows(uint32_t dst, const void *base, int64_t stride, int col_byte, int row0, int t0,
                                          int t1, bool whole, bool col_ok, int lane) {
    const char *src = static_cast<const char *>(base) + (row0 + (lane >> 3)) * stride + col_byte;
    if (whole) {
        if (col_ok) {
#pragma unroll
            for (int k = 0; k < ROWS; k += 4, src += 4 * stride)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + k * 128 + lane * 16), "l"(src) : "memory");
        }
    } else {
#pragma unroll
        for (int k = 0; k < ROWS; k += 4) {
            const int row = row0 + k + (lane >> 3);
            const bool ok = col_ok && row >= t0 && row < t1;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + k * 128 + lane * 16),
                         "l"(ok ? src + k * stride : static_cast<const char *>(base)), "r"(ok ? 16 : 0) : "memory");
        }
    }
}
// Zeros in a worker's ring of `words` 16-byte words, for the lanes that copy nothing.
__device__ __forceinline__ void clear_ring(uint32_t *mine, int words, bool col_ok, int lane) {
    if (!col_ok)
        for (int k = lane; k < words; k += 32) reinterpret_cast<uint4 *>(mine)[k] = make_uint4(0, 0, 0, 0);
    __syncwarp();
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's groups are in flight; then the whole warp's rows are there.
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncwarp();
}

// A worker's results go back through the slot they were made from, each word in
// the place of the input it replaces, and out in 16-byte words.
template <int ROWS>
__device__ __forceinline__ void store_rows(void *base, int64_t stride, int col_byte, const uint32_t *src, int row0, int t0,
                                           int t1, bool whole, bool col_ok, int lane) {
    char *dst = static_cast<char *>(base) + (row0 + (lane >> 3)) * stride + col_byte;
    const uint4 *from = reinterpret_cast<const uint4 *>(src) + lane;
    if (whole) {
        if (col_ok) {
#pragma unroll
            for (int k = 0; k < ROWS; k += 4, dst += 4 * stride) *reinterpret_cast<uint4 *>(dst) = from[k * 8];
        }
    } else {
#pragma unroll
        for (int k = 0; k < ROWS; k += 4, dst += 4 * stride) {
            const int row = row0 + k + (lane >> 3);
            if (col_ok && row >= t0 && row < t1) *reinterpret_cast<uint4 *>(dst) = from[k * 8];
        }
    }
}

// ---------------------------------------------------------------------------
// Exchange.  The workers of a CTA publish their rows' runs and go on with the
// next tile; a ninth warp, the conductor, composes them, sends the CTA's run to
// the cluster, meets the other conductors in the cluster's barrier and leaves
// each worker the state its rows start from.  The conductor stores nothing to
// global memory, so its release has little to wait for; the workers' arrivals
// carry no data to other CTAs and are relaxed.
// ---------------------------------------------------------------------------
// EARLY: a worker publishes the next tile's run before it meets the conductor for
// this one, so the workers' words and barriers are there twice, for two steps in
// turn.  72000 tokens x 2048 channels, s = 1, one sequence: forward 162 against
// 178 us; the backward's runs come late in its step, 303 against 298 us.
template <typename V, bool EARLY> struct alignas(16) Exchange {
    Run<V> warp[EARLY ? 2 : 1][kWorkers][32];  // the workers' runs; then, in the place of P, what the rows start from
    Run<V> cta[2][kMaxCluster][32];            // the runs of the cluster's CTAs, two steps in turn
    uint32_t warp_reset[EARLY ? 2 : 1][kWorkers], cta_reset[2][kMaxCluster];
    static __device__ __forceinline__ int turn(int step) { return EARLY ? step & 1 : 0; }

    // Named barriers.  1 and 2: the runs, all workers.  From 3: the starts, the conductor and a worker, or a pair of
    // them (EARLY: 16 barriers do not go round), so that no worker waits for all the others.
    static __device__ __forceinline__ void runs_published(int step) {
        asm volatile("barrier.cta.arrive %0, %1;" ::"r"(1 + turn(step)), "n"(kThreads) : "memory");
    }
    static __device__ __forceinline__ void await_runs(int step) {
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + turn(step)), "n"(kThreads) : "memory");
    }
    static __device__ __forceinline__ void starts_published(int step) {
#pragma unroll
        for (int w = 0; w < kWorkers; w += EARLY ? 2 : 1)
            asm volatile("barrier.cta.arrive %0, %1;" ::"r"(3 + w + turn(step)), "n"(EARLY ? 96 : 64) : "memory");
    }
    static __device__ __forceinline__ void await_starts(int step, int warp) {
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(3 + (EARLY ? warp & ~1 : warp) + turn(step)), "n"(EARLY ? 96 : 64)
                     : "memory");
    }
};

__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_release() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Bits of the n flags that are set.
__device__ __forceinline__ uint32_t reset_bits(const uint32_t *flags, int n, int lane) {
    return __ballot_sync(0xffffffffu, lane < n && flags[lane] != 0);
}

// Applies run r to a state; a reset leaves q alone.
template <typename V> __device__ __forceinline__ V apply(const Run<V> &r, V h, bool reset) {
    return reset ? r.q : fma2(r.P, h, r.q);
}

// Where this CTA's runs go in the cluster's CTAs (a conductor's registers).
template <typename V, bool EARLY> struct Outbox {
    uint32_t run[kMaxCluster], reset;
    __device__ __forceinline__ Outbox(Exchange<V, EARLY> &ex, int rank, int csize, int lane) {
        const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&ex.cta[0][rank][lane]);
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(run[k]) : "r"(mine), "r"(k < csize ? k : 0));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(reset)
            : "r"((uint32_t)__cvta_generic_to_shared(&ex.cta_reset[0][rank])), "r"(lane < csize ? lane : 0));
    }
    __device__ __forceinline__ void send(int buf, int csize, int lane, const Run<V> &r, uint32_t resets) const {
        const uint32_t off = buf * (uint32_t)sizeof(Exchange<V, EARLY>::cta[0]);
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
            if (k < csize) {
                if constexpr (sizeof(V) == 8) {
                    const float2 u = f2_get(r.P), v = f2_get(r.q);
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(run[k] + off), "f"(u.x), "f"(u.y),
                                 "f"(v.x), "f"(v.y) : "memory");
                } else {
                    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(run[k] + off), "f"(r.P), "f"(r.q)
                                 : "memory");
                }
            }
        if (lane < csize)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(reset + buf * (uint32_t)sizeof(Exchange<V, EARLY>::cta_reset[0])),
                         "r"(resets) : "memory");
    }
};

// The conductor's part of one step, between the workers' runs and their
// starts; `meanwhile` runs while the cluster gathers.  REVERSE: the last worker
// comes first.  `state` moves past the cluster's tiles.  Its length is what the
// cluster waits for, so steps without a reset take the short way.
template <bool REVERSE, bool ONE, typename V, bool EARLY, typename F>
__device__ __forceinline__ void conduct(const Outbox<V, EARLY> &out, Exchange<V, EARLY> &ex, int step, int rank, int csize, int lane,
                                        V &state, F meanwhile) {
    const int buf = step & 1;
    auto &warp = ex.warp[ex.turn(step)];
    const uint32_t resets = reset_bits(ex.warp_reset[ex.turn(step)], kWorkers, lane);
    Run<V> r[kWorkers];
#pragma unroll
    for (int k = 0; k < kWorkers; ++k) r[k] = warp[REVERSE ? kWorkers - 1 - k : k][lane];
    Run<V> all = r[0];
    if (resets == 0) {
#pragma unroll
        for (int k = 1; k < kWorkers; ++k) {
            all.q = fma2(r[k].P, all.q, r[k].q);
            all.P = mul2(all.P, r[k].P);
        }
    } else {
#pragma unroll
        for (int k = 1; k < kWorkers; ++k)
            all.q = apply(r[k], all.q, (resets >> (REVERSE ? kWorkers - 1 - k : k)) & 1u);
    }
    V mine = state;
    if constexpr (ONE) {
        meanwhile();
#pragma unroll
        for (int k = 0; k < kWorkers; ++k) {
            const int w = REVERSE ? kWorkers - 1 - k : k;
            warp[w][lane].P = mine;
            mine = apply(r[k], mine, (resets >> w) & 1u);
        }
        ex.starts_published(step);
        state = mine;
        return;
    }
    out.send(buf, csize, lane, all, resets);
    cluster_arrive_release();
    meanwhile();
    cluster_wait();
    const uint32_t cta_resets = reset_bits(ex.cta_reset[buf], csize, lane);
    if (cta_resets == 0) {
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            if (k == rank) mine = state;
            if (k < csize) {
                const Run<V> c = ex.cta[buf][k][lane];
                state = fma2(c.P, state, c.q);
            }
        }
#pragma unroll
        for (int k = 0; k < kWorkers; ++k) {
            warp[REVERSE ? kWorkers - 1 - k : k][lane].P = mine;
            mine = fma2(r[k].P, mine, r[k].q);
        }
    } else {
        for (int k = 0; k < csize; ++k) {
            if (k == rank) mine = state;
            state = apply(ex.cta[buf][k][lane], state, (cta_resets >> k) & 1u);
        }
#pragma unroll
        for (int k = 0; k < kWorkers; ++k) {
            const int w = REVERSE ? kWorkers - 1 - k : k;
            warp[w][lane].P = mine;
            mine = apply(r[k], mine, (resets >> w) & 1u);
        }
    }
    ex.starts_published(step);
}

// The tiles of one team: a cluster, or one CTA of it (`solo`).  Where the
// cluster's sequences fall evenly into a part for each CTA, each goes through its
// own and there is nothing to exchange.  16 even sequences, 72000 x 2048, when this
// was added: s = 1 168 us alone and 174 together, backward 224 and 294; s = sqrt(1 -
// a^2) 175 and 236, 339 and 374: a part a fifth over its share is about where they
// meet.
template <int ROWS> struct Span {
    static constexpr int kTile = kWorkers * ROWS;
    int t0, t1, tile0, tiles, steps;
    bool solo;
    __device__ __forceinline__ Span(const ScanArgs &p, int csize, int rank, int lane) {
        const int at = range_start(p, (int)blockIdx.y * csize + (lane < csize ? lane : csize), (int)gridDim.y * csize);
        const int len = __shfl_down_sync(0xffffffffu, at, 1) - at;
        const int most = __reduce_max_sync(0xffffffffu, lane < csize ? len : 0);
        t0 = __shfl_sync(0xffffffffu, at, 0);
        t1 = __shfl_sync(0xffffffffu, at, csize);
        solo = csize == 1 || (int64_t)most * csize * kShare <= (int64_t)(t1 - t0) * kSolo;
        if (solo) {
            t0 = __shfl_sync(0xffffffffu, at, rank);
            t1 = __shfl_sync(0xffffffffu, at, rank + 1);
        }
        tile0 = t0 / kTile;
        tiles = t1 > t0 ? (t1 + kTile - 1) / kTile - tile0 : 0;
        steps = solo ? tiles : (tiles + csize - 1) / csize;
    }
};

// Sequence edges among the rows of a worker's tile.
struct Marks {
    uint32_t starts, ends;
    int seq, row0;
    bool whole;  // every row is within [t0, t1)
    bool near0;  // every log-gate is in [-1/2, 0]
};

constexpr int kStagesFwd = 3, kStagesBwd = 3;  // tiles of a worker's ring

// ---------------------------------------------------------------------------
// Forward.  grid.x: column x cluster rank, grid.y: ranges of the token axis.
// Each tile's rows are gone through twice, once for their run and once from
// their start.  Two forms:
//  - HOLD false: the next tile's run is made while this one's is exchanged, and
//    the second pass makes the decays and inputs again from shared memory;
//  - HOLD true: they stay in registers between the passes, and only the SM's
//    other CTA is at work during the exchange.
// s = 1: 72000 tokens x 2048 channels, one sequence: 161 against 191 us (HOLD).
// s = sqrt(1 - a^2) in bf16, 20000 tokens, one sequence: clusters of 8 (2048
// channels) 77 against 69 us (HOLD), of 7 87 and 79, of 6 89 and 89, of 5 (3008
// channels) 103 and 102, with s = 1 - a 94 and 103, of 4 114 and 125; 72000
// tokens in 16 ragged sequences, clusters of 4: 226 and 236; CTAs that go alone
// (8 x 4096 tokens): 97 and 79.  float32 (one channel per lane, half the
// arithmetic): 170 and 202, alone 142 both.  At 512 channels, where an SM has one
// CTA at most: 150 and 189.
// ---------------------------------------------------------------------------
enum { kRemake, kHoldAlone, kHold };  // HOLD never, where CTAs go alone, always

template <typename T, int MODE, bool HOLD, bool ONE>
__device__ __forceinline__ void forward_tiles(const ScanArgs &p, int width, const Span<kRowsFwd> &sp,
                                              Exchange<typename Lane<T>::V, true> &ex, uint4 *ring, int csize, int rank, int col0) {
    using L = Lane<T>;
    using V = typename L::V;
    constexpr int kRows = kRowsFwd, kTile = kWorkers * kRows;
    constexpr int kSlotWords = kRows * 32, kSlotBytes = kSlotWords * 4;  // one tensor's rows of a worker
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = col0 + lane * L::kCols;
    const bool live = col < width;

    if (warp == kWorkers) {
        const Outbox<V, true> out(ex, rank, csize, lane);
        V state = L::splat(0.f);  // the state ahead of the cluster's tiles
        for (int step = 0; step < sp.steps; ++step) {
            ex.await_runs(step);
            conduct<false, ONE>(out, ex, step, rank, csize, lane, state, [] {});
        }
        return;
    }

    uint32_t *mine = reinterpret_cast<uint32_t *>(ring) + warp * (kStagesFwd * 2 * kSlotWords);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(mine);
    const bool col_ok = col0 + (lane & 7) * (16 / (int)sizeof(T)) < width;
    const int col_byte = col0 * (int)sizeof(T) + (lane & 7) * 16;
    clear_ring(mine, kStagesFwd * 2 * kSlotBytes / 16, col_ok, lane);
    const int first_row = (sp.tile0 + rank) * kTile + warp * kRows, stride = csize * kTile;
    const int64_t packed = (int64_t)width * (int)sizeof(T);
    int load_slot = 0, load_row = first_row;
    auto load = [&](int step) {  // called for one step after the other
        if (step < sp.steps) {
            const uint32_t dst = ring_at + load_slot * (2 * kSlotBytes);
            const bool whole = load_row >= sp.t0 && load_row + kRows <= sp.t1;
            copy_rows<kRows>(dst, p.log_gate, p.gate_stride * (int)sizeof(T), col_byte, load_row, sp.t0, sp.t1, whole, col_ok,
                             lane);
            copy_rows<kRows>(dst + kSlotBytes, p.x, p.x_stride * (int)sizeof(T), col_byte, load_row, sp.t0, sp.t1, whole, col_ok, lane);
            load_slot = load_slot + 1 == kStagesFwd ? 0 : load_slot + 1;
            load_row += stride;
        }
        copies_commit();
    };
    auto first_state = [&](int seq, int i) {
        const int s = __shfl_sync(0xffffffffu, seq, i);
        return p.init && live ? L::load_state(p.init + (int64_t)s * width + col) : L::splat(0.f);
    };
    auto all_near0 = [&](const uint32_t *src) {
        if constexpr (MODE == SSE_INPUT_PLAIN) return false;
        // 16 bytes at a time: as 4-byte words the compiler keeps them for the rows' factors and spills.
        const uint4 *words = reinterpret_cast<const uint4 *>(src - lane) + lane;
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < kRows / 4; ++i) {
            const uint4 u = words[i * 32];
            bits = further(further(bits, u.x, u.y, T()), u.z, u.w, T());
        }
        return (bool)__all_sync(0xffffffffu, near0(bits, T()));
    };
    // a and s x of row i of a slot
    auto make_row = [&](auto near, const uint32_t *src, int i, V &a, V &b) {
        V s;
        factors<T, MODE, decltype(near)::value>(L::unpack(src[i * 32]), a, s);
        b = L::unpack(src[kSlotWords + i * 32]);
        if constexpr (MODE != SSE_INPUT_PLAIN) b = mul2(b, s);
    };
    V held_a[HOLD ? kRows : 1], held_b[HOLD ? kRows : 1];
    auto hold_rows = [&](auto near, const uint32_t *src) {
#pragma unroll
        for (int i = 0; i < (HOLD ? kRows : 0); ++i) make_row(near, src, i, held_a[i], held_b[i]);
    };
    auto row_of = [&](auto near, const uint32_t *src, int i, V &a, V &b) {
        if constexpr (HOLD) {
            a = held_a[i];
            b = held_b[i];
        } else {
            make_row(near, src, i, a, b);
        }
    };

    Edges<kRows> ed;
    ed.lo = ed.hi = 0;
    // The run of one tile's rows.  `entry`: the initial state that enters at the last start among them (HOLD: it goes
    // into the row's held input).
    auto run_of = [&](auto near, Run<V> &run, const uint32_t *src) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            V a, b;
            row_of(near, src, i, a, b);
            run.q = fma2(a, run.q, b);
            run.P = mul2(run.P, a);
        }
    };
    auto first_pass = [&](Marks &m, V &entry, Run<V> &run, int row0, const uint32_t *src) {
        ed.find(p, row0, sp.t0, sp.t1, lane);
        m = Marks{ed.starts, ed.ends, ed.seq, row0, row0 >= sp.t0 && row0 + kRows <= sp.t1, all_near0(src)};
        if constexpr (HOLD) {
            if (m.near0)
                hold_rows(std::true_type{}, src);
            else
                hold_rows(std::false_type{}, src);
        }
        run = Run<V>{L::splat(1.f), L::splat(0.f)};
        if (m.starts == 0) {
            if (!HOLD && m.near0)
                run_of(std::true_type{}, run, src);
            else
                run_of(std::false_type{}, run, src);
        } else {
#pragma unroll(HOLD ? kRows : 1)
            for (int i = 0; i < kRows; ++i) {
                V a, b;
                row_of(std::false_type{}, src, i, a, b);
                if ((m.starts >> i) & 1u) {
                    // Read here and not again for the sequence that leaves these rows: where the final state is written
                    // over the initial one, another worker may have done so by the second pass.
                    if constexpr (HOLD) {
                        held_b[i] = fma2(a, first_state(m.seq, i), b);
                        run.q = held_b[i];
                    } else {
                        entry = first_state(m.seq, i);
                        run.q = fma2(a, entry, b);
                    }
                } else {
                    run.q = fma2(a, run.q, b);
                }
            }
            run.P = L::splat(0.f);
        }
    };
    auto publish = [&](const Marks &m, const Run<V> &run, int step) {
        ex.warp[step & 1][warp][lane] = run;
        if (lane == 0) ex.warp_reset[step & 1][warp] = m.starts;
        ex.runs_published(step);
    };
    auto states_of = [&](auto near, V h, uint32_t *src) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            V a, b;
            row_of(near, src, i, a, b);
            h = fma2(a, h, b);
            src[kSlotWords + i * 32] = L::pack(h);
        }
    };
    auto second_pass = [&](const Marks &m, const V &entry, V h, uint32_t *src) {
        if (p.checkpoints && live && m.row0 % kScanCheckpoint == 0 && m.row0 >= sp.t0 && m.row0 < sp.t1)
            L::store_state(p.checkpoints + (int64_t)(m.row0 / kScanCheckpoint) * width + col, h);
        if ((m.starts | m.ends) == 0) {
            if (!HOLD && m.near0)
                states_of(std::true_type{}, h, src);
            else
                states_of(std::false_type{}, h, src);
        } else {
            [[maybe_unused]] const int last = 31 - __clz(m.starts);
#pragma unroll(HOLD ? kRows : 1)
            for (int i = 0; i < kRows; ++i) {
                V a, b;
                row_of(std::false_type{}, src, i, a, b);
                const bool start = (m.starts >> i) & 1u;
                if constexpr (HOLD) {
                    h = start ? b : fma2(a, h, b);
                } else {
                    if (start) h = i == last ? entry : first_state(m.seq, i);  // the others end among these rows
                    h = fma2(a, h, b);
                }
                src[kSlotWords + i * 32] = L::pack(h);
                if ((m.ends >> i) & 1u) {
                    const int s = __shfl_sync(0xffffffffu, m.seq, i);
                    if (p.final_state && live) L::store_state(p.final_state + (int64_t)s * width + col, h);
                }
            }
        }
        __syncwarp();
        store_rows<kRows>(p.out, packed, col_byte, src - lane + kSlotWords, m.row0, sp.t0, sp.t1, m.whole, col_ok, lane);
        __syncwarp();  // the slot is free
    };
    auto slot = [&](int at) { return mine + at * (2 * kSlotWords) + lane; };
    // The workers' part in the cluster's barrier carries nothing.
    if (!ONE && sp.steps > 0) cluster_arrive_relaxed();
    auto take_start = [&](int step) {
        ex.await_starts(step, warp);
        const V h = ex.warp[step & 1][warp][lane].P;
        if (!ONE) {
            cluster_wait();
            if (step + 1 < sp.steps) cluster_arrive_relaxed();
        }
        return h;
    };
    Marks now;
    V entry = L::splat(0.f);
    Run<V> run;
    for (int k = 0; k < kStagesFwd; ++k) load(k);
    if constexpr (HOLD) {
        int at = 0, row0 = first_row;
        for (int step = 0; step < sp.steps; ++step, row0 += stride) {
            copies_wait<kStagesFwd - 1>();
            first_pass(now, entry, run, row0, slot(at));
            publish(now, run, step);
            const V h = take_start(step);
            second_pass(now, entry, h, slot(at));
            load(step + kStagesFwd);
            at = at + 1 == kStagesFwd ? 0 : at + 1;
        }
    } else if (sp.steps > 0) {
        Marks next;
        V next_entry = entry;
        copies_wait<kStagesFwd - 1>();
        first_pass(now, entry, run, first_row, slot(0));
        publish(now, run, 0);
        int at = 0;
        for (int step = 0; step < sp.steps; ++step) {
            const bool more = step + 1 < sp.steps;
            const int next_at = at + 1 == kStagesFwd ? 0 : at + 1;
            if (more) {
                copies_wait<kStagesFwd - 2>();
                first_pass(next, next_entry, run, now.row0 + stride, slot(next_at));
                publish(next, run, step + 1);
            }
            const V h = take_start(step);
            second_pass(now, entry, h, slot(at));
            load(step + kStagesFwd);
            now = next;
            entry = next_entry;
            at = next_at;
        }
    }
}

template <typename T, int MODE, int FORM>
__global__ void __launch_bounds__(kThreads, 2) scan_forward_kernel(ScanArgs p, int width) {
    using L = Lane<T>;
    extern __shared__ uint4 ring[];
    __shared__ Exchange<typename L::V, true> ex;
    const int csize = cg::this_cluster().num_blocks(), rank = cg::this_cluster().block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col0 = (int)(blockIdx.x / csize) * 32 * L::kCols;
    const Span<kRowsFwd> sp(p, csize, rank, lane);
    if (sp.solo) {
        forward_tiles<T, MODE, FORM != kRemake, true>(p, width, sp, ex, ring, 1, 0, col0);
    } else {
        cluster_arrive_relaxed();  // every CTA has started before the first run is sent
        cluster_wait();
        forward_tiles<T, MODE, FORM == kHold, false>(p, width, sp, ex, ring, csize, rank, col0);
    }
    const int col = col0 + lane * L::kCols;
    if (p.final_state && col < width && warp < kWorkers) {  // empty sequences keep their initial state
        const int n = gridDim.y * csize * kWorkers;
        for (int s = ((int)blockIdx.y * csize + rank) * kWorkers + warp; s < p.num_seqs; s += n)
            if (__ldg(p.cu_seqlens + s) >= __ldg(p.cu_seqlens + s + 1)) {
                const int64_t i = (int64_t)s * width + col;
                L::store_state(p.final_state + i, p.init ? L::load_state(p.init + i) : L::splat(0.f));
            }
    }
}

// ---------------------------------------------------------------------------
// Backward: the tiles from the last to the first.  What later tokens hand back,
// e_t = a_t (d_out_t + e_{t+1}), is the same kind of run in the other direction
// and goes through the cluster; a tile's states come from its checkpoint and the
// CTA's own rows, composed by the conductor in the same step.
// ---------------------------------------------------------------------------
template <typename V> struct BackShared {
    Exchange<V, false> ex;        // adjoint runs
    Run<V> fwd[kWorkers][32];     // the workers' state runs; then, in the place of P, the state ahead of its rows
    uint32_t fwd_reset[kWorkers];
};

template <typename T, int MODE, bool ONE>
__device__ __forceinline__ void backward_tiles(const ScanArgs &p, int width, const Span<kRowsBwd> &sp,
                                               BackShared<typename Lane<T>::V> &sh, uint4 *ring, int csize, int rank, int col0) {
    using L = Lane<T>;
    using V = typename L::V;
    constexpr int kRows = kRowsBwd, kTile = kWorkers * kRows;
    constexpr int kSlotWords = kRows * 32, kSlotBytes = kSlotWords * 4;  // one tensor's rows of a worker
    Exchange<V, false> &ex = sh.ex;
    auto &fwd = sh.fwd;
    auto &fwd_reset = sh.fwd_reset;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = col0 + lane * L::kCols;
    const bool live = col < width;
    const int last_tile = sp.tile0 + sp.tiles - 1 - rank;  // rank 0 has the last; below tile0 there are no rows

    if (warp == kWorkers) {
        auto checkpoint = [&](int step) {
            const int row = (last_tile - step * csize) * kTile;
            return live && row > sp.t0 ? L::load_state(p.checkpoints + (int64_t)(row / kScanCheckpoint) * width + col)
                                       : L::splat(0.f);
        };
        const Outbox<V, false> out(ex, rank, csize, lane);
        V check = sp.steps > 0 ? checkpoint(0) : L::splat(0.f);
        V adjoint = L::splat(0.f);  // what the tokens behind the cluster's tiles hand back
        for (int step = 0; step < sp.steps; ++step) {
            V state = check;
            if (step + 1 < sp.steps) check = checkpoint(step + 1);
            ex.await_runs(step);
            conduct<true, ONE>(out, ex, step, rank, csize, lane, adjoint, [&] {
                const uint32_t resets = reset_bits(fwd_reset, kWorkers, lane);
#pragma unroll
                for (int w = 0; w < kWorkers; ++w) {
                    const Run<V> r = fwd[w][lane];
                    fwd[w][lane].P = state;
                    state = apply(r, state, (resets >> w) & 1u);
                }
            });
        }
        return;
    }

    uint32_t *mine = reinterpret_cast<uint32_t *>(ring) + warp * (kStagesBwd * 3 * kSlotWords);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(mine);
    const bool col_ok = col0 + (lane & 7) * (16 / (int)sizeof(T)) < width;
    const int col_byte = col0 * (int)sizeof(T) + (lane & 7) * 16;
    clear_ring(mine, kStagesBwd * 3 * kSlotBytes / 16, col_ok, lane);
    const int first_row = last_tile * kTile + warp * kRows, stride = csize * kTile;
    const int64_t packed = (int64_t)width * (int)sizeof(T);
    int load_slot = 0, load_row = first_row;
    auto load = [&](int step) {  // called for one step after the other
        if (step < sp.steps) {
            const uint32_t dst = ring_at + load_slot * (3 * kSlotBytes);
            const bool whole = load_row >= sp.t0 && load_row + kRows <= sp.t1;
            copy_rows<kRows>(dst, p.log_gate, p.gate_stride * (int)sizeof(T), col_byte, load_row, sp.t0, sp.t1, whole, col_ok,
                             lane);
            copy_rows<kRows>(dst + kSlotBytes, p.x, p.x_stride * (int)sizeof(T), col_byte, load_row, sp.t0, sp.t1, whole, col_ok, lane);
            copy_rows<kRows>(dst + 2 * kSlotBytes, p.d_out, packed, col_byte, load_row, sp.t0, sp.t1, whole, col_ok, lane);
            load_slot = load_slot + 1 == kStagesBwd ? 0 : load_slot + 1;
            load_row -= stride;
        }
        copies_commit();
    };

    Edges<kRows> ed;
    ed.lo = ed.hi = 0;
    auto first_state = [&](int seq, int i) {
        const int q = __shfl_sync(0xffffffffu, seq, i);
        return p.init && live ? L::load_state(p.init + (int64_t)q * width + col) : L::splat(0.f);
    };
    auto last_adjoint = [&](int seq, int i) {
        const int q = __shfl_sync(0xffffffffu, seq, i);
        return p.d_final && live ? L::load_state(p.d_final + (int64_t)q * width + col) : L::splat(0.f);
    };
    auto all_near0 = [&](const uint32_t *src) {
        if constexpr (MODE == SSE_INPUT_PLAIN) return false;
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < kRows; i += 2) bits = further(bits, src[i * 32], src[(i + 1) * 32], T());
        return (bool)__all_sync(0xffffffffu, near0(bits, T()));
    };
    // a and s x of row i of a slot
    auto step_of = [&](auto near, const uint32_t *src, int i, V &a, V &b) {
        V s;
        factors<T, MODE, decltype(near)::value>(L::unpack(src[i * 32]), a, s);
        b = L::unpack(src[kSlotWords + i * 32]);
        if constexpr (MODE != SSE_INPUT_PLAIN) b = mul2(b, s);
    };
    // The tile's state run and, since a run of decays is the same both ways, its
    // adjoint run in one sweep: q_back = sum over rows of (a_first ... a_row) d_row.
    auto runs_of = [&](auto near, Run<V> &run, Run<V> &back, const uint32_t *src) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            V a, b;
            step_of(near, src, i, a, b);
            run.q = fma2(a, run.q, b);
            run.P = mul2(run.P, a);
            back.q = fma2(run.P, L::unpack(src[2 * kSlotWords + i * 32]), back.q);
        }
        back.P = run.P;
    };
    auto first_pass = [&](Marks &m, Run<V> &run, Run<V> &back, int row0, const uint32_t *src) {
        ed.find(p, row0, sp.t0, sp.t1, lane);
        m = Marks{ed.starts, ed.ends, ed.seq, row0, row0 >= sp.t0 && row0 + kRows <= sp.t1, all_near0(src)};
        run = back = Run<V>{L::splat(1.f), L::splat(0.f)};
        if ((m.starts | m.ends) == 0) {
            if (m.near0)
                runs_of(std::true_type{}, run, back, src);
            else
                runs_of(std::false_type{}, run, back, src);
        } else {
            for (int i = 0; i < kRows; ++i) {
                V a, b;
                step_of(std::false_type{}, src, i, a, b);
                run.q = fma2(a, (m.starts >> i) & 1u ? first_state(m.seq, i) : run.q, b);
                run.P = mul2(run.P, a);
            }
            for (int j = kRows - 1; j >= 0; --j) {
                const V a = decay<T>(L::unpack(src[j * 32])), d = L::unpack(src[2 * kSlotWords + j * 32]);
                back.q = mul2(a, add2(d, (m.ends >> j) & 1u ? last_adjoint(m.seq, j) : back.q));
            }
            back.P = m.ends ? L::splat(0.f) : run.P;
            if (m.starts) run.P = L::splat(0.f);
        }
    };
    auto publish = [&](const Marks &m, const Run<V> &run, const Run<V> &back) {
        fwd[warp][lane] = run;
        ex.warp[0][warp][lane] = back;
        if (lane == 0) {
            fwd_reset[warp] = m.starts;
            ex.warp_reset[0][warp] = m.ends;
        }
        ex.runs_published(0);
    };
    // EDGES: sequences begin or end among the rows.
    auto rows_of = [&](auto edges, auto near, const Marks &m, V state, V e, uint32_t *src) {
        constexpr bool EDGES = decltype(edges)::value;
        // forwards for the states, then backwards: dh = d + e, dx = s dh, d_log_gate = dh (a h_before + s' x)
        V a[kRows], slope[kRows];
        [[maybe_unused]] V s[MODE == SSE_INPUT_PLAIN ? 1 : kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (EDGES && ((m.starts >> i) & 1u)) state = first_state(m.seq, i);
            const V b = L::unpack(src[kSlotWords + i * 32]);
            V si, ds;
            factors<T, MODE, decltype(near)::value, true>(L::unpack(src[i * 32]), a[i], si, &ds);
            slope[i] = mul2(a[i], state);
            if constexpr (MODE == SSE_INPUT_PLAIN) {
                state = add2(slope[i], b);
            } else {
                s[i] = si;
                state = fma2(si, b, slope[i]);
                slope[i] = fma2(ds, b, slope[i]);
            }
        }
#pragma unroll
        for (int j = kRows - 1; j >= 0; --j) {
            if (EDGES && ((m.ends >> j) & 1u)) e = last_adjoint(m.seq, j);
            const V dh = add2(L::unpack(src[2 * kSlotWords + j * 32]), e);
            e = mul2(a[j], dh);
            V gx = dh;
            if constexpr (MODE != SSE_INPUT_PLAIN) gx = mul2(dh, s[j]);
            src[kSlotWords + j * 32] = L::pack(gx);
            src[2 * kSlotWords + j * 32] = L::pack(mul2(dh, slope[j]));
            if (EDGES && ((m.starts >> j) & 1u)) {
                const int q = __shfl_sync(0xffffffffu, m.seq, j);
                if (p.d_init && live) L::store_state(p.d_init + (int64_t)q * width + col, e);
            }
        }
    };
    auto second_pass = [&](const Marks &m, V state, V e, uint32_t *src) {
        if ((m.starts | m.ends) != 0)
            rows_of(std::true_type{}, std::false_type{}, m, state, e, src);
        else if (m.near0)
            rows_of(std::false_type{}, std::true_type{}, m, state, e, src);
        else
            rows_of(std::false_type{}, std::false_type{}, m, state, e, src);
        __syncwarp();
        store_rows<kRows>(p.dx, packed, col_byte, src - lane + kSlotWords, m.row0, sp.t0, sp.t1, m.whole, col_ok, lane);
        store_rows<kRows>(p.d_log_gate, packed, col_byte, src - lane + 2 * kSlotWords, m.row0, sp.t0, sp.t1, m.whole, col_ok, lane);
        __syncwarp();  // the slot is free
    };
    if (sp.steps > 0) {
        Marks now, next;
        Run<V> run, back;
        int slot = 0, row0 = first_row;
        for (int k = 0; k < kStagesBwd; ++k) load(k);
        copies_wait<kStagesBwd - 1>();
        first_pass(now, run, back, row0, mine + lane);
        publish(now, run, back);
        if (!ONE) cluster_arrive_relaxed();
        for (int step = 0; step < sp.steps; ++step) {
            const bool more = step + 1 < sp.steps;
            const int next_slot = slot + 1 == kStagesBwd ? 0 : slot + 1;
            if (more) {
                row0 -= stride;
                copies_wait<kStagesBwd - 2>();
                first_pass(next, run, back, row0, mine + next_slot * (3 * kSlotWords) + lane);
            }
            ex.await_starts(step, warp);
            const V e = ex.warp[0][warp][lane].P, state = fwd[warp][lane].P;
            if (!ONE) cluster_wait();
            if (more) {
                publish(next, run, back);
                if (!ONE) cluster_arrive_relaxed();
            }
            second_pass(now, state, e, mine + slot * (3 * kSlotWords) + lane);
            load(step + kStagesBwd);
            now = next;
            slot = next_slot;
        }
    }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 2) scan_backward_kernel(ScanArgs p, int width) {
    using L = Lane<T>;
    extern __shared__ uint4 ring[];
    __shared__ BackShared<typename L::V> sh;
    const int csize = cg::this_cluster().num_blocks(), rank = cg::this_cluster().block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col0 = (int)(blockIdx.x / csize) * 32 * L::kCols;
    const Span<kRowsBwd> sp(p, csize, rank, lane);
    if (sp.solo) {
        backward_tiles<T, MODE, true>(p, width, sp, sh, ring, 1, 0, col0);
    } else {
        cluster_arrive_relaxed();
        cluster_wait();
        backward_tiles<T, MODE, false>(p, width, sp, sh, ring, csize, rank, col0);
    }
    const int col = col0 + lane * L::kCols;
    if (p.d_init && col < width && warp < kWorkers) {  // empty sequences hand the final state's gradient through
        const int n = gridDim.y * csize * kWorkers;
        for (int q = ((int)blockIdx.y * csize + rank) * kWorkers + warp; q < p.num_seqs; q += n)
            if (__ldg(p.cu_seqlens + q) >= __ldg(p.cu_seqlens + q + 1)) {
                const int64_t i = (int64_t)q * width + col;
                L::store_state(p.d_init + i, p.d_final ? L::load_state(p.d_final + i) : L::splat(0.f));
            }
    }
}

// One token of each sequence: 16 bytes of a row per thread.
template <typename T, int MODE>
__global__ void __launch_bounds__(128) scan_step_kernel(ScanArgs p, int width, int words) {
    using L = Lane<T>;
    using V = typename L::V;
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    const int64_t row = i / words;
    if (row >= p.num_seqs) return;
    const int col = (int)(i - row * words) * (16 / (int)sizeof(T));
    const uint4 ux = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.x) + row * p.x_stride + col));
    const uint4 ug = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.log_gate) + row * p.gate_stride + col));
    const uint32_t x[4] = {ux.x, ux.y, ux.z, ux.w}, g[4] = {ug.x, ug.y, ug.z, ug.w};
    float *state = p.final_state + row * width + col;
    V h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = L::load_state(state + k * L::kCols);
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        V a, s, b = L::unpack(x[k]);
        factors<T, MODE, false>(L::unpack(g[k]), a, s);
        if constexpr (MODE != SSE_INPUT_PLAIN) b = mul2(b, s);
        h[k] = fma2(a, h[k], b);
        L::store_state(state + k * L::kCols, h[k]);
        o[k] = L::pack(h[k]);
    }
    *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + row * width + col) = make_uint4(o[0], o[1], o[2], o[3]);
}

enum What { kForward, kBackward, kStep };

// Clusters of c CTAs that the current device holds at a time, two CTAs per SM (a
// property of the device, asked for once: every kernel here has the same two).
int clusters_held(int c) {
    static std::atomic<int> known[16][kMaxCluster + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 16) return c == 1 ? 304 : 256 / c;
    int n = known[dev][c].load(std::memory_order_relaxed);
    if (n > 0) return n;
    const auto kernel = scan_forward_kernel<__nv_bfloat16, SSE_INPUT_PLAIN, kRemake>;
    constexpr int kSmem = kWorkers * kRowsFwd * 128 * 2 * kStagesFwd;
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = kSmem;
    cfg.gridDim = dim3(c);
    cfg.blockDim = kThreads;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)c, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        return c == 1 ? 304 : 256 / c;
    }
    known[dev][c].store(n, std::memory_order_relaxed);
    return n;
}

// Cluster size and ranges of the token axis: as many CTAs as the GPU holds at a
// time (a second wave of clusters would double the time: at 2560 channels and
// 20000 tokens, 40 clusters of 7 took 99 us where 40 of 6 take 72).  A GB300 held
// 304, 152, 97, 74, 58, 46, 38, 36 clusters of 1 to 8.  Larger clusters wait longer
// for each other; more ranges of whole sequences split uneven lengths less evenly.
// The two factors below are fitted to times of forwards and backwards at 2048
// channels: 72001 tokens in 16 sequences cut at random, s = sqrt(1 - a^2), 249, 224,
// 197, 240, 238 us with clusters of 8, 4, 3, 2, 1 in 1, 2, 3, 4, 8 ranges; in 5
// (32768 tokens) 114, 107, 107, 143 with 8, 4, 3, 2.  (Clusters of 1 are rated far
// below what they took there.)  The host knows how many sequences there are and not
// how long: a batch in which one has 90 % of 72000 tokens beside 15 short ones gets
// the clusters of 3 that suit even ones, 231 to 306 us forward and 481 to 531
// backward, where that sequence alone would get clusters of 8.
void choose_clusters(int columns, int64_t tiles, int num_seqs, int &csize, int &ranges) {
    double best = 0;
    for (int c = kMaxCluster; c >= 1; --c) {
        const int held = clusters_held(c);
        if (c > 1 && (columns > held || c > tiles)) continue;
        int64_t r = held / columns;
        if (r > num_seqs) r = num_seqs;
        if (r > tiles / c) r = tiles / c;
        if (r < 1) r = 1;
        const double rate = (double)columns * c * r / ((1 + 0.04 * c) * (r > 1 ? 1 + 0.06 * r * r * r / num_seqs : 1));
        if (rate > best) {
            best = rate;
            csize = c;
            ranges = (int)r;
        }
    }
}

struct Choice {
    int csize, ranges, form;  // form: of the forward's rows
};

Choice choose(const sse_scan_config_t &cfg, bool forward, int64_t total_tokens, int num_seqs) {
    const int columns = (cfg.width * (cfg.dtype == SSE_BF16 ? 2 : 4) + 127) / 128;
    const int tile = kWorkers * (forward ? kRowsFwd : kRowsBwd);
    Choice c{1, 1, kRemake};
    choose_clusters(columns, (total_tokens + tile - 1) / tile, num_seqs, c.csize, c.ranges);
    // held: costly bf16 input factors with two CTAs on a quarter of the SMs or more
    if (cfg.input_scale != SSE_INPUT_PLAIN && cfg.dtype == SSE_BF16 && columns * c.csize * c.ranges >= 192)
        c.form = c.csize >= 7 ? kHold : kHoldAlone;
    return c;
}

template <typename T, int MODE>
cudaError_t launch_t(What what, const sse_scan_config_t &scan, const ScanArgs &a, cudaStream_t stream) {
    const int width = scan.width;
    if (what == kStep) {
        const int words = width * (int)sizeof(T) / 16;
        const int64_t blocks = ((int64_t)a.num_seqs * words + 127) / 128;
        if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
        scan_step_kernel<T, MODE><<<(unsigned)blocks, 128, 0, stream>>>(a, width, words);
        return cudaGetLastError();
    }
    const int columns = (width + 32 * Lane<T>::kCols - 1) / (32 * Lane<T>::kCols);
    const int tile = kWorkers * (what == kForward ? kRowsFwd : kRowsBwd);
    const Choice c = choose(scan, what == kForward, a.total_tokens, a.num_seqs);
    constexpr bool kHeavy = MODE != SSE_INPUT_PLAIN && sizeof(T) == 2;
    const auto kernel = what == kBackward      ? scan_backward_kernel<T, MODE>
                        : c.form == kHold      ? scan_forward_kernel<T, MODE, kHeavy ? kHold : kRemake>
                        : c.form == kHoldAlone ? scan_forward_kernel<T, MODE, kHeavy ? kHoldAlone : kRemake>
                                               : scan_forward_kernel<T, MODE, kRemake>;
    const size_t smem = (size_t)tile * 128 * (what == kForward ? 2 * kStagesFwd : 3 * kStagesBwd);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = smem;
    cfg.gridDim = dim3(columns * c.csize, c.ranges);
    cfg.blockDim = kThreads;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)c.csize, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, width);
}

template <typename T>
cudaError_t launch_mode(What what, const sse_scan_config_t &cfg, const ScanArgs &a, cudaStream_t stream) {
    switch (cfg.input_scale) {
    case SSE_INPUT_PLAIN: return launch_t<T, SSE_INPUT_PLAIN>(what, cfg, a, stream);
    case SSE_INPUT_COMPLEMENT: return launch_t<T, SSE_INPUT_COMPLEMENT>(what, cfg, a, stream);
    default: return launch_t<T, SSE_INPUT_UNIT>(what, cfg, a, stream);
    }
}

cudaError_t launch(What what, const sse_scan_config_t &cfg, const ScanArgs &a, cudaStream_t stream) {
    return cfg.dtype == SSE_BF16 ? launch_mode<__nv_bfloat16>(what, cfg, a, stream)
                                 : launch_mode<float>(what, cfg, a, stream);
}

}  // namespace

cudaError_t launch_scan_forward(const sse_scan_config_t &cfg, const ScanArgs &a, cudaStream_t stream) {
    return launch(kForward, cfg, a, stream);
}
cudaError_t launch_scan_backward(const sse_scan_config_t &cfg, const ScanArgs &a, cudaStream_t stream) {
    return launch(kBackward, cfg, a, stream);
}
cudaError_t launch_scan_step(const sse_scan_config_t &cfg, const ScanArgs &a, cudaStream_t stream) {
    return launch(kStep, cfg, a, stream);
}

}  // namespace sse

// What a forward of these sizes takes, for tests: its form, and the clusters.  Not part of the ABI.
extern "C" int sse_debug_scan_form(const sse_scan_config_t *cfg, int32_t total_tokens, int32_t num_seqs, int32_t *csize,
                                   int32_t *ranges) {
    const sse::Choice c = sse::choose(*cfg, true, total_tokens, num_seqs);
    *csize = c.csize;
    *ranges = c.ranges;
    return c.form;
}
