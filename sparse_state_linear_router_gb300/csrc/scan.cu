// scan.cu -- the gated linear recurrence h_t = a_t h_{t-1} + s(a_t) x_t, one
// state per channel: forward, backward and one step.
//
// A run of steps composes to h -> P h + q (P the product of its decays, q what
// it makes of a zero state), and runs compose in order, so a long sequence is
// split over warps and CTAs: each makes its rows' (P, q), the runs ahead are
// composed to the state the rows start from, and the rows are gone through
// again from that state.  Rows stay in registers between the two, so HBM is
// read once and written once.
//
//  - A lane has 4 bytes of a row (two bf16 channels, or one float32), a warp
//    one 128-byte line of each of kRows consecutive rows, a CTA 8 x kRows rows.
//  - The CTAs of a cluster take consecutive tiles of the same 128-byte column
//    and hand their (P, q) to each other through distributed shared memory;
//    then the cluster moves on by its size.  Nothing waits on global memory, no
//    workspace, and the order of every product and sum is fixed.
//  - The batch's packed token axis is one axis: a sequence's first row starts
//    from its own initial state (a reset: P = 0), its last one writes the final
//    state, so uneven lengths cost nothing.  A reset is a select and no
//    product with zero: a NaN of one sequence does not reach the next.
//  - Loads of the next tile are issued before the cluster's barrier.
//
// Bound by HBM: 6 bytes and about 20 (plain) to 45 (unit) instructions per two
// bf16 channels forward, 10 bytes backward.
#include <type_traits>

#include <cooperative_groups.h>

#include "f32x2.cuh"
#include "sse_internal.cuh"

namespace sse {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;  // the portable cluster size
constexpr int kSms = 152;
constexpr int kRowsFwd = 16;  // rows per warp and tile
constexpr int kRowsBwd = 8;
static_assert(kWarps * kRowsBwd == kScanCheckpoint, "the backward's tiles start at checkpoints");
static_assert((kWarps * kRowsFwd) % kScanCheckpoint == 0, "checkpoints are at warps' first rows");

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
template <typename F> __device__ __forceinline__ F2 each(F2 x, F2 y, F f) {
    const float2 v = f2_get(x), w = f2_get(y);
    return f2(f(v.x, w.x), f(v.y, w.y));
}
template <typename F> __device__ __forceinline__ float each(float x, float y, F f) { return f(x, y); }
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

// a = exp(la) = 2^(la log2 e).  The product's rounding error, |la| 2^-24 of the
// result, is put back to first order: 2^(t + r) = 2^t (1 + r ln 2).  Below
// e^-150 (the least float32 is e^-103) the result is 0; -infinity stops there.
template <typename T> __device__ __forceinline__ typename Lane<T>::V decay(typename Lane<T>::V la) {
    using L = Lane<T>;
    la = each(la, [](float x) { return max_nan(x, -150.f); });
    const auto t = mul2(la, L::splat(1.44269504f));
    auto r = fma2(la, L::splat(1.44269504f), each(t, [](float x) { return -x; }));
    r = fma2(la, L::splat(1.92596303e-8f), r);  // log2 e - 1.44269504f
    const auto a = each(t, [](float x) { return ex2(x); });
    return fma2(a, mul2(r, L::splat(0.693147181f)), a);
}

// 1 - exp(u) for u <= 0, e = exp(u): its Taylor series up to u^8 / 8! for u >
// -1/2 (the next term is 10^-8 of the sum), where 1 - e would cancel.
template <typename T>
__device__ __forceinline__ typename Lane<T>::V one_minus_exp(typename Lane<T>::V u, typename Lane<T>::V e) {
    using L = Lane<T>;
    auto p = L::splat(-1.f / 40320);
    p = fma2(p, u, L::splat(-1.f / 5040));
    p = fma2(p, u, L::splat(-1.f / 720));
    p = fma2(p, u, L::splat(-1.f / 120));
    p = fma2(p, u, L::splat(-1.f / 24));
    p = fma2(p, u, L::splat(-1.f / 6));
    p = fma2(p, u, L::splat(-1.f / 2));
    p = fma2(p, u, L::splat(-1.f));
    p = mul2(p, u);
    return each(u, p, e, [](float x, float series, float ex) { return x > -0.5f ? series : 1.f - ex; });
}

// The input factor s(a) of MODE (sse_input_scale_t; not for PLAIN).
template <typename T, int MODE>
__device__ __forceinline__ typename Lane<T>::V input_factor(typename Lane<T>::V la, typename Lane<T>::V a) {
    if constexpr (MODE == SSE_INPUT_COMPLEMENT) {
        return one_minus_exp<T>(la, a);
    } else {
        const auto s2 = one_minus_exp<T>(add2(la, la), mul2(a, a));
        return each(s2, [](float v) { return v * rsqrtf(fmaxf(v, 1e-37f)); });  // 0 at 0
    }
}

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

// The packed tokens of one cluster: from the first sequence start at or after
// the range's share of the tokens to that of the next range.
__device__ __forceinline__ int range_start(const ScanArgs &p, int r, int ranges) {
    const int T = p.total_tokens, S = p.num_seqs;
    if (r >= ranges) return clamp_token(__ldg(p.cu_seqlens + S), T);
    if (r == 0) return clamp_token(__ldg(p.cu_seqlens), T);
    const int t = (int)((int64_t)T * r / ranges);
    const int s = sequence_of(p.cu_seqlens, S, t - 1) + 1;  // the first with cu[s] >= t
    return clamp_token(__ldg(p.cu_seqlens + (s < S ? s : S)), T);
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

// ROWS rows of one token tensor, the lane's 4 bytes of each; zeros outside
// [t0, t1) (decay 1, input 0: such rows change nothing).
template <typename T, int ROWS>
__device__ __forceinline__ void load_rows(uint32_t (&u)[ROWS], const void *base, int64_t stride, int col, int row0,
                                          int t0, int t1, bool live) {
    const T *q = static_cast<const T *>(base) + (int64_t)row0 * stride + col;
    if (row0 >= t0 && row0 + ROWS <= t1) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) u[i] = live ? __ldg(reinterpret_cast<const uint32_t *>(q + i * stride)) : 0u;
    } else {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            u[i] = live && row0 + i >= t0 && row0 + i < t1 ? __ldg(reinterpret_cast<const uint32_t *>(q + i * stride))
                                                           : 0u;
    }
}

// What the warps and CTAs tell each other, in two buffers in turn: one step's
// runs are read while the next step's are written.
template <typename V> struct Exchange {
    Run<V> warp[2][kWarps][32];
    Run<V> cta[2][kMaxCluster][32];
    uint32_t warp_reset[2][kWarps];
    uint32_t cta_reset[2][kMaxCluster];
};

// Bits of the warps (or CTAs) whose run holds a reset.
__device__ __forceinline__ uint32_t reset_bits(const uint32_t *flags, int n, int lane) {
    return __ballot_sync(0xffffffffu, lane < n && flags[lane] != 0);
}

// Applies run r to a state; a reset leaves q alone.
template <typename V> __device__ __forceinline__ V apply(const Run<V> &r, V h, bool reset) {
    return reset ? r.q : fma2(r.P, h, r.q);
}
// `first`, then r; `reset`: r holds a reset.
template <typename V> __device__ __forceinline__ void append(Run<V> &first, const Run<V> &r, bool reset) {
    first.q = apply(r, first.q, reset);
    first.P = mul2(first.P, r.P);
}

// Hands this CTA's run to every CTA of the cluster (one warp calls it).
template <typename V>
__device__ __forceinline__ void tell_cluster(cg::cluster_group &cluster, Exchange<V> &ex, int buf, int rank, int csize,
                                             const Run<V> &r, bool reset, int lane) {
    for (int k = 0; k < csize; ++k) {
        *cluster.map_shared_rank(&ex.cta[buf][rank][lane], k) = r;
        if (lane == 0) *cluster.map_shared_rank(&ex.cta_reset[buf][rank], k) = reset;
    }
}

// The state the CTA's tile starts from; `state` moves on past the cluster's tiles.
template <typename V>
__device__ __forceinline__ V through_cluster(const Exchange<V> &ex, int buf, int rank, int csize, V &state, int lane) {
    const uint32_t resets = reset_bits(ex.cta_reset[buf], csize, lane);
    V mine = state;
    for (int k = 0; k < csize; ++k) {
        if (k == rank) mine = state;
        state = apply(ex.cta[buf][k][lane], state, (resets >> k) & 1u);
    }
    return mine;
}

// ---------------------------------------------------------------------------
// Forward.  grid.x: column x cluster rank, grid.y: ranges of the token axis.
// ---------------------------------------------------------------------------
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 2) scan_forward_kernel(ScanArgs p, int width) {
    using L = Lane<T>;
    using V = typename L::V;
    constexpr int R = kRowsFwd;
    __shared__ Exchange<V> ex;
    cg::cluster_group cluster = cg::this_cluster();
    const int csize = cluster.num_blocks(), rank = cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = ((int)(blockIdx.x / csize) * 32 + lane) * L::kCols;
    const bool live = col < width;
    if (csize > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // every CTA has started

    const int t0 = range_start(p, blockIdx.y, gridDim.y), t1 = range_start(p, blockIdx.y + 1, gridDim.y);
    constexpr int kTile = kWarps * R;
    const int tile0 = t0 / kTile;
    const int tiles = t1 > t0 ? (t1 + kTile - 1) / kTile - tile0 : 0;
    const int steps = (tiles + csize - 1) / csize;

    uint32_t xr[R], gr[R];
    int row0 = (tile0 + rank) * kTile + warp * R;
    if (steps > 0) {
        load_rows<T, R>(gr, p.log_gate, p.gate_stride, col, row0, t0, t1, live);
        load_rows<T, R>(xr, p.x, p.x_stride, col, row0, t0, t1, live);
    }
    if (csize > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");

    V state = L::splat(0.f);  // the state ahead of the cluster's tiles
    Edges<R> ed;
    ed.lo = ed.hi = 0;
    for (int step = 0; step < steps; ++step) {
        const int buf = step & 1;
        V a[R], b[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const V la = L::unpack(gr[i]);
            a[i] = decay<T>(la);
            b[i] = L::unpack(xr[i]);
            if constexpr (MODE != SSE_INPUT_PLAIN) b[i] = mul2(b[i], input_factor<T, MODE>(la, a[i]));
        }
        const int next = row0 + csize * kTile;
        if (step + 1 < steps) {
            load_rows<T, R>(gr, p.log_gate, p.gate_stride, col, next, t0, t1, live);
            load_rows<T, R>(xr, p.x, p.x_stride, col, next, t0, t1, live);
        }
        ed.find(p, row0, t0, t1, lane);
        Run<V> run{L::splat(1.f), L::splat(0.f)};
        if (ed.starts == 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                run.q = fma2(a[i], run.q, b[i]);
                run.P = mul2(run.P, a[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if ((ed.starts >> i) & 1u) {
                    // the initial state enters here and is not read again: it may be the final state's buffer
                    const int s = __shfl_sync(0xffffffffu, ed.seq, i);
                    const V init = p.init && live ? L::load_state(p.init + (int64_t)s * width + col) : L::splat(0.f);
                    b[i] = fma2(a[i], init, b[i]);
                    run.q = b[i];
                    run.P = L::splat(0.f);
                } else {
                    run.q = fma2(a[i], run.q, b[i]);
                    run.P = mul2(run.P, a[i]);
                }
            }
        }
        ex.warp[buf][warp][lane] = run;
        if (lane == 0) ex.warp_reset[buf][warp] = ed.starts;
        __syncthreads();
        const uint32_t resets = reset_bits(ex.warp_reset[buf], kWarps, lane);
        Run<V> ahead{L::splat(1.f), L::splat(0.f)};  // the CTA's warps before this one
        for (int w = 0; w < warp; ++w) append(ahead, ex.warp[buf][w][lane], (resets >> w) & 1u);
        if (warp == kWarps - 1) {
            Run<V> all = ahead;
            append(all, run, ed.starts != 0);
            if (csize > 1)
                tell_cluster(cluster, ex, buf, rank, csize, all, resets != 0, lane);
            else
                ex.cta[buf][0][lane] = all, ex.cta_reset[buf][0] = resets != 0;
        }
        if (csize > 1) {
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        } else {
            __syncthreads();
        }
        V h = through_cluster(ex, buf, rank, csize, state, lane);
        h = apply(ahead, h, (resets & ((1u << warp) - 1u)) != 0);
        if (p.checkpoints && live && row0 % kScanCheckpoint == 0 && row0 >= t0 && row0 < t1)
            L::store_state(p.checkpoints + (int64_t)(row0 / kScanCheckpoint) * width + col, h);
        T *out = static_cast<T *>(p.out) + (int64_t)row0 * width + col;
        if ((ed.starts | ed.ends) == 0 && row0 >= t0 && row0 + R <= t1) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                h = fma2(a[i], h, b[i]);
                if (live) *reinterpret_cast<uint32_t *>(out + (int64_t)i * width) = L::pack(h);
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                h = (ed.starts >> i) & 1u ? b[i] : fma2(a[i], h, b[i]);
                if (live && row0 + i >= t0 && row0 + i < t1)
                    *reinterpret_cast<uint32_t *>(out + (int64_t)i * width) = L::pack(h);
                if ((ed.ends >> i) & 1u) {
                    const int s = __shfl_sync(0xffffffffu, ed.seq, i);
                    if (p.final_state && live) L::store_state(p.final_state + (int64_t)s * width + col, h);
                }
            }
        }
        row0 = next;
    }
    // empty sequences keep their initial state
    if (p.final_state && live) {
        const int n = gridDim.y * csize * kWarps;
        for (int s = ((int)blockIdx.y * csize + rank) * kWarps + warp; s < p.num_seqs; s += n)
            if (__ldg(p.cu_seqlens + s) >= __ldg(p.cu_seqlens + s + 1)) {
                const int64_t i = (int64_t)s * width + col;
                L::store_state(p.final_state + i, p.init ? L::load_state(p.init + i) : L::splat(0.f));
            }
    }
}

// ---------------------------------------------------------------------------
// Backward: the tiles from the last to the first.  A tile's states come from
// its checkpoint and the CTA's own rows; what later tokens hand back,
// e_t = a_t (d_out_t + e_{t+1}), is the same kind of run in the other
// direction and goes through the cluster.
// ---------------------------------------------------------------------------
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads, 2) scan_backward_kernel(ScanArgs p, int width) {
    using L = Lane<T>;
    using V = typename L::V;
    constexpr int R = kRowsBwd;
    __shared__ Exchange<V> ex;                   // adjoint runs
    __shared__ Run<V> fwd[2][kWarps][32];        // state runs of the CTA's warps
    __shared__ uint32_t fwd_reset[2][kWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int csize = cluster.num_blocks(), rank = cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = ((int)(blockIdx.x / csize) * 32 + lane) * L::kCols;
    const bool live = col < width;
    if (csize > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    const int t0 = range_start(p, blockIdx.y, gridDim.y), t1 = range_start(p, blockIdx.y + 1, gridDim.y);
    constexpr int kTile = kWarps * R;
    const int tile0 = t0 / kTile;
    const int tiles = t1 > t0 ? (t1 + kTile - 1) / kTile - tile0 : 0;
    const int steps = (tiles + csize - 1) / csize;

    uint32_t xr[R], gr[R], dr[R];
    V check = L::splat(0.f);  // the state ahead of the tile
    // rank 0 has the last tile; a tile below tile0 has no rows in [t0, t1)
    auto load = [&](int tile) {
        const int row = tile * kTile + warp * R;
        load_rows<T, R>(gr, p.log_gate, p.gate_stride, col, row, t0, t1, live);
        load_rows<T, R>(xr, p.x, p.x_stride, col, row, t0, t1, live);
        load_rows<T, R>(dr, p.d_out, width, col, row, t0, t1, live);
        check = live && tile * kTile > t0 ? L::load_state(p.checkpoints + (int64_t)tile * width + col) : L::splat(0.f);
    };
    int tile = tile0 + tiles - 1 - rank;
    if (steps > 0) load(tile);
    if (csize > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");

    V adjoint = L::splat(0.f);  // what the tokens behind the cluster's tiles hand back
    Edges<R> ed;
    ed.lo = ed.hi = 0;
    for (int step = 0; step < steps; ++step) {
        const int buf = step & 1, row0 = tile * kTile + warp * R;
        V a[R], h[R], s[MODE == SSE_INPUT_PLAIN ? 1 : R];  // h: first the inputs s x, then the states before each row
        uint32_t x[R], d[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const V la = L::unpack(gr[i]);
            a[i] = decay<T>(la);
            x[i] = xr[i];
            d[i] = dr[i];
            h[i] = L::unpack(x[i]);
            if constexpr (MODE != SSE_INPUT_PLAIN) {
                s[i] = input_factor<T, MODE>(la, a[i]);
                h[i] = mul2(h[i], s[i]);
            }
        }
        V state = check;
        if (step + 1 < steps) load(tile - csize);
        ed.find(p, row0, t0, t1, lane);
        const uint32_t starts = ed.starts, ends = ed.ends;
        auto first_state = [&](int i) {
            const int sq = __shfl_sync(0xffffffffu, ed.seq, i);
            return p.init && live ? L::load_state(p.init + (int64_t)sq * width + col) : L::splat(0.f);
        };
        auto last_adjoint = [&](int i) {
            const int sq = __shfl_sync(0xffffffffu, ed.seq, i);
            return p.d_final && live ? L::load_state(p.d_final + (int64_t)sq * width + col) : L::splat(0.f);
        };
        Run<V> run{L::splat(1.f), L::splat(0.f)}, back{L::splat(1.f), L::splat(0.f)};
        if ((starts | ends) == 0) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                run.q = fma2(a[i], run.q, h[i]);
                run.P = mul2(run.P, a[i]);
                const int j = R - 1 - i;
                back.q = mul2(a[j], add2(L::unpack(d[j]), back.q));
            }
            back.P = run.P;
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                run.q = fma2(a[i], (starts >> i) & 1u ? first_state(i) : run.q, h[i]);
                run.P = mul2(run.P, a[i]);
                const int j = R - 1 - i;
                back.q = mul2(a[j], add2(L::unpack(d[j]), (ends >> j) & 1u ? last_adjoint(j) : back.q));
            }
            back.P = run.P;
            if (starts) run.P = L::splat(0.f);
            if (ends) back.P = L::splat(0.f);
        }
        fwd[buf][warp][lane] = run;
        ex.warp[buf][warp][lane] = back;
        if (lane == 0) {
            fwd_reset[buf][warp] = starts;
            ex.warp_reset[buf][warp] = ends;
        }
        __syncthreads();
        const uint32_t fresets = reset_bits(fwd_reset[buf], kWarps, lane);
        const uint32_t bresets = reset_bits(ex.warp_reset[buf], kWarps, lane);
        Run<V> behind{L::splat(1.f), L::splat(0.f)};  // the CTA's warps of later rows
        for (int w = kWarps - 1; w > warp; --w) append(behind, ex.warp[buf][w][lane], (bresets >> w) & 1u);
        if (warp == 0) {
            Run<V> all = behind;
            append(all, back, ends != 0);
            if (csize > 1)
                tell_cluster(cluster, ex, buf, rank, csize, all, bresets != 0, lane);
            else
                ex.cta[buf][0][lane] = all, ex.cta_reset[buf][0] = bresets != 0;
        }
        if (csize > 1)
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        // the states before each row, while the cluster gathers
        for (int w = 0; w < warp; ++w) state = apply(fwd[buf][w][lane], state, (fresets >> w) & 1u);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const V in = h[i];
            if ((starts >> i) & 1u) state = first_state(i);
            h[i] = state;
            state = fma2(a[i], state, in);
        }
        if (csize > 1)
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        else
            __syncthreads();
        V e = through_cluster(ex, buf, rank, csize, adjoint, lane);
        e = apply(behind, e, (bresets >> (warp + 1)) != 0);
        const int64_t at = (int64_t)row0 * width + col;
        T *dx = static_cast<T *>(p.dx) + at, *dg = static_cast<T *>(p.d_log_gate) + at;
        const bool whole = row0 >= t0 && row0 + R <= t1;
#pragma unroll
        for (int j = R - 1; j >= 0; --j) {
            if ((ends >> j) & 1u) e = last_adjoint(j);
            const V dh = add2(L::unpack(d[j]), e);
            e = mul2(a[j], dh);
            V gx = dh, slope = mul2(a[j], h[j]);
            if constexpr (MODE != SSE_INPUT_PLAIN) {
                gx = mul2(dh, s[j]);
                const V ds = MODE == SSE_INPUT_COMPLEMENT
                                 ? each(a[j], [](float v) { return -v; })
                                 : each(a[j], s[j], [](float v, float f) { return f > 0.f ? __fdividef(-v * v, f) : 0.f; });
                slope = fma2(ds, L::unpack(x[j]), slope);
            }
            if (live && (whole || (row0 + j >= t0 && row0 + j < t1))) {
                *reinterpret_cast<uint32_t *>(dx + (int64_t)j * width) = L::pack(gx);
                *reinterpret_cast<uint32_t *>(dg + (int64_t)j * width) = L::pack(mul2(dh, slope));
            }
            if ((starts >> j) & 1u) {
                const int sq = __shfl_sync(0xffffffffu, ed.seq, j);
                if (p.d_init && live) L::store_state(p.d_init + (int64_t)sq * width + col, e);
            }
        }
        tile -= csize;
    }
    if (p.d_init && live) {  // empty sequences hand the final state's gradient through
        const int n = gridDim.y * csize * kWarps;
        for (int q = ((int)blockIdx.y * csize + rank) * kWarps + warp; q < p.num_seqs; q += n)
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
        const V la = L::unpack(g[k]), a = decay<T>(la);
        V b = L::unpack(x[k]);
        if constexpr (MODE != SSE_INPUT_PLAIN) b = mul2(b, input_factor<T, MODE>(la, a));
        h[k] = fma2(a, h[k], b);
        L::store_state(state + k * L::kCols, h[k]);
        o[k] = L::pack(h[k]);
    }
    *reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + row * width + col) = make_uint4(o[0], o[1], o[2], o[3]);
}

enum What { kForward, kBackward, kStep };

template <typename T, int MODE>
cudaError_t launch_t(What what, const ScanArgs &a, int width, cudaStream_t stream) {
    if (what == kStep) {
        const int words = width * (int)sizeof(T) / 16;
        const int64_t blocks = ((int64_t)a.num_seqs * words + 127) / 128;
        if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
        scan_step_kernel<T, MODE><<<(unsigned)blocks, 128, 0, stream>>>(a, width, words);
        return cudaGetLastError();
    }
    // As many CTAs as the GPU holds (two per SM): the cluster takes what the
    // columns leave, but no more tiles than there are; with fewer columns the
    // token axis is split into ranges of whole sequences as well.
    const int columns = (width + 32 * Lane<T>::kCols - 1) / (32 * Lane<T>::kCols);
    const int tile = kWarps * (what == kForward ? kRowsFwd : kRowsBwd);
    const int64_t tiles = ((int64_t)a.total_tokens + tile - 1) / tile;
    int csize = 2 * kSms / columns;
    csize = csize > kMaxCluster ? kMaxCluster : csize < 1 ? 1 : csize;
    if (csize > tiles) csize = tiles < 1 ? 1 : (int)tiles;
    int64_t ranges = 2 * kSms / (columns * csize);
    if (ranges > a.num_seqs) ranges = a.num_seqs;
    if (ranges > tiles / csize) ranges = tiles / csize;
    if (ranges < 1) ranges = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(columns * csize, (unsigned)ranges);
    cfg.blockDim = kThreads;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)csize, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, what == kForward ? scan_forward_kernel<T, MODE> : scan_backward_kernel<T, MODE>, a,
                              width);
}

template <typename T>
cudaError_t launch_mode(What what, const sse_scan_config_t &cfg, const ScanArgs &a, cudaStream_t stream) {
    switch (cfg.input_scale) {
    case SSE_INPUT_PLAIN: return launch_t<T, SSE_INPUT_PLAIN>(what, a, cfg.width, stream);
    case SSE_INPUT_COMPLEMENT: return launch_t<T, SSE_INPUT_COMPLEMENT>(what, a, cfg.width, stream);
    default: return launch_t<T, SSE_INPUT_UNIT>(what, a, cfg.width, stream);
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
