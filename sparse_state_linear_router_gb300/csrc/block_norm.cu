// block_norm.cu -- the norms before and after a block, fused with the block's
// gate, the channel scale and the residual stream:
//   r' = residual_scale r + branch_scale c act(z) o_hat w_after,
//        o_hat = o rstd_group,  rstd = rsqrt(mean u^2 + eps)
//   x' = r_hat w_before,        r_hat = r' rstd_row
// Gradients, with p = dr' branch_scale c w_after:
//   dr'  = d_residual_out + rstd_row (dx' w_before - r_hat mean(dx' w_before r_hat))
//   d_r  = residual_scale dr'
//   dz   = p o_hat act'(z),   d_oh = p act(z)
//   do   = rstd_group (d_oh - o_hat mean_group(d_oh o_hat))
//   C_j  = sum over tokens of dr' act(z) o_hat:  dw_after = branch_scale c C,
//          dc = branch_scale w_after C;  dw_before_j = sum of dx' r_hat
//
// Bound by HBM: about 16 to 40 operations per element against 4 to 16 bytes.
// A team of threads covers a row, 16 bytes per thread and tensor, and goes from
// row to row; each thread copies its own words of the rows ahead to shared
// memory asynchronously (no barrier: nobody else reads them), so the loads of
// the next rows are in flight while this one is summed.  Sums over the row go
// through shuffles and one word per warp of shared memory; sums over a group of
// columns through shuffles where the group is a power of two of lanes.
#include "f32x2.cuh"
#include "sse_internal.cuh"

namespace sse {
namespace {

constexpr int kSms = 152;

// How the sum of squares of the norm after the block is shared.
enum { kGroupNone, kGroupRow, kGroupShuffle, kGroupShared };

// One 16-byte word of a row as float32 pairs.
template <typename T> struct Row {
    static constexpr int kE = 16 / sizeof(T);  // elements
    static constexpr int kP = kE / 2;          // pairs
    static __device__ __forceinline__ void unpack(uint4 u, F2 (&f)[kP]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            if constexpr (sizeof(T) == 2)
                f[i] = f2_bits(w[i] << 16, w[i] & 0xffff0000u);
            else
                f[i] = f2_bits(w[2 * i], w[2 * i + 1]);
        }
    }
    static __device__ __forceinline__ void store(void *base, int64_t i, const F2 (&f)[kP]) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < kP; ++k) {
            const float2 v = f2_get(f[k]);
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
                w[k] = *reinterpret_cast<const uint32_t *>(&b);
            } else {
                w[2 * k] = __float_as_uint(v.x);
                w[2 * k + 1] = __float_as_uint(v.y);
            }
        }
        *reinterpret_cast<uint4 *>(static_cast<T *>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ F2 both(float x) { return f2(x, x); }

// 1 / (1 + exp(-z))
__device__ __forceinline__ F2 sigmoid2(F2 z) {
    const float2 t = f2_get(mul2(z, both(-1.44269504f)));
    float ex, ey, x, y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ex) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ey) : "f"(t.y));
    const float2 u = f2_get(add2(f2(ex, ey), both(1.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(u.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(u.y));
    return f2(x, y);
}

// act(z) of one word in the place of z, and with GRAD its derivative.
template <bool GRAD, int P> __device__ __forceinline__ void act(int gate, F2 (&z)[P], F2 (&d)[P]) {
    if (gate == SSE_GATE_SILU) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const F2 s = sigmoid2(z[i]);
            if (GRAD) d[i] = mul2(s, fma2(z[i], fma2(s, both(-1.f), both(1.f)), both(1.f)));
            z[i] = mul2(z[i], s);
        }
    } else if (gate == SSE_GATE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            z[i] = sigmoid2(z[i]);
            if (GRAD) d[i] = mul2(z[i], fma2(z[i], both(-1.f), both(1.f)));
        }
    } else if (GRAD) {
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = both(1.f);
    }
}

__device__ __forceinline__ float fold(F2 v) {
    const float2 f = f2_get(v);
    return f.x + f.y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The team of one row: blockDim.x threads (whole warps), blockDim.y rows per
// CTA.  Every thread of the CTA makes the same calls (they synchronize).
struct Team {
    float *warp_words;  // [2][rows][2][32]: this row's words, two buffers in turn; zero behind the last warp
    float *vec_words;   // [rows][words of a row]: kGroupShared only
    int turn;
    __device__ __forceinline__ void clear() {  // before the first sum
        for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 4 * 32 * (int)blockDim.y; i += blockDim.x * blockDim.y)
            warp_words[i] = 0.f;
        __syncthreads();
    }
    __device__ __forceinline__ float gather(const float *w) const {
        float s = 0.f;
        for (int k = 0; k < (int)blockDim.x >> 5; k += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(w + k);
            s += (v.x + v.y) + (v.z + v.w);
        }
        return s;
    }
    // Sums of N (1 or 2) values per thread over the team.
    template <int N> __device__ __forceinline__ void row_sum(float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
        if (blockDim.x == 32) return;
        float *w = warp_words + (turn * blockDim.y + threadIdx.y) * 64;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) w[i * 32 + (threadIdx.x >> 5)] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = gather(w + i * 32);
    }
};

// Sums over each group of the row; in: per 16-byte word v (0 for a word past
// the row), out: the sum of the word's group.  gw: words of a group.
template <int VPT>
__device__ __forceinline__ void group_sum(Team &tm, int mode, int gw, int nv, float (&v)[VPT]) {
    if (mode == kGroupRow) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) s += v[i];
        float t[1] = {s};
        tm.row_sum<1>(t);
#pragma unroll
        for (int i = 0; i < VPT; ++i) v[i] = t[0];
    } else if (mode == kGroupShuffle) {  // a power of two of neighbouring lanes
        for (int o = gw >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < VPT; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    } else {
        float *w = tm.vec_words + threadIdx.y * nv;
        __syncthreads();  // the sums of the call before have been read
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (j < nv) w[j] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (j < nv) {
                const int j0 = j / gw * gw;
                float s = 0.f;
                for (int k = 0; k < gw; ++k) s += w[j0 + k];
                v[i] = s;
            }
        }
    }
}

struct NormShape {
    int width, nv;       // columns and 16-byte words of a row
    int mode, gw;        // group mode, words of a group
    int stages;          // rows of a thread's ring
    int gate;
    float eps, rs, bs;
    float inv_width, inv_group;
};

// A thread's ring of rows: `tensors` tensors x VPT words per row.  The slot of a
// row is free again when its words have been taken to registers.
template <typename T, int VPT> struct Ring {
    uint32_t at;          // this thread's first word in shared memory
    int words, stages;    // words of one stage in the CTA's ring, stages
    int threads;
    __device__ __forceinline__ Ring(const void *smem, int tensors, int n_stages) {
        threads = blockDim.x * blockDim.y;
        at = (uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
        words = tensors * VPT * threads;
        stages = n_stages;
    }
    __device__ __forceinline__ uint32_t slot(int stage, int tensor, int i) const {
        return at + (stage * words + (tensor * VPT + i) * threads) * 16;
    }
    // Copies the thread's words of one tensor's row (zeros past its end).
    __device__ __forceinline__ void fetch(int stage, int tensor, const void *base, int64_t first, int nv, bool live) const {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            const bool ok = live && j < nv;
            const T *src = static_cast<const T *>(base) + (ok ? first + j * Row<T>::kE : 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot(stage, tensor, i)), "l"(src),
                         "r"(ok ? 16 : 0) : "memory");
        }
    }
    __device__ __forceinline__ uint4 take(int stage, int tensor, int i) const {
        uint4 u;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(slot(stage, tensor, i)) : "memory");
        return u;
    }
};
__device__ __forceinline__ void fetches_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for the oldest of `stages` groups.
__device__ __forceinline__ void fetches_wait(int stages) {
    if (stages == 3)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 2)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// coef = branch_scale c w_after of the thread's columns, and w_before
template <typename T, int VPT>
__device__ __forceinline__ void load_coef(const BlockNormArgs &a, const NormShape &n, F2 (&coef)[VPT][Row<T>::kP],
                                          F2 (&wb)[VPT][Row<T>::kP]) {
    constexpr int E = Row<T>::kE, P = Row<T>::kP;
    auto times = [](F2 (&c)[P], const float *w) {
#pragma unroll
        for (int k = 0; k < P; k += 2) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(w + 2 * k));
            c[k] = mul2(c[k], f2(v.x, v.y));
            c[k + 1] = mul2(c[k + 1], f2(v.z, v.w));
        }
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int k = 0; k < P; ++k) {
            coef[i][k] = both(n.bs);
            wb[i][k] = both(1.f);
        }
        if (j < n.nv) {
            if (a.w_after) times(coef[i], a.w_after + j * E);
            if (a.channel) times(coef[i], a.channel + j * E);
            if (a.w_before) times(wb[i], a.w_before + j * E);
        }
    }
}

template <typename T, int VPT, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_forward_kernel(BlockNormArgs a, NormShape n) {
    constexpr int E = Row<T>::kE, P = Row<T>::kP;
    extern __shared__ uint4 smem[];
    const int has_o = a.o != nullptr, has_z = a.z != nullptr, has_r = a.r != nullptr;
    const Ring<T, VPT> ring(smem, has_o + has_z + has_r, n.stages);
    Team tm;
    tm.warp_words = reinterpret_cast<float *>(smem + ring.words * n.stages);
    tm.vec_words = tm.warp_words + 4 * 32 * blockDim.y;
    tm.turn = 0;
    const int64_t step = (int64_t)gridDim.x * blockDim.y, first = (int64_t)blockIdx.x * blockDim.y;
    auto fetch = [&](int stage, int64_t row) {
        const bool live = row < a.T;
        if (has_o) ring.fetch(stage, 0, a.o, row * a.o_stride, n.nv, live);
        if (has_z) ring.fetch(stage, has_o, a.z, row * a.z_stride, n.nv, live);
        if (has_r) ring.fetch(stage, has_o + has_z, a.r, row * a.r_stride, n.nv, live);
        fetches_commit();
    };
    for (int k = 0; k < n.stages; ++k) fetch(k, first + k * step + threadIdx.y);
    F2 coef[VPT][P], wb[VPT][P];
    load_coef<T, VPT>(a, n, coef, wb);
    tm.clear();
    int stage = 0;
    for (int64_t base = first; base < a.T; base += step) {
        const int64_t row = base + threadIdx.y;
        const bool live = row < a.T;
        F2 u[VPT][P];
        uint4 uz[VPT], ur[VPT];
        fetches_wait(n.stages);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint4 none = make_uint4(0, 0, 0, 0);
            Row<T>::unpack(has_o ? ring.take(stage, 0, i) : none, u[i]);
            uz[i] = has_z ? ring.take(stage, has_o, i) : none;
            ur[i] = has_r ? ring.take(stage, has_o + has_z, i) : none;
        }
        fetch(stage, row + n.stages * step);
        stage = stage + 1 == n.stages ? 0 : stage + 1;
        if (n.mode != kGroupNone) {
            float ss[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                F2 t = both(0.f);
#pragma unroll
                for (int k = 0; k < P; ++k) t = fma2(u[i][k], u[i][k], t);
                ss[i] = fold(t);
            }
            group_sum<VPT>(tm, n.mode, n.gw, n.nv, ss);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const F2 rstd = both(rsqrtf(fmaf(ss[i], n.inv_group, n.eps)));
#pragma unroll
                for (int k = 0; k < P; ++k) u[i][k] = mul2(u[i][k], rstd);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
#pragma unroll
            for (int k = 0; k < P; ++k) u[i][k] = mul2(u[i][k], coef[i][k]);
            if (has_z) {
                F2 z[P], none[P];
                Row<T>::unpack(uz[i], z);
                act<false>(n.gate, z, none);
#pragma unroll
                for (int k = 0; k < P; ++k) u[i][k] = mul2(u[i][k], z[k]);
            }
            if (has_r) {
                F2 r[P];
                Row<T>::unpack(ur[i], r);
#pragma unroll
                for (int k = 0; k < P; ++k)
                    u[i][k] = has_o ? fma2(both(n.rs), r[k], u[i][k]) : mul2(both(n.rs), r[k]);
            }
            if (a.r_out && live && j < n.nv) Row<T>::store(a.r_out, row * n.width + j * E, u[i]);
        }
        if (a.next) {
            F2 t = both(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int k = 0; k < P; ++k) t = fma2(u[i][k], u[i][k], t);
            float sum[1] = {fold(t)};
            tm.row_sum<1>(sum);
            const F2 rstd = both(rsqrtf(fmaf(sum[0], n.inv_width, n.eps)));
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int j = threadIdx.x + i * blockDim.x;
#pragma unroll
                for (int k = 0; k < P; ++k) u[i][k] = mul2(mul2(u[i][k], rstd), wb[i][k]);
                if (live && j < n.nv) Row<T>::store(a.next, row * n.width + j * E, u[i]);
            }
        }
    }
}

template <typename T, int VPT, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_backward_kernel(BlockNormArgs a, NormShape n) {
    constexpr int E = Row<T>::kE, P = Row<T>::kP;
    extern __shared__ uint4 smem[];
    const int has_o = a.o != nullptr, has_z = a.z != nullptr, has_d = a.d_r_out != nullptr, has_n = a.d_next != nullptr;
    const int at_z = has_o, at_d = has_o + has_z, at_n = at_d + has_d;  // the tensors' places in a stage
    const Ring<T, VPT> ring(smem, at_n + 2 * has_n, n.stages);
    Team tm;
    tm.warp_words = reinterpret_cast<float *>(smem + ring.words * n.stages);
    tm.vec_words = tm.warp_words + 4 * 32 * blockDim.y;
    tm.turn = 0;
    const int64_t step = (int64_t)gridDim.x * blockDim.y, first = (int64_t)blockIdx.x * blockDim.y;
    auto fetch = [&](int stage, int64_t row) {
        const bool live = row < a.T;
        if (has_n) {
            ring.fetch(stage, at_n, a.r, row * a.r_stride, n.nv, live);
            ring.fetch(stage, at_n + 1, a.d_next, row * n.width, n.nv, live);
        }
        if (has_d) ring.fetch(stage, at_d, a.d_r_out, row * n.width, n.nv, live);
        if (has_o) ring.fetch(stage, 0, a.o, row * a.o_stride, n.nv, live);
        if (has_z) ring.fetch(stage, at_z, a.z, row * a.z_stride, n.nv, live);
        fetches_commit();
    };
    for (int k = 0; k < n.stages; ++k) fetch(k, first + k * step + threadIdx.y);
    F2 coef[VPT][P], wb[VPT][P];
    load_coef<T, VPT>(a, n, coef, wb);
    tm.clear();
    F2 sum_c[VPT][P], sum_b[VPT][P];  // C_j and dw_before of the thread's columns
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < P; ++k) sum_c[i][k] = sum_b[i][k] = both(0.f);
    int stage = 0;
    for (int64_t base = first; base < a.T; base += step) {
        const int64_t row = base + threadIdx.y;
        const bool live = row < a.T;
        F2 d[VPT][P];
        uint4 uo[VPT], uz[VPT], ur[VPT], un[VPT];
        fetches_wait(n.stages);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const uint4 none = make_uint4(0, 0, 0, 0);
            uo[i] = has_o ? ring.take(stage, 0, i) : none;
            uz[i] = has_z ? ring.take(stage, at_z, i) : none;
            Row<T>::unpack(has_d ? ring.take(stage, at_d, i) : none, d[i]);
            ur[i] = has_n ? ring.take(stage, at_n, i) : none;
            un[i] = has_n ? ring.take(stage, at_n + 1, i) : none;
        }
        fetch(stage, row + n.stages * step);
        stage = stage + 1 == n.stages ? 0 : stage + 1;
        if (has_n) {
            F2 ss = both(0.f), dot = both(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                F2 r[P], g[P];
                Row<T>::unpack(ur[i], r);
                Row<T>::unpack(un[i], g);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    ss = fma2(r[k], r[k], ss);
                    dot = fma2(mul2(g[k], wb[i][k]), r[k], dot);
                }
            }
            float sums[2] = {fold(ss), fold(dot)};
            tm.row_sum<2>(sums);
            const float rstd = rsqrtf(fmaf(sums[0], n.inv_width, n.eps));
            const F2 minus_mean = both(-(sums[1] * rstd * n.inv_width)), rr = both(rstd);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                F2 r[P], g[P];
                Row<T>::unpack(ur[i], r);
                Row<T>::unpack(un[i], g);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const F2 hat = mul2(r[k], rr);
                    sum_b[i][k] = fma2(g[k], hat, sum_b[i][k]);
                    d[i][k] = fma2(rr, fma2(hat, minus_mean, mul2(g[k], wb[i][k])), d[i][k]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (a.d_r && live && j < n.nv) {
                F2 v[P];
#pragma unroll
                for (int k = 0; k < P; ++k) v[k] = mul2(both(n.rs), d[i][k]);
                Row<T>::store(a.d_r, row * n.width + j * E, v);
            }
        }
        if (!has_o) continue;
        F2 o[VPT][P];
        float rstd[VPT], dot[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            Row<T>::unpack(uo[i], o[i]);
            rstd[i] = 1.f;
        }
        if (n.mode != kGroupNone) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                F2 t = both(0.f);
#pragma unroll
                for (int k = 0; k < P; ++k) t = fma2(o[i][k], o[i][k], t);
                rstd[i] = fold(t);
            }
            group_sum<VPT>(tm, n.mode, n.gw, n.nv, rstd);
#pragma unroll
            for (int i = 0; i < VPT; ++i) rstd[i] = rsqrtf(fmaf(rstd[i], n.inv_group, n.eps));
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            F2 av[P], da[P];
#pragma unroll
            for (int k = 0; k < P; ++k) o[i][k] = mul2(o[i][k], both(rstd[i]));
            if (has_z) {
                Row<T>::unpack(uz[i], av);
                act<true>(n.gate, av, da);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    da[k] = mul2(mul2(mul2(d[i][k], coef[i][k]), o[i][k]), da[k]);
                    d[i][k] = mul2(d[i][k], av[k]);
                }
                if (live && j < n.nv) Row<T>::store(a.d_z, row * n.width + j * E, da);
            }
            F2 t = both(0.f);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                sum_c[i][k] = fma2(d[i][k], o[i][k], sum_c[i][k]);
                d[i][k] = mul2(d[i][k], coef[i][k]);
                t = fma2(d[i][k], o[i][k], t);
            }
            dot[i] = fold(t);
        }
        if (n.mode != kGroupNone) {
            group_sum<VPT>(tm, n.mode, n.gw, n.nv, dot);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const F2 minus_mean = both(-dot[i] * n.inv_group), rr = both(rstd[i]);
#pragma unroll
                for (int k = 0; k < P; ++k) d[i][k] = mul2(rr, fma2(o[i][k], minus_mean, d[i][k]));
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (live && j < n.nv) Row<T>::store(a.d_o, row * n.width + j * E, d[i]);
        }
    }
    // column sums of this team: one partial row of each
    const int64_t rows = (int64_t)gridDim.x * blockDim.y;
    const int64_t mine = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < n.nv) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
                if (a.d_w_after || a.d_channel)
                    *reinterpret_cast<float2 *>(a.partials + mine * n.width + j * E + 2 * k) = f2_get(sum_c[i][k]);
                if (a.d_w_before)
                    *reinterpret_cast<float2 *>(a.partials + (rows + mine) * n.width + j * E + 2 * k) = f2_get(sum_b[i][k]);
            }
        }
    }
}

// The weights' gradients from the partial rows, in a fixed order: 32 columns
// per CTA, 32 interleaved runs of rows, then their sum.
__global__ void __launch_bounds__(1024) norm_weight_grads_kernel(BlockNormArgs a, NormShape n, int rows) {
    __shared__ float part[2][32][33];
    const int c = threadIdx.x, col = blockIdx.x * 32 + c;
    float s[2] = {0.f, 0.f};
    if (col < n.width) {
        for (int r = threadIdx.y; r < rows; r += 32) {
            if (a.d_w_after || a.d_channel) s[0] += a.partials[(int64_t)r * n.width + col];
            if (a.d_w_before) s[1] += a.partials[((int64_t)rows + r) * n.width + col];
        }
    }
    part[0][threadIdx.y][c] = s[0];
    part[1][threadIdx.y][c] = s[1];
    __syncthreads();
    if (threadIdx.y < 2) {
        // lane c of row y sums column c of array y
        float t = 0.f;
        for (int r = 0; r < 32; ++r) t += part[threadIdx.y][r][c];
        if (col < n.width) {
            if (threadIdx.y == 0) {
                const float w = a.w_after ? a.w_after[col] : 1.f, ch = a.channel ? a.channel[col] : 1.f;
                if (a.d_w_after) a.d_w_after[col] = n.bs * ch * t;
                if (a.d_channel) a.d_channel[col] = n.bs * w * t;
            } else if (a.d_w_before) {
                a.d_w_before[col] = t;
            }
        }
    }
}

struct NormPlan {
    NormShape n;
    int vpt, threads, rows;  // words per thread, threads of a row, rows per CTA
    int per_sm;              // CTAs on an SM
    size_t team_bytes;       // shared memory of the sums
};

NormPlan plan_norm(const sse_norm_config_t &c, bool after, bool backward) {
    NormPlan p{};
    const int E = c.dtype == SSE_BF16 ? 8 : 4;
    const int group = c.group ? c.group : c.width;
    p.n.width = c.width;
    p.n.nv = c.width / E;
    p.n.gw = group / E;
    const bool pow2 = (p.n.gw & (p.n.gw - 1)) == 0;
    p.n.mode = !after ? kGroupNone : group == c.width ? kGroupRow : pow2 && p.n.gw <= 32 ? kGroupShuffle : kGroupShared;
    p.n.gate = c.gate;
    p.n.eps = c.eps;
    p.n.rs = c.residual_scale;
    p.n.bs = c.branch_scale;
    p.n.inv_width = 1.f / c.width;
    p.n.inv_group = 1.f / group;
    p.vpt = p.n.nv > 1024 ? 2 : 1;
    p.threads = ((p.n.nv + p.vpt - 1) / p.vpt + 31) / 32 * 32;
    p.rows = p.threads >= 256 ? 1 : 256 / p.threads;
    // registers: 64 per thread forward, 80 backward (64 above 512 threads)
    const int most = backward ? 768 : 1024;
    p.per_sm = most / (p.threads * p.rows);
    if (p.per_sm < 1) p.per_sm = 1;
    p.team_bytes = sizeof(float) * (4 * 32 * p.rows + (p.n.mode == kGroupShared ? p.rows * p.n.nv : 0));
    return p;
}

int norm_grid(const NormPlan &p, int64_t T) {
    const int64_t need = (T + p.rows - 1) / p.rows, most = (int64_t)kSms * p.per_sm;
    return (int)(need < most ? need : most);
}

template <typename T, int VPT, int MAXT, int FWD, int BWD>
cudaError_t launch_t(NormPlan p, const BlockNormArgs &a, bool backward, int tensors, cudaStream_t stream) {
    // three rows ahead where the SM's shared memory holds them, else two or one
    const size_t row_bytes = (size_t)tensors * VPT * p.threads * p.rows * 16, room = size_t(220) * 1024 / p.per_sm;
    p.n.stages = 3;
    while (p.n.stages > 1 && p.n.stages * row_bytes + p.team_bytes > room) --p.n.stages;
    const size_t smem = p.n.stages * row_bytes + p.team_bytes;
    const auto kernel = backward ? norm_backward_kernel<T, VPT, MAXT, BWD> : norm_forward_kernel<T, VPT, MAXT, FWD>;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<norm_grid(p, a.T), dim3(p.threads, p.rows), smem, stream>>>(a, p.n);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rows(const NormPlan &p, const BlockNormArgs &a, bool backward, cudaStream_t stream) {
    const int tensors = (a.o != nullptr) + (a.z != nullptr) +
                        (backward ? (a.d_r_out != nullptr) + 2 * (a.d_next != nullptr) : (a.r != nullptr));
    if (p.vpt == 2) return launch_t<T, 2, 1024, 1, 1>(p, a, backward, tensors, stream);
    if (p.threads * p.rows <= 256) return launch_t<T, 1, 256, 4, 3>(p, a, backward, tensors, stream);
    if (p.threads <= 384) return launch_t<T, 1, 384, 2, 2>(p, a, backward, tensors, stream);
    if (p.threads <= 512) return launch_t<T, 1, 512, 2, 1>(p, a, backward, tensors, stream);
    return launch_t<T, 1, 1024, 1, 1>(p, a, backward, tensors, stream);
}

}  // namespace

int64_t block_norm_partial_rows(const sse_norm_config_t &cfg, int64_t T) {
    const NormPlan p = plan_norm(cfg, true, true);
    return (int64_t)norm_grid(p, T) * p.rows;
}

cudaError_t launch_block_norm(const sse_norm_config_t &cfg, const BlockNormArgs &a, cudaStream_t stream) {
    const NormPlan p = plan_norm(cfg, a.w_after != nullptr, false);
    return cfg.dtype == SSE_BF16 ? launch_rows<__nv_bfloat16>(p, a, false, stream)
                                 : launch_rows<float>(p, a, false, stream);
}

cudaError_t launch_block_norm_backward(const sse_norm_config_t &cfg, const BlockNormArgs &a, cudaStream_t stream) {
    const NormPlan p = plan_norm(cfg, a.w_after != nullptr, true);
    if (a.T > 0) {
        const cudaError_t e = cfg.dtype == SSE_BF16 ? launch_rows<__nv_bfloat16>(p, a, true, stream)
                                                    : launch_rows<float>(p, a, true, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.d_w_after || a.d_channel || a.d_w_before) {
        const int rows = norm_grid(p, a.T) * p.rows;
        norm_weight_grads_kernel<<<(cfg.width + 31) / 32, dim3(32, 32), 0, stream>>>(a, p.n, rows);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

}  // namespace sse
