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
// Each row is read once into registers, 16 bytes per thread and tensor, by a
// team of threads that covers it; sums over the row or a group of it go
// through shuffles and one word per warp of shared memory.
#include "sse_internal.cuh"

namespace sse {
namespace {

constexpr int kSms = 152;

// How the sum of squares of the norm after the block is shared.
enum { kGroupNone, kGroupRow, kGroupShuffle, kGroupShared };

template <typename T> struct Row {
    static constexpr int kE = 16 / sizeof(T);  // elements of one 16-byte word
    static __device__ __forceinline__ uint4 load(const void *base, int64_t i) {
        return *reinterpret_cast<const uint4 *>(static_cast<const T *>(base) + i);
    }
    static __device__ __forceinline__ void unpack(uint4 u, float *f) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            if (sizeof(T) == 2)
                f[i] = __uint_as_float(i & 1 ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
            else
                f[i] = __uint_as_float(w[i]);
        }
    }
    static __device__ __forceinline__ void store(void *base, int64_t i, const float *f) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (sizeof(T) == 2) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
                w[k] = *reinterpret_cast<const uint32_t *>(&b);
            } else {
                w[k] = __float_as_uint(f[k]);
            }
        }
        *reinterpret_cast<uint4 *>(static_cast<T *>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// act(z); with GRAD also its derivative.
template <bool GRAD> __device__ __forceinline__ float act(int gate, float z, float &d) {
    if (gate == SSE_GATE_LINEAR) {
        if (GRAD) d = 1.f;
        return z;
    }
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    if (gate == SSE_GATE_SIGMOID) {
        if (GRAD) d = s * (1.f - s);
        return s;
    }
    if (GRAD) d = s * fmaf(z, 1.f - s, 1.f);
    return z * s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The team of one row: blockDim.x threads (whole warps), blockDim.y rows per
// CTA.  Every thread of the CTA makes the same calls (they synchronize).
struct Team {
    float *warp_words;  // [2][rows][32]: this row's words, two buffers in turn
    float *vec_words;   // [rows][words of a row]: kGroupShared only
    int turn;
    // Sum of one value per thread over the team.
    __device__ __forceinline__ float row_sum(float v) {
        v = warp_sum(v);
        const int warps = blockDim.x >> 5;
        if (warps == 1) return v;
        float *w = warp_words + (turn * blockDim.y + threadIdx.y) * 32;
        turn ^= 1;
        if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = v;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        return warp_sum(lane < warps ? w[lane] : 0.f);
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
        s = tm.row_sum(s);
#pragma unroll
        for (int i = 0; i < VPT; ++i) v[i] = s;
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
    int gate;
    float eps, rs, bs;
    float inv_width, inv_group;
};

// coef = branch_scale c w_after of the thread's columns
template <typename T, int VPT>
__device__ __forceinline__ void load_coef(const BlockNormArgs &a, const NormShape &n, float (&coef)[VPT][Row<T>::kE],
                                          float (&wb)[VPT][Row<T>::kE]) {
    constexpr int E = Row<T>::kE;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            coef[i][e] = n.bs;
            wb[i][e] = 0.f;
        }
        if (j < n.nv) {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                if (a.w_after) {
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(a.w_after + j * E + e));
                    coef[i][e] *= w.x; coef[i][e + 1] *= w.y; coef[i][e + 2] *= w.z; coef[i][e + 3] *= w.w;
                }
                if (a.channel) {
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(a.channel + j * E + e));
                    coef[i][e] *= w.x; coef[i][e + 1] *= w.y; coef[i][e + 2] *= w.z; coef[i][e + 3] *= w.w;
                }
                if (a.w_before) {
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(a.w_before + j * E + e));
                    wb[i][e] = w.x; wb[i][e + 1] = w.y; wb[i][e + 2] = w.z; wb[i][e + 3] = w.w;
                }
            }
        }
    }
}

template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_forward_kernel(BlockNormArgs a, NormShape n) {
    constexpr int E = Row<T>::kE;
    extern __shared__ float smem[];
    Team tm{smem, smem + 2 * blockDim.y * 32, 0};
    float coef[VPT][E], wb[VPT][E];
    load_coef<T, VPT>(a, n, coef, wb);
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < a.T; base += step) {
        const int64_t row = base + threadIdx.y;
        const bool live = row < a.T;
        float u[VPT][E], z[VPT][E], r[VPT][E];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            uint4 uo = make_uint4(0, 0, 0, 0), uz = uo, ur = uo;
            if (live && j < n.nv) {
                if (a.o) uo = Row<T>::load(a.o, row * a.o_stride + j * E);
                if (a.z) uz = Row<T>::load(a.z, row * a.z_stride + j * E);
                if (a.r) ur = Row<T>::load(a.r, row * a.r_stride + j * E);
            }
            Row<T>::unpack(uo, u[i]);
            Row<T>::unpack(uz, z[i]);
            Row<T>::unpack(ur, r[i]);
        }
        if (n.mode != kGroupNone) {
            float ss[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                ss[i] = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) ss[i] = fmaf(u[i][e], u[i][e], ss[i]);
            }
            group_sum<VPT>(tm, n.mode, n.gw, n.nv, ss);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const float rstd = rsqrtf(fmaf(ss[i], n.inv_group, n.eps));
#pragma unroll
                for (int e = 0; e < E; ++e) u[i][e] *= rstd;
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float d, v = coef[i][e] * u[i][e];
                if (n.gate != SSE_GATE_NONE) v *= act<false>(n.gate, z[i][e], d);
                u[i][e] = a.r ? (a.o ? fmaf(n.rs, r[i][e], v) : n.rs * r[i][e]) : v;
            }
            if (a.r_out && live && j < n.nv) Row<T>::store(a.r_out, row * n.width + j * E, u[i]);
        }
        if (a.next) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) ss = fmaf(u[i][e], u[i][e], ss);
            const float rstd = rsqrtf(fmaf(tm.row_sum(ss), n.inv_width, n.eps));
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int j = threadIdx.x + i * blockDim.x;
#pragma unroll
                for (int e = 0; e < E; ++e) u[i][e] *= rstd * wb[i][e];
                if (live && j < n.nv) Row<T>::store(a.next, row * n.width + j * E, u[i]);
            }
        }
    }
}

template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_backward_kernel(BlockNormArgs a, NormShape n) {
    constexpr int E = Row<T>::kE;
    extern __shared__ float smem[];
    Team tm{smem, smem + 2 * blockDim.y * 32, 0};
    float coef[VPT][E], wb[VPT][E];
    load_coef<T, VPT>(a, n, coef, wb);
    float sum_c[VPT][E], sum_b[VPT][E];  // C_j and dw_before of the thread's columns
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) sum_c[i][e] = sum_b[i][e] = 0.f;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    for (int64_t base = (int64_t)blockIdx.x * blockDim.y; base < a.T; base += step) {
        const int64_t row = base + threadIdx.y;
        const bool live = row < a.T;
        float d[VPT][E], o[VPT][E], z[VPT][E];
        uint4 ur[VPT], un[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            uint4 uo = make_uint4(0, 0, 0, 0), uz = uo, ud = uo;
            ur[i] = un[i] = uo;
            if (live && j < n.nv) {
                if (a.o) uo = Row<T>::load(a.o, row * a.o_stride + j * E);
                if (a.z) uz = Row<T>::load(a.z, row * a.z_stride + j * E);
                if (a.d_r_out) ud = Row<T>::load(a.d_r_out, row * n.width + j * E);
                if (a.d_next) {
                    ur[i] = Row<T>::load(a.r, row * a.r_stride + j * E);
                    un[i] = Row<T>::load(a.d_next, row * n.width + j * E);
                }
            }
            Row<T>::unpack(uo, o[i]);
            Row<T>::unpack(uz, z[i]);
            Row<T>::unpack(ud, d[i]);
        }
        if (a.d_next) {
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float r[E], g[E];
                Row<T>::unpack(ur[i], r);
                Row<T>::unpack(un[i], g);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    ss = fmaf(r[e], r[e], ss);
                    dot = fmaf(g[e] * wb[i][e], r[e], dot);
                }
            }
            const float rstd = rsqrtf(fmaf(tm.row_sum(ss), n.inv_width, n.eps));
            const float mean = tm.row_sum(dot) * rstd * n.inv_width;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float r[E], g[E];
                Row<T>::unpack(ur[i], r);
                Row<T>::unpack(un[i], g);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float hat = r[e] * rstd;
                    sum_b[i][e] = fmaf(g[e], hat, sum_b[i][e]);
                    d[i][e] = fmaf(rstd, fmaf(g[e], wb[i][e], -hat * mean), d[i][e]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (a.d_r && live && j < n.nv) {
                float v[E];
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = n.rs * d[i][e];
                Row<T>::store(a.d_r, row * n.width + j * E, v);
            }
        }
        if (!a.o) continue;
        float rstd[VPT], dot[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) rstd[i] = 1.f;
        if (n.mode != kGroupNone) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                rstd[i] = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) rstd[i] = fmaf(o[i][e], o[i][e], rstd[i]);
            }
            group_sum<VPT>(tm, n.mode, n.gw, n.nv, rstd);
#pragma unroll
            for (int i = 0; i < VPT; ++i) rstd[i] = rsqrtf(fmaf(rstd[i], n.inv_group, n.eps));
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            float dz[E];
            dot[i] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float da = 0.f, av = 1.f;
                o[i][e] *= rstd[i];
                if (n.gate != SSE_GATE_NONE) av = act<true>(n.gate, z[i][e], da);
                const float p = d[i][e] * coef[i][e];
                sum_c[i][e] = fmaf(d[i][e] * av, o[i][e], sum_c[i][e]);
                dz[e] = p * o[i][e] * da;
                d[i][e] = p * av;
                dot[i] = fmaf(d[i][e], o[i][e], dot[i]);
            }
            if (a.d_z && live && j < n.nv) Row<T>::store(a.d_z, row * n.width + j * E, dz);
        }
        if (n.mode != kGroupNone) {
            group_sum<VPT>(tm, n.mode, n.gw, n.nv, dot);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    d[i][e] = rstd[i] * fmaf(-o[i][e], dot[i] * n.inv_group, d[i][e]);
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
            for (int e = 0; e < E; e += 4) {
                if (a.d_w_after || a.d_channel)
                    *reinterpret_cast<float4 *>(a.partials + mine * n.width + j * E + e) =
                        make_float4(sum_c[i][e], sum_c[i][e + 1], sum_c[i][e + 2], sum_c[i][e + 3]);
                if (a.d_w_before)
                    *reinterpret_cast<float4 *>(a.partials + (rows + mine) * n.width + j * E + e) =
                        make_float4(sum_b[i][e], sum_b[i][e + 1], sum_b[i][e + 2], sum_b[i][e + 3]);
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
    size_t smem;
};

NormPlan plan_norm(const sse_norm_config_t &c, bool after) {
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
    p.smem = sizeof(float) * (2 * 32 * p.rows + (p.n.mode == kGroupShared ? p.rows * p.n.nv : 0));
    return p;
}

int norm_grid(const NormPlan &p, int64_t T) {
    const int64_t need = (T + p.rows - 1) / p.rows;
    const int64_t most = (int64_t)kSms * (p.threads * p.rows <= 256 ? 4 : p.threads <= 512 ? 2 : 1);
    return (int)(need < most ? need : most);
}

template <typename T, int VPT, int MAXT>
cudaError_t launch_t(const NormPlan &p, const BlockNormArgs &a, bool backward, cudaStream_t stream) {
    const dim3 block(p.threads, p.rows);
    const int grid = norm_grid(p, a.T);
    if (backward)
        norm_backward_kernel<T, VPT, MAXT><<<grid, block, p.smem, stream>>>(a, p.n);
    else
        norm_forward_kernel<T, VPT, MAXT><<<grid, block, p.smem, stream>>>(a, p.n);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rows(const NormPlan &p, const BlockNormArgs &a, bool backward, cudaStream_t stream) {
    if (p.vpt == 2) return launch_t<T, 2, 1024>(p, a, backward, stream);
    if (p.threads * p.rows <= 256) return launch_t<T, 1, 256>(p, a, backward, stream);
    if (p.threads <= 512) return launch_t<T, 1, 512>(p, a, backward, stream);
    return launch_t<T, 1, 1024>(p, a, backward, stream);
}

}  // namespace

int64_t block_norm_partial_rows(const sse_norm_config_t &cfg, int64_t T) {
    const NormPlan p = plan_norm(cfg, true);
    return (int64_t)norm_grid(p, T) * p.rows;
}

cudaError_t launch_block_norm(const sse_norm_config_t &cfg, const BlockNormArgs &a, cudaStream_t stream) {
    const NormPlan p = plan_norm(cfg, a.w_after != nullptr);
    return cfg.dtype == SSE_BF16 ? launch_rows<__nv_bfloat16>(p, a, false, stream)
                                 : launch_rows<float>(p, a, false, stream);
}

cudaError_t launch_block_norm_backward(const sse_norm_config_t &cfg, const BlockNormArgs &a, cudaStream_t stream) {
    const NormPlan p = plan_norm(cfg, a.w_after != nullptr);
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
