// layer_norm.cu -- the layer norm with the residual stream in front of it:
//   r' = x + residual,  d = r' - mean r',  rstd = rsqrt(mean d^2 + eps)
//   out = d rstd w + b
// Gradients, with x_hat = d rstd and p = dy w:
//   dx = rstd (p - mean p - x_hat mean(p x_hat)) + d_r',  dw = sum dy x_hat,  db = sum dy
//
// Bound by HBM (about 10 to 20 operations per element against 4 to 16 bytes).  A
// team of warps covers a row, up to four 16-byte words per thread (two in the
// backward) that stay in registers, so every tensor is read once.  A warp forms
// its own mean m and the squares about it by shuffles; the warps' moments are
// joined as moments are, mean = sum n m / W and M2 = sum M2 + n (m - mean)^2, so a
// row takes one barrier and no sum of squares about a distant zero.  The
// backward's sums p and p (x - m) go with them: sum p (x - mean) is the sum of
// [p (x - m)] + (m - mean) [p] over the warps.  Rows of one warp take no barrier.
#include "f32x2.cuh"
#include "sse_internal.cuh"

namespace sse {
namespace {

constexpr int kSms = 152;

template <typename T> struct Word {
    static constexpr int kE = 16 / sizeof(T), kP = kE / 2;  // elements, pairs
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
    static __device__ __forceinline__ uint4 pack(const F2 (&f)[kP]) {
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
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ F2 both(float x) { return f2(x, x); }
__device__ __forceinline__ float fold(F2 v) {
    const float2 f = f2_get(v);
    return f.x + f.y;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// At most 2^-22.9 off, once per row.
__device__ __forceinline__ float rsqrt_ftz(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct LnShape {
    int width, nv;  // columns and 16-byte words of a row
    int warps;      // of a row's team
    float eps, inv_width;
};

// Elements of a row that warp w of a team has (its words are w * 32 * VPT and on).
__device__ __forceinline__ int warp_elements(const LnShape &n, int w, int vpt, int e) {
    const int left = n.nv - w * 32 * vpt;
    return (left < 32 * vpt ? left : 32 * vpt) * e;
}

// Joins the warps' words {mean, M2, sum p, sum p (x - mean)} of a row; all threads of the team call it.  `turn` alternates
// between the rows, so that one barrier a row is enough.
template <int N>
__device__ __forceinline__ void join(const LnShape &n, float4 &v, int vpt, int e, int warp, int lane, int turn, float4 *words) {
    if (n.warps == 1) return;
    if (lane == 0) words[turn * 32 + warp] = v;
    __syncthreads();
    float mean = 0.f;
    for (int w = 0; w < n.warps; ++w) mean = fmaf((float)warp_elements(n, w, vpt, e), words[turn * 32 + w].x, mean);
    mean *= n.inv_width;
    float4 t = make_float4(mean, 0.f, 0.f, 0.f);
    for (int w = 0; w < n.warps; ++w) {
        const float4 u = words[turn * 32 + w];
        const float d = u.x - mean;
        t.y += fmaf((float)warp_elements(n, w, vpt, e) * d, d, u.y);
        if constexpr (N == 4) {
            t.z += u.z;
            t.w += fmaf(d, u.z, u.w);
        }
    }
    v = t;
}

// Words of a row: warp w, word i, lane l has word (w * VPT + i) * 32 + l.
template <typename T, int VPT>
__global__ void __launch_bounds__(VPT == 4 ? 512 : 256) layer_norm_kernel(LayerNormArgs a, LnShape n) {
    constexpr int E = Word<T>::kE, P = Word<T>::kP;
    __shared__ float4 words[64];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int warp = n.warps == 1 ? 0 : wid;
    const int64_t rows_on = n.warps == 1 ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const int64_t first = n.warps == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + wid : blockIdx.x;
    const float mine = (float)warp_elements(n, warp, VPT, E), inv_mine = 1.f / mine;
    int turn = 0;
    for (int64_t row = first; row < a.T; row += rows_on) {
        F2 v[VPT][P];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = (warp * VPT + i) * 32 + lane;
            uint4 u = make_uint4(0, 0, 0, 0), s = u;
            if (j < n.nv) {
                u = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.x_stride + j * E);
                if (a.r) s = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.r) + row * a.r_stride + j * E);
            }
            Word<T>::unpack(u, v[i]);
            if (a.r) {
                F2 w[P];
                Word<T>::unpack(s, w);
#pragma unroll
                for (int k = 0; k < P; ++k) v[i][k] = add2(v[i][k], w[k]);
            }
        }
        F2 t = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int k = 0; k < P; ++k) t = add2(t, v[i][k]);
        float4 m = make_float4(warp_sum(fold(t)) * inv_mine, 0.f, 0.f, 0.f);
        t = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if ((warp * VPT + i) * 32 + lane < n.nv)
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const F2 d = add2(v[i][k], both(-m.x));
                    t = fma2(d, d, t);
                }
        m.y = warp_sum(fold(t));
        join<2>(n, m, VPT, E, warp, lane, turn, words);
        turn ^= 1;
        const float rstd = rsqrt_ftz(fmaf(m.y, n.inv_width, n.eps));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = (warp * VPT + i) * 32 + lane;
            if (j >= n.nv) continue;
            const int64_t at = row * n.width + j * E;
            if (a.r_out) *reinterpret_cast<uint4 *>(static_cast<T *>(a.r_out) + at) = Word<T>::pack(v[i]);
            F2 y[P];
#pragma unroll
            for (int k = 0; k < P; ++k) {
                y[k] = mul2(add2(v[i][k], both(-m.x)), both(rstd));
                float2 b = make_float2(0.f, 0.f);
                if (a.bias) b = __ldg(reinterpret_cast<const float2 *>(a.bias + j * E + 2 * k));
                if (a.weight) {
                    const float2 w = __ldg(reinterpret_cast<const float2 *>(a.weight + j * E + 2 * k));
                    y[k] = fma2(y[k], f2(w.x, w.y), f2(b.x, b.y));
                } else {
                    y[k] = add2(y[k], f2(b.x, b.y));
                }
            }
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + at) = Word<T>::pack(y);
        }
    }
}

template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) layer_norm_backward_kernel(LayerNormArgs a, LnShape n) {
    constexpr int E = Word<T>::kE, P = Word<T>::kP;
    __shared__ float4 words[64];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int warp = n.warps == 1 ? 0 : wid;
    const int64_t rows_on = n.warps == 1 ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const int64_t first = n.warps == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + wid : blockIdx.x;
    const float inv_mine = 1.f / (float)warp_elements(n, warp, VPT, E);
    F2 sum_w[VPT][P], sum_b[VPT][P];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < P; ++k) sum_w[i][k] = sum_b[i][k] = both(0.f);
    int turn = 0;
    for (int64_t row = first; row < a.T; row += rows_on) {
        F2 v[VPT][P], d[VPT][P];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = (warp * VPT + i) * 32 + lane;
            uint4 u = make_uint4(0, 0, 0, 0), s = u;
            if (j < n.nv) {
                u = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.x_stride + j * E);
                s = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.d_out) + row * n.width + j * E);
            }
            Word<T>::unpack(u, v[i]);
            Word<T>::unpack(s, d[i]);
        }
        F2 t = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int k = 0; k < P; ++k) t = add2(t, v[i][k]);
        float4 m;
        m.x = warp_sum(fold(t)) * inv_mine;
        F2 sq = both(0.f), sp = both(0.f), sx = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = (warp * VPT + i) * 32 + lane;
            if (j >= n.nv) continue;
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const F2 c = add2(v[i][k], both(-m.x));
                F2 p = d[i][k];
                if (a.weight) {
                    const float2 w = __ldg(reinterpret_cast<const float2 *>(a.weight + j * E + 2 * k));
                    p = mul2(p, f2(w.x, w.y));
                }
                sq = fma2(c, c, sq);
                sp = add2(sp, p);
                sx = fma2(p, c, sx);
            }
        }
        m.y = warp_sum(fold(sq));
        m.z = warp_sum(fold(sp));
        m.w = warp_sum(fold(sx));
        join<4>(n, m, VPT, E, warp, lane, turn, words);
        turn ^= 1;
        const float rstd = rsqrt_ftz(fmaf(m.y, n.inv_width, n.eps));
        const float mean_p = m.z * n.inv_width, slope = m.w * n.inv_width * rstd * rstd;  // mean(p x_hat) rstd
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = (warp * VPT + i) * 32 + lane;
            if (j >= n.nv) continue;
            const int64_t at = row * n.width + j * E;
            F2 e[P];
            if (a.d_r_out)
                Word<T>::unpack(*reinterpret_cast<const uint4 *>(static_cast<const T *>(a.d_r_out) + at), e);
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const F2 c = add2(v[i][k], both(-m.x));
                sum_w[i][k] = fma2(d[i][k], mul2(c, both(rstd)), sum_w[i][k]);
                sum_b[i][k] = add2(sum_b[i][k], d[i][k]);
                F2 p = d[i][k];
                if (a.weight) {
                    const float2 w = __ldg(reinterpret_cast<const float2 *>(a.weight + j * E + 2 * k));
                    p = mul2(p, f2(w.x, w.y));
                }
                p = mul2(fma2(c, both(-slope), add2(p, both(-mean_p))), both(rstd));
                e[k] = a.d_r_out ? add2(p, e[k]) : p;
            }
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.dx) + at) = Word<T>::pack(e);
        }
    }
    griddep_launch_dependents();
    // this team's column sums: one partial row of each
    if (first < rows_on)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = (warp * VPT + i) * 32 + lane;
            if (j >= n.nv) continue;
#pragma unroll
            for (int k = 0; k < P; ++k) {
                if (a.d_weight)
                    *reinterpret_cast<float2 *>(a.partials + first * n.width + j * E + 2 * k) = f2_get(sum_w[i][k]);
                if (a.d_bias)
                    *reinterpret_cast<float2 *>(a.partials + (rows_on + first) * n.width + j * E + 2 * k) = f2_get(sum_b[i][k]);
            }
        }
}

// The weights' gradients from the partial rows, in a fixed order: 32 columns of
// one array (blockIdx.y: dw, db) per CTA, 32 interleaved runs of rows, then their
// sum.  Launched as a dependent of the gradient kernel.
__global__ void __launch_bounds__(1024) layer_norm_weights_kernel(LayerNormArgs a, int width, int rows) {
    __shared__ float part[32][33];
    const int c = threadIdx.x, col = blockIdx.x * 32 + c;
    float *to = blockIdx.y ? a.d_bias : a.d_weight;
    griddep_wait();
    if (!to) return;
    const float *from = a.partials + (blockIdx.y ? (int64_t)rows * width : 0) + col;
    float s = 0.f;
    if (col < width) {
#pragma unroll 8
        for (int r = threadIdx.y; r < rows; r += 32) s += from[(int64_t)r * width];
    }
    part[threadIdx.y][c] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < width) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += part[r][c];
        to[col] = t;
    }
}

struct LnPlan {
    LnShape n;
    int vpt, threads, teams;  // words per thread, threads of a CTA, rows that a CTA has at a time
    int grid;
};

// Up to `most` words per thread.  Rows of one warp share a CTA of four.
LnPlan plan(const sse_layer_norm_config_t &c, int64_t T, bool backward) {
    LnPlan p{};
    const int most = backward ? 2 : 4;
    p.n.width = c.width;
    p.n.nv = c.width / (c.dtype == SSE_BF16 ? 8 : 4);
    p.n.eps = c.eps;
    p.n.inv_width = 1.f / c.width;
    p.n.warps = (p.n.nv + 32 * most - 1) / (32 * most);
    p.vpt = (p.n.nv + 32 * p.n.warps - 1) / (32 * p.n.warps);
    p.n.warps = (p.n.nv + 32 * p.vpt - 1) / (32 * p.vpt);
    p.teams = p.n.warps == 1 ? 4 : 1;
    p.threads = 32 * p.n.warps * p.teams;
    // as many as an SM holds: 64 registers a thread forward, 128 backward (64 where a row has more than 512 threads)
    int per_sm = (backward ? p.threads > 512 ? 1024 : 512 : 1024) / p.threads;
    if (per_sm < 1) per_sm = 1;
    const int64_t need = (T + p.teams - 1) / p.teams, hold = (int64_t)kSms * per_sm;
    p.grid = (int)(need < hold ? need : hold);
    return p;
}

template <typename T> cudaError_t launch_forward(const LnPlan &p, const LayerNormArgs &a, cudaStream_t s) {
    switch (p.vpt) {
    case 1: layer_norm_kernel<T, 1><<<p.grid, p.threads, 0, s>>>(a, p.n); break;
    case 2: layer_norm_kernel<T, 2><<<p.grid, p.threads, 0, s>>>(a, p.n); break;
    case 3: layer_norm_kernel<T, 3><<<p.grid, p.threads, 0, s>>>(a, p.n); break;
    default: layer_norm_kernel<T, 4><<<p.grid, p.threads, 0, s>>>(a, p.n);
    }
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_backward(const LnPlan &p, const LayerNormArgs &a, cudaStream_t s) {
    if (p.vpt == 1)
        layer_norm_backward_kernel<T, 1, 512><<<p.grid, p.threads, 0, s>>>(a, p.n);
    else if (p.threads <= 512)
        layer_norm_backward_kernel<T, 2, 512><<<p.grid, p.threads, 0, s>>>(a, p.n);
    else
        layer_norm_backward_kernel<T, 2, 1024><<<p.grid, p.threads, 0, s>>>(a, p.n);
    return cudaGetLastError();
}

}  // namespace

int64_t layer_norm_partial_rows(const sse_layer_norm_config_t &cfg, int64_t T) {
    const LnPlan p = plan(cfg, T, true);
    return (int64_t)p.grid * p.teams;
}

cudaError_t launch_layer_norm(const sse_layer_norm_config_t &cfg, const LayerNormArgs &a, cudaStream_t stream) {
    const LnPlan p = plan(cfg, a.T, false);
    return cfg.dtype == SSE_BF16 ? launch_forward<__nv_bfloat16>(p, a, stream) : launch_forward<float>(p, a, stream);
}

cudaError_t launch_layer_norm_backward(const sse_layer_norm_config_t &cfg, const LayerNormArgs &a, cudaStream_t stream) {
    const LnPlan p = plan(cfg, a.T, true);
    if (a.T > 0) {
        const cudaError_t e = cfg.dtype == SSE_BF16 ? launch_backward<__nv_bfloat16>(p, a, stream)
                                                    : launch_backward<float>(p, a, stream);
        if (e != cudaSuccess) return e;
    }
    if (!a.d_weight && !a.d_bias) return cudaSuccess;
    return launch_dependent(layer_norm_weights_kernel, dim3((cfg.width + 31) / 32, 2), dim3(32, 32), 0, stream, a, cfg.width,
                            p.grid * p.teams);
}

}  // namespace sse
