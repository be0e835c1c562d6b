// selective.cu -- the selective state space scan: per channel c and state n, with
// D_t = softplus(delta_t + delta_bias) and a_t[n] = exp(D_t A[n]),
//   h_t[n] = a_t[n] h_{t-1}[n] + D_t B_t[n] x_t
//   y_t = sum_n C_t[n] h_t[n] + skip x_t,   out_t = y_t silu(gate_t)
// Gradients, with dy = d_out silu(gate) and g_t[n] = C_t[n] dy_t + a_{t+1}[n] g_{t+1}[n]:
//   d_gate = d_out y silu'(gate),  dx = skip dy + D sum_n B g
//   dD = x sum_n B g + sum_n A g a h_{t-1},  d_delta = dD softplus'
//   dB[n] = sum_c g D x,  dC[n] = sum_c dy h  (over the channels of the group)
//   dA = sum_t D g a h_{t-1},  d_skip = sum_t dy x,  d_delta_bias = sum_t d_delta
#include "sse_internal.cuh"

namespace sse {
namespace {

template <typename T> __device__ __forceinline__ float load(const void *p, int64_t i) {
    if constexpr (sizeof(T) == 2)
        return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    else
        return static_cast<const float *>(p)[i];
}
template <typename T> __device__ __forceinline__ void store(void *p, int64_t i, float v) {
    if constexpr (sizeof(T) == 2)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(p)[i] = v;
}

__device__ __forceinline__ float sigmoid(float u) { return 1.f / (1.f + expf(-u)); }
__device__ __forceinline__ float softplus(float u) { return fmaxf(u, 0.f) + log1pf(expf(-fabsf(u))); }

__device__ __forceinline__ int clamp_token(int t, int T) { return t < 0 ? 0 : t > T ? T : t; }

template <int L> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int L> __device__ __forceinline__ float channels_sum(float v) {  // over the channels of a warp
#pragma unroll
    for (int o = 16; o >= L; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// L lanes of a channel, four states each.  A warp has 32 / L channels of one group (`per` channels a group, `warps`
// warps a group), the lanes behind a group's end nothing.
struct Place {
    int c, g;  // channel and group
    bool live;
};
template <int L> __device__ __forceinline__ Place place(int width, int groups, int lane) {
    const int per = width / groups, warps = (per + 32 / L - 1) / (32 / L);
    const int w = blockIdx.x;
    Place p;
    p.g = w / warps;
    const int i = (w - p.g * warps) * (32 / L) + lane / L;
    p.live = i < per;
    p.c = p.g * per + (p.live ? i : per - 1);
    return p;
}

struct Token {  // of a channel
    float x, d, raw, B[4], C[4];
};
template <typename T>
__device__ __forceinline__ Token token(const SelectiveArgs &a, int64_t t, int c, int at, float bias) {
    Token k;
    k.x = load<T>(a.x, t * a.x_stride + c);
    k.raw = load<T>(a.delta, t * a.delta_stride + c) + bias;
    k.d = softplus(k.raw);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        k.B[n] = load<T>(a.B, t * a.b_stride + at + n);
        k.C[n] = load<T>(a.C, t * a.c_stride + at + n);
    }
    return k;
}

template <typename T, int L>
__global__ void __launch_bounds__(32) selective_forward_kernel(SelectiveArgs a, sse_selective_config_t cfg) {
    const int lane = threadIdx.x, N = 4 * L;
    const Place p = place<L>(cfg.width, cfg.groups, lane);
    const int n0 = lane % L * 4, at = p.g * N + n0;
    const float bias = a.delta_bias ? a.delta_bias[p.c] : 0.f, skip = a.skip ? a.skip[p.c] : 0.f;
    float A[4], h[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) A[n] = a.A[(int64_t)p.c * N + n0 + n];
    for (int q = blockIdx.y; q < a.num_seqs; q += gridDim.y) {
        const int t0 = clamp_token(a.cu_seqlens[q], a.total_tokens), t1 = clamp_token(a.cu_seqlens[q + 1], a.total_tokens);
        const int64_t state = ((int64_t)q * cfg.width + p.c) * N + n0;
#pragma unroll
        for (int n = 0; n < 4; ++n) h[n] = a.init ? a.init[state + n] : 0.f;
        for (int t = t0; t < t1; ++t) {
            if (a.checkpoints && t % kSelectiveCheckpoint == 0 && p.live)
                for (int n = 0; n < 4; ++n)
                    a.checkpoints[((int64_t)(t / kSelectiveCheckpoint) * cfg.width + p.c) * N + n0 + n] = h[n];
            const Token k = token<T>(a, t, p.c, at, bias);
            float y = 0.f;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                h[n] = fmaf(expf(k.d * A[n]), h[n], k.d * k.x * k.B[n]);
                y = fmaf(k.C[n], h[n], y);
            }
            y = fmaf(skip, k.x, lanes_sum<L>(y));
            if (a.gate) {
                const float z = load<T>(a.gate, (int64_t)t * a.gate_stride + p.c);
                y *= z * sigmoid(z);
            }
            if (p.live && n0 == 0) store<T>(a.out, (int64_t)t * cfg.width + p.c, y);
        }
        if (a.final_state && p.live)
#pragma unroll
            for (int n = 0; n < 4; ++n) a.final_state[state + n] = h[n];
    }
}

// Partial sums: of B's and C's gradients [warps of a group][T][groups][2][N], of A's and the two vectors' [S][width][N + 2].
template <typename T, int L>
__global__ void __launch_bounds__(32) selective_backward_kernel(SelectiveArgs a, sse_selective_config_t cfg, float *token_sums,
                                                                float *weight_sums) {
    constexpr int kRows = kSelectiveCheckpoint;
    const int lane = threadIdx.x, N = 4 * L;
    const Place p = place<L>(cfg.width, cfg.groups, lane);
    const int n0 = lane % L * 4, at = p.g * N + n0;
    const int part = blockIdx.x % (gridDim.x / cfg.groups);
    const float bias = a.delta_bias ? a.delta_bias[p.c] : 0.f, skip = a.skip ? a.skip[p.c] : 0.f;
    float A[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) A[n] = a.A[(int64_t)p.c * N + n0 + n];
    for (int q = blockIdx.y; q < a.num_seqs; q += gridDim.y) {
        const int t0 = clamp_token(a.cu_seqlens[q], a.total_tokens), t1 = clamp_token(a.cu_seqlens[q + 1], a.total_tokens);
        const int64_t state = ((int64_t)q * cfg.width + p.c) * N + n0;
        float e[4], dA[4] = {0.f, 0.f, 0.f, 0.f}, d_skip = 0.f, d_bias = 0.f;  // e = a_{t+1} g_{t+1}
#pragma unroll
        for (int n = 0; n < 4; ++n) e[n] = a.d_final ? a.d_final[state + n] : 0.f;
        for (int lo = t1 > t0 ? (t1 - 1) / kRows * kRows : t0 - 1; lo + kRows > t0 && t1 > t0; lo -= kRows) {
            const int s0 = max(lo, t0), s1 = min(lo + kRows, t1);
            float before[kRows][4], h[4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
                h[n] = s0 > t0 ? a.checkpoints[((int64_t)(s0 / kRows) * cfg.width + p.c) * N + n0 + n]
                       : a.init ? a.init[state + n] : 0.f;
            for (int t = s0; t < s1; ++t) {
                const Token k = token<T>(a, t, p.c, at, bias);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    before[t - s0][n] = h[n];
                    h[n] = fmaf(expf(k.d * A[n]), h[n], k.d * k.x * k.B[n]);
                }
            }
            for (int t = s1 - 1; t >= s0; --t) {
                const Token k = token<T>(a, t, p.c, at, bias);
                const float d_out = load<T>(a.d_out, (int64_t)t * cfg.width + p.c);
                float dy = d_out, z = 0.f, s = 0.f;
                if (a.gate) {
                    z = load<T>(a.gate, (int64_t)t * a.gate_stride + p.c);
                    s = sigmoid(z);
                    dy *= z * s;
                }
                float y = 0.f, Bg = 0.f, Aw = 0.f;
                float *sums = token_sums + (((int64_t)part * a.total_tokens + t) * cfg.groups + p.g) * 2 * N + n0;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float dec = expf(k.d * A[n]), u = dec * before[t - s0][n], b = k.d * k.x;
                    const float now = fmaf(b, k.B[n], u);
                    y = fmaf(k.C[n], now, y);
                    const float g = fmaf(k.C[n], dy, e[n]);
                    e[n] = dec * g;
                    const float w = g * u;
                    Bg = fmaf(k.B[n], g, Bg);
                    Aw = fmaf(A[n], w, Aw);
                    dA[n] = fmaf(k.d, w, dA[n]);
                    const float dB = channels_sum<L>(p.live ? g * b : 0.f), dC = channels_sum<L>(p.live ? dy * now : 0.f);
                    if (lane < L) {
                        sums[n] = dB;
                        sums[N + n] = dC;
                    }
                }
                y = fmaf(skip, k.x, lanes_sum<L>(y));
                Bg = lanes_sum<L>(Bg);
                Aw = lanes_sum<L>(Aw);
                const float dd = fmaf(k.x, Bg, Aw) * sigmoid(k.raw);
                d_skip = fmaf(dy, k.x, d_skip);
                d_bias += dd;
                if (p.live && n0 == 0) {
                    const int64_t i = (int64_t)t * cfg.width + p.c;
                    store<T>(a.dx, i, fmaf(skip, dy, k.d * Bg));
                    store<T>(a.d_delta, i, dd);
                    if (a.gate) store<T>(a.d_gate, i, d_out * y * s * (1.f + z * (1.f - s)));
                }
            }
        }
        if (p.live) {
            float *w = weight_sums + ((int64_t)q * cfg.width + p.c) * (N + 2);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (a.d_init) a.d_init[state + n] = e[n];
                w[n0 + n] = dA[n];
            }
            if (n0 == 0) {
                w[N] = d_skip;
                w[N + 1] = d_bias;
            }
        }
    }
}

template <typename T>
__global__ void selective_tokens_kernel(SelectiveArgs a, sse_selective_config_t cfg, const float *sums, int parts) {
    const int64_t row = (int64_t)cfg.groups * cfg.state, i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, t = i / row;
    if (t >= clamp_token(a.cu_seqlens[a.num_seqs], a.total_tokens)) return;
    const int g = (int)(i - t * row) / cfg.state, n = (int)(i % cfg.state);
    float dB = 0.f, dC = 0.f;
    for (int p = 0; p < parts; ++p) {
        const float *s = sums + (((int64_t)p * a.total_tokens + t) * cfg.groups + g) * 2 * cfg.state + n;
        dB += s[0];
        dC += s[cfg.state];
    }
    store<T>(a.d_B, i, dB);
    store<T>(a.d_C, i, dC);
}

__global__ void selective_weights_kernel(SelectiveArgs a, sse_selective_config_t cfg, const float *sums) {
    const int N = cfg.state, i = blockIdx.x * blockDim.x + threadIdx.x, c = i / (N + 2), n = i % (N + 2);
    if (c >= cfg.width) return;
    float s = 0.f;
    for (int q = 0; q < a.num_seqs; ++q) s += sums[(int64_t)q * cfg.width * (N + 2) + i];
    if (n < N)
        a.d_A[(int64_t)c * N + n] = s;
    else if (n == N && a.d_skip)
        a.d_skip[c] = s;
    else if (n == N + 1 && a.d_delta_bias)
        a.d_delta_bias[c] = s;
}

template <typename T, int L>
__global__ void __launch_bounds__(256) selective_step_kernel(SelectiveArgs a, sse_selective_config_t cfg) {
    constexpr int N = 4 * L;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, channel = i / L;
    const int64_t b = channel / cfg.width;
    const bool live = b < a.num_seqs;
    if (!__any_sync(0xffffffffu, live)) return;
    const int64_t t = live ? b : a.num_seqs - 1;
    const int c = live ? (int)(channel - b * cfg.width) : cfg.width - 1, n0 = (int)(i % L) * 4;
    const int g = c / (cfg.width / cfg.groups);
    const Token k = token<T>(a, t, c, g * N + n0, a.delta_bias ? a.delta_bias[c] : 0.f);
    float *state = a.final_state + (t * cfg.width + c) * N + n0;
    float4 h = *reinterpret_cast<const float4 *>(state);
    const float4 A = *reinterpret_cast<const float4 *>(a.A + (int64_t)c * N + n0);
    const float u = k.d * k.x;
    h.x = fmaf(expf(k.d * A.x), h.x, u * k.B[0]);
    h.y = fmaf(expf(k.d * A.y), h.y, u * k.B[1]);
    h.z = fmaf(expf(k.d * A.z), h.z, u * k.B[2]);
    h.w = fmaf(expf(k.d * A.w), h.w, u * k.B[3]);
    float y = lanes_sum<L>(fmaf(k.C[0], h.x, fmaf(k.C[1], h.y, fmaf(k.C[2], h.z, k.C[3] * h.w))));
    if (!live) return;
    *reinterpret_cast<float4 *>(state) = h;
    if (n0) return;
    if (a.skip) y = fmaf(a.skip[c], k.x, y);
    if (a.gate) {
        const float z = load<T>(a.gate, t * a.gate_stride + c);
        y *= z * sigmoid(z);
    }
    store<T>(a.out, t * cfg.width + c, y);
}

int warps_of_group(const sse_selective_config_t &c) {
    const int per = c.width / c.groups, channels = 128 / c.state;
    return (per + channels - 1) / channels;
}

enum What { kForward, kBackward, kStep };

template <typename T, int L>
cudaError_t launch_t(What what, const sse_selective_config_t &c, const SelectiveArgs &a, cudaStream_t s) {
    if (what == kStep) {
        const int64_t blocks = ((int64_t)a.num_seqs * c.width * L + 255) / 256;
        if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
        selective_step_kernel<T, L><<<(unsigned)blocks, 256, 0, s>>>(a, c);
        return cudaGetLastError();
    }
    const int warps = warps_of_group(c);
    const dim3 grid(warps * c.groups, a.num_seqs < 1 ? 1 : a.num_seqs < 65535 ? a.num_seqs : 65535);
    if (what == kForward) {
        selective_forward_kernel<T, L><<<grid, 32, 0, s>>>(a, c);
        return cudaGetLastError();
    }
    float *token_sums = reinterpret_cast<float *>(a.workspace);
    float *weight_sums = token_sums + (int64_t)warps * a.total_tokens * c.groups * 2 * c.state;
    if (a.num_seqs > 0) selective_backward_kernel<T, L><<<grid, 32, 0, s>>>(a, c, token_sums, weight_sums);
    const int64_t n = (int64_t)a.total_tokens * c.groups * c.state;
    if (n > 0) selective_tokens_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, c, token_sums, warps);
    selective_weights_kernel<<<(c.width * (c.state + 2) + 255) / 256, 256, 0, s>>>(a, c, weight_sums);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_state(What what, const sse_selective_config_t &c, const SelectiveArgs &a, cudaStream_t s) {
    switch (c.state) {
    case 8: return launch_t<T, 2>(what, c, a, s);
    case 16: return launch_t<T, 4>(what, c, a, s);
    case 32: return launch_t<T, 8>(what, c, a, s);
    default: return launch_t<T, 16>(what, c, a, s);
    }
}

cudaError_t launch(What what, const sse_selective_config_t &c, const SelectiveArgs &a, cudaStream_t s) {
    return c.dtype == SSE_BF16 ? launch_state<__nv_bfloat16>(what, c, a, s) : launch_state<float>(what, c, a, s);
}

}  // namespace

size_t selective_forward_workspace(const sse_selective_config_t &, int64_t, int32_t) { return 0; }
size_t selective_backward_workspace(const sse_selective_config_t &c, int64_t T, int32_t S) {
    return sizeof(float) * ((size_t)warps_of_group(c) * T * c.groups * 2 * c.state + (size_t)S * c.width * (c.state + 2));
}
cudaError_t launch_selective_forward(const sse_selective_config_t &cfg, const SelectiveArgs &a, cudaStream_t stream) {
    return launch(kForward, cfg, a, stream);
}
cudaError_t launch_selective_backward(const sse_selective_config_t &cfg, const SelectiveArgs &a, cudaStream_t stream) {
    return launch(kBackward, cfg, a, stream);
}
cudaError_t launch_selective_step(const sse_selective_config_t &cfg, const SelectiveArgs &a, cudaStream_t stream) {
    return launch(kStep, cfg, a, stream);
}

}  // namespace sse
