// scan.cu -- the gated linear recurrence: forward, backward and one step.
#include "sse_internal.cuh"

namespace sse {
namespace {

constexpr int kThreads = 128;

// a = exp(la), s(a) and ds/dla of the input scale MODE (sse_input_scale_t).
template <int MODE>
__device__ __forceinline__ void decay(float la, float &a, float &s, float &ds) {
    a = expf(la);
    s = 1.f;
    ds = 0.f;
    if (MODE == SSE_INPUT_COMPLEMENT) {
        s = -expm1f(la);
        ds = -a;
    } else if (MODE == SSE_INPUT_UNIT) {
        s = sqrtf(-expm1f(2.f * la));
        ds = s > 0.f ? -a * a / s : 0.f;
    }
}

// One thread per (sequence, channel), token after token.
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) scan_forward_kernel(ScanArgs p, int width) {
    const int col = blockIdx.x * kThreads + threadIdx.x;
    if (col >= width) return;
    const T *x = static_cast<const T *>(p.x), *g = static_cast<const T *>(p.log_gate);
    for (int s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        const int t0 = p.cu_seqlens[s], t1 = p.cu_seqlens[s + 1];
        float h = p.init ? p.init[(int64_t)s * width + col] : 0.f;
        for (int64_t t = t0; t < t1; ++t) {
            if (p.checkpoints && t % kScanCheckpoint == 0)
                p.checkpoints[t / kScanCheckpoint * width + col] = h;
            float a, sc, ds;
            decay<MODE>(Elem<T>::load(g + t * p.gate_stride + col), a, sc, ds);
            h = fmaf(a, h, sc * Elem<T>::load(x + t * p.x_stride + col));
            Elem<T>::store(static_cast<T *>(p.out) + t * width + col, h);
        }
        if (p.final_state) p.final_state[(int64_t)s * width + col] = h;
    }
}

// The same, backwards; each block of kScanCheckpoint tokens recomputes its states from its checkpoint.
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) scan_backward_kernel(ScanArgs p, int width) {
    const int col = blockIdx.x * kThreads + threadIdx.x;
    if (col >= width) return;
    const T *x = static_cast<const T *>(p.x), *g = static_cast<const T *>(p.log_gate);
    const T *dy = static_cast<const T *>(p.d_out);
    float before[kScanCheckpoint];
    for (int s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        const int t0 = p.cu_seqlens[s], t1 = p.cu_seqlens[s + 1];
        float e = p.d_final ? p.d_final[(int64_t)s * width + col] : 0.f;
        for (int64_t hi = t1; hi > t0;) {
            const int64_t blk = (hi - 1) / kScanCheckpoint * kScanCheckpoint;
            const int64_t lo = blk > t0 ? blk : t0;
            float h = blk > t0 ? p.checkpoints[blk / kScanCheckpoint * width + col]
                               : (p.init ? p.init[(int64_t)s * width + col] : 0.f);
            float a, sc, ds;
            for (int64_t t = lo; t < hi; ++t) {
                before[t - lo] = h;
                decay<MODE>(Elem<T>::load(g + t * p.gate_stride + col), a, sc, ds);
                h = fmaf(a, h, sc * Elem<T>::load(x + t * p.x_stride + col));
            }
            for (int64_t t = hi - 1; t >= lo; --t) {
                decay<MODE>(Elem<T>::load(g + t * p.gate_stride + col), a, sc, ds);
                const float dh = Elem<T>::load(dy + t * width + col) + e;
                const float xv = Elem<T>::load(x + t * p.x_stride + col);
                Elem<T>::store(static_cast<T *>(p.dx) + t * width + col, sc * dh);
                Elem<T>::store(static_cast<T *>(p.d_log_gate) + t * width + col,
                               dh * (MODE == SSE_INPUT_PLAIN ? a * before[t - lo] : fmaf(ds, xv, a * before[t - lo])));
                e = a * dh;
            }
            hi = lo;
        }
        if (p.d_init) p.d_init[(int64_t)s * width + col] = e;
    }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanArgs p, int width) {
    const int col = blockIdx.x * kThreads + threadIdx.x;
    if (col >= width) return;
    for (int64_t s = blockIdx.y; s < p.num_seqs; s += gridDim.y) {
        float a, sc, ds;
        decay<MODE>(Elem<T>::load(static_cast<const T *>(p.log_gate) + s * p.gate_stride + col), a, sc, ds);
        float *st = p.final_state + s * width + col;
        const float h = fmaf(a, *st, sc * Elem<T>::load(static_cast<const T *>(p.x) + s * p.x_stride + col));
        *st = h;
        Elem<T>::store(static_cast<T *>(p.out) + s * width + col, h);
    }
}

enum { kForward, kBackward, kStep };

template <typename T, int MODE>
cudaError_t launch_t(int what, const ScanArgs &a, int width, cudaStream_t stream) {
    const dim3 grid((width + kThreads - 1) / kThreads, a.num_seqs < 65535 ? a.num_seqs : 65535);
    if (what == kForward)
        scan_forward_kernel<T, MODE><<<grid, kThreads, 0, stream>>>(a, width);
    else if (what == kBackward)
        scan_backward_kernel<T, MODE><<<grid, kThreads, 0, stream>>>(a, width);
    else
        scan_step_kernel<T, MODE><<<grid, kThreads, 0, stream>>>(a, width);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_mode(int what, const sse_scan_config_t &cfg, const ScanArgs &a, cudaStream_t stream) {
    switch (cfg.input_scale) {
    case SSE_INPUT_PLAIN: return launch_t<T, SSE_INPUT_PLAIN>(what, a, cfg.width, stream);
    case SSE_INPUT_COMPLEMENT: return launch_t<T, SSE_INPUT_COMPLEMENT>(what, a, cfg.width, stream);
    default: return launch_t<T, SSE_INPUT_UNIT>(what, a, cfg.width, stream);
    }
}

cudaError_t launch(int what, const sse_scan_config_t &cfg, const ScanArgs &a, cudaStream_t stream) {
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
