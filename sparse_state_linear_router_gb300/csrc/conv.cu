// conv.cu -- the short causal convolution, one filter of K taps per channel:
//   u_t = bias + sum_j w[j] x_{t - (K - 1) + j},  out_t = act(u_t)
// with the rows before a sequence from its state.  Gradients, with g_t =
// d_out_t act'(u_t), zero outside the sequence:
//   dx_p = sum_j w[j] g_{p + K - 1 - j}  (+ d_final of the last K - 1 rows; rows p
//   before the sequence are the initial state's),  dw[j] = sum_t g_t x_{t-(K-1)+j},
//   db = sum_t g_t
//
// Bound by HBM: 2 K + 6 operations per element against 4 to 8 bytes (backward 6 K
// + 20 against 6 to 12).  A thread has four columns and a run of tokens, whose last
// K - 1 rows (and, in the backward, K - 1 gradients g) stay in registers, so a row
// is read once but for the K - 1 rows in front of a run (backward: and behind it).
// The packed token axis is one axis: runs are cut without regard to sequences, and
// a sequence's first row takes the state's rows into the window.  Rows inside a
// sequence come in batches of four by asynchronous copies, two or three batches
// ahead.
//
// Measured on a GB300, K = 4 with SiLU, 32768 x 2048 in bf16: forward 47 to 50 us (HBM
// floor at 6.77 TB/s: 40), backward 94 (59), of which the activation is 18.  One row
// after another took 290 us together, batches loaded to registers 52 and 116.
// float32, 16384 x 2048: 53 to 58 and 83 (40, 59); a fourth batch in the backward's ring
// leaves it two CTAs less on an SM, and 103 us.
#include "quad.cuh"

namespace sse {
namespace {

constexpr int kWarps = 4;  // runs of a CTA
constexpr int kBatch = 4;   // rows copied and summed at a time

// A thread's ring of rows in shared memory: its own quads of one tensor (four batches) or two (three).  The thread that
// copies a quad is the one that reads it, so there is no barrier.
template <typename T, int TENSORS> struct Ring {
    using Raw = typename Quad<T>::Raw;
    static constexpr int kGroups = TENSORS == 1 ? 4 : 3;
    static constexpr int kBytes = kGroups * kBatch * TENSORS * 32 * kWarps * (int)sizeof(Raw);
    static __device__ __forceinline__ char *slot(char *smem, int group, int row, int tensor) {
        return smem + (((group * kBatch + row) * TENSORS + tensor) * 32 * kWarps + threadIdx.x) * sizeof(Raw);
    }
    static __device__ __forceinline__ void copy(char *to, const T *from) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                     "n"(sizeof(Raw)) : "memory");
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // Until the oldest of kGroups batches is there.
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kGroups - 1) : "memory"); }
};

// What a thread has of the filter.
template <int K> struct Filter {
    F2 w[K][2], b[2];
    __device__ __forceinline__ Filter(const ConvArgs &a, int col) {
        float v[4 * K];
        const float4 *at = reinterpret_cast<const float4 *>(a.weight + (int64_t)col * K);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const float4 f = __ldg(at + i);
            v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
            w[j][0] = f2(v[j], v[K + j]);
            w[j][1] = f2(v[2 * K + j], v[3 * K + j]);
        }
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.bias) f = __ldg(reinterpret_cast<const float4 *>(a.bias + col));
        b[0] = f2(f.x, f.y);
        b[1] = f2(f.z, f.w);
    }
};

// The last K rows, the newest last, as they were stored.
template <typename T, int K> struct Window {
    using Raw = typename Quad<T>::Raw;
    Raw row[K];
    __device__ __forceinline__ void push(Raw u) {
#pragma unroll
        for (int i = 0; i + 1 < K; ++i) row[i] = row[i + 1];
        row[K - 1] = u;
    }
    static __device__ __forceinline__ Raw of(const ConvArgs &a, int t, int col) {
        return *reinterpret_cast<const Raw *>(static_cast<const T *>(a.x) + (int64_t)t * a.x_stride + col);
    }
    // State row i of sequence q.
    static __device__ __forceinline__ int64_t state_at(int q, int i, int width, int col) {
        return ((int64_t)q * (K - 1) + i) * width + col;
    }
    // The rows before token t of sequence q, which begins at `start`: rows 1 to K - 1.
    __device__ __forceinline__ void before(const ConvArgs &a, int t, int q, int start, int width, int col) {
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            const int r = t - (K - 1) + i;
            row[i + 1] = r >= start ? of(a, r, col)
                         : a.init   ? *reinterpret_cast<const Raw *>(static_cast<const T *>(a.init) +
                                                                   state_at(q, r - start + K - 1, width, col))
                                    : Quad<T>::zero();
        }
    }
    // u of the newest row.
    __device__ __forceinline__ void sum(const Filter<K> &f, F2 (&u)[2]) const {
        u[0] = f.b[0], u[1] = f.b[1];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            F2 x[2];
            Quad<T>::unpack(row[j], x);
            u[0] = fma2(f.w[j][0], x[0], u[0]);
            u[1] = fma2(f.w[j][1], x[1], u[1]);
        }
    }
};

// A sequence's state as it is; zeros where there is none.
template <typename T, int K>
__device__ __forceinline__ void copy_state(T *to, const T *from, int q, int width, int col) {
    using Raw = typename Quad<T>::Raw;
    Raw row[K - 1];
#pragma unroll
    for (int i = 0; i < K - 1; ++i)
        row[i] = from ? *reinterpret_cast<const Raw *>(from + Window<T, K>::state_at(q, i, width, col)) : Quad<T>::zero();
#pragma unroll
    for (int i = 0; i < K - 1; ++i) *reinterpret_cast<Raw *>(to + Window<T, K>::state_at(q, i, width, col)) = row[i];
}

// Runs: gridDim.y CTAs of kWarps warps, `run` tokens each.
template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(32 * kWarps, 6) conv_forward_kernel(ConvArgs a, int width, int run) {
    using Raw = typename Quad<T>::Raw;
    using Rows = Ring<T, 1>;
    const int lane = threadIdx.x & 31;
    const int col = (blockIdx.x * 32 + lane) * 4, lanes = min(32, (width - blockIdx.x * 128) / 4);  // of the warp, with columns
    if (col >= width) return;
    const int id = blockIdx.y * kWarps + (threadIdx.x >> 5), runs = gridDim.y * kWarps;
    const int end_of_all = clamp_token(__ldg(a.cu_seqlens + a.num_seqs), a.total_tokens);
    int t = id * run, t0 = t;
    const int t1 = min(t + run, end_of_all);
    extern __shared__ __align__(16) char smem[];
    const Filter<K> f(a, col);
    if (t < t1) {
        int q = sequence_of(a.cu_seqlens, a.num_seqs, t);
        int start = __ldg(a.cu_seqlens + q), end = __ldg(a.cu_seqlens + q + 1);
        Window<T, K> win;
        win.before(a, t, q, start, width, col);
        while (t < t1) {
            if (t == end) {  // the next sequence that has tokens
                for (bool next = true; end <= t && q + 1 < a.num_seqs; next = false) {
                    const int s = next ? 0 : sequence_of(a.cu_seqlens, a.num_seqs, t);  // past a row of empty ones
                    q = s > q ? s : q + 1;
                    start = __ldg(a.cu_seqlens + q);
                    end = __ldg(a.cu_seqlens + q + 1);
                }
                win.before(a, t, q, start, width, col);
            }
            // whole batches of one sequence
            const int batches = (min(t1, end) - t) / kBatch;
            auto copy = [&](int k) {
                if (k < batches)
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        Rows::copy(Rows::slot(smem, k % Rows::kGroups, i, 0),
                                         static_cast<const T *>(a.x) + (int64_t)(t0 + k * kBatch + i) * a.x_stride + col);
                Rows::commit();
            };
            if (batches > 0) {
                t0 = t;
                for (int k = 0; k + 1 < Rows::kGroups; ++k) copy(k);
            }
            for (int k = 0; k < batches; ++k) {
                copy(k + Rows::kGroups - 1);
                Rows::wait();
                F2 x[K - 1 + kBatch][2];
#pragma unroll
                for (int i = 0; i < K - 1; ++i) Quad<T>::unpack(win.row[i + 1], x[i]);
                Raw r[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    r[i] = *reinterpret_cast<const Raw *>(Rows::slot(smem, k % Rows::kGroups, i, 0));
                    Quad<T>::unpack(r[i], x[K - 1 + i]);
                    F2 u[2] = {f.b[0], f.b[1]};
#pragma unroll
                    for (int j = 0; j < K; ++j) {
                        u[0] = fma2(f.w[j][0], x[i + j][0], u[0]);
                        u[1] = fma2(f.w[j][1], x[i + j][1], u[1]);
                    }
                    if constexpr (SILU) {
                        u[0] = mul2(u[0], sigmoid2<T>(u[0]));
                        u[1] = mul2(u[1], sigmoid2<T>(u[1]));
                    }
                    *reinterpret_cast<Raw *>(static_cast<T *>(a.out) + (int64_t)(t + i) * width + col) = Quad<T>::pack(u);
                }
#pragma unroll
                for (int i = 1; i < K; ++i) win.row[i] = r[kBatch - K + i];
                t += kBatch;
            }
            for (const int stop = min(t1, min(end, t + kBatch)); t < stop; ++t) {
                win.push(Window<T, K>::of(a, t, col));
                F2 u[2];
                win.sum(f, u);
                if constexpr (SILU) {
                    u[0] = mul2(u[0], sigmoid2<T>(u[0]));
                    u[1] = mul2(u[1], sigmoid2<T>(u[1]));
                }
                *reinterpret_cast<Raw *>(static_cast<T *>(a.out) + (int64_t)t * width + col) = Quad<T>::pack(u);
            }
            if (t == end && a.final_state)
#pragma unroll
                for (int i = 0; i < K - 1; ++i)
                    *reinterpret_cast<Raw *>(static_cast<T *>(a.final_state) + Window<T, K>::state_at(q, i, width, col)) =
                        win.row[i + 1];
        }
    }
    if (a.final_state)  // empty sequences keep their state
        each_empty(a.cu_seqlens, a.num_seqs, id, runs, lane, lanes, [&](int q) {
            copy_state<T, K>(static_cast<T *>(a.final_state), static_cast<const T *>(a.init), q, width, col);
        });
}

template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(32 * kWarps, 4) conv_backward_kernel(ConvArgs a, int width, int run) {
    using Raw = typename Quad<T>::Raw;
    using Rows = Ring<T, 2>;
    __shared__ float4 part[kWarps][K + 1][32];
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (blockIdx.x * 32 + lane) * 4;
    const bool live = col < width;
    const int id = blockIdx.y * kWarps + warp, runs = gridDim.y * kWarps;
    const int end_of_all = clamp_token(__ldg(a.cu_seqlens + a.num_seqs), a.total_tokens);
    const int t0 = id * run, t1 = min(t0 + run, end_of_all);
    F2 dw[K][2], db[2];
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][0] = dw[j][1] = both(0.f);
    db[0] = db[1] = both(0.f);
    if (live && t0 < t1) {
        const Filter<K> f(a, col);
        int q = sequence_of(a.cu_seqlens, a.num_seqs, t0);
        // The run's part of one sequence after the other: rows [s0, s1) of the gradient, and the rows of the initial
        // state where the sequence begins in the run.  Row p is complete with g_{p + K - 1}.
        for (int s0 = t0; s0 < t1 && q < a.num_seqs; ++q) {
            const int start = __ldg(a.cu_seqlens + q), end = __ldg(a.cu_seqlens + q + 1);
            if (end <= s0) {  // past a row of empty ones
                q = max(q, sequence_of(a.cu_seqlens, a.num_seqs, s0) - 1);
                continue;
            }
            const int s1 = min(end, t1);
            Window<T, K> win;
            win.before(a, s0, q, start, width, col);
            F2 g[K][2];
#pragma unroll
            for (int j = 0; j < K; ++j) g[j][0] = g[j][1] = both(0.f);
            for (int t = s0; t < s1 + K - 1;) {
                // Whole batches whose gradients need nothing but rows of this run and sequence.  Behind each: K - 1 rows of the
                // window and of g.
                const int batches = t == s0 + K - 1 ? (s1 - t) / kBatch : 0, from = t;
                auto copy = [&](int k) {
                    if (k < batches)
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            const int64_t row = from + k * kBatch + i;
                            Rows::copy(Rows::slot(smem, k % Rows::kGroups, i, 0), static_cast<const T *>(a.x) + row * a.x_stride + col);
                            Rows::copy(Rows::slot(smem, k % Rows::kGroups, i, 1), static_cast<const T *>(a.d_out) + row * width + col);
                        }
                    Rows::commit();
                };
                if (batches > 0)
                    for (int k = 0; k + 1 < Rows::kGroups; ++k) copy(k);
                for (int k = 0; k < batches; ++k) {
                    copy(k + Rows::kGroups - 1);
                    Rows::wait();
                    F2 x[K - 1 + kBatch][2], gs[K - 1 + kBatch][2];
#pragma unroll
                    for (int i = 0; i < K - 1; ++i) {
                        Quad<T>::unpack(win.row[i + 1], x[i]);
                        gs[i][0] = g[i + 1][0], gs[i][1] = g[i + 1][1];
                    }
                    Raw rx[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        rx[i] = *reinterpret_cast<const Raw *>(Rows::slot(smem, k % Rows::kGroups, i, 0));
                        Quad<T>::unpack(rx[i], x[K - 1 + i]);
                        Quad<T>::unpack(*reinterpret_cast<const Raw *>(Rows::slot(smem, k % Rows::kGroups, i, 1)), gs[K - 1 + i]);
                        F2 dx[2] = {both(0.f), both(0.f)};
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            if constexpr (SILU) {  // silu' = s (1 + u (1 - s))
                                F2 u = f.b[c];
#pragma unroll
                                for (int j = 0; j < K; ++j) u = fma2(f.w[j][c], x[i + j][c], u);
                                const F2 s = sigmoid2<T>(u);
                                gs[K - 1 + i][c] = mul2(gs[K - 1 + i][c], mul2(s, fma2(u, fma2(s, both(-1.f), both(1.f)), both(1.f))));
                            }
                            const F2 gr = gs[K - 1 + i][c];
#pragma unroll
                            for (int j = 0; j < K; ++j) {
                                dw[j][c] = fma2(gr, x[i + j][c], dw[j][c]);
                                dx[c] = fma2(f.w[j][c], gs[K - 1 + i - j][c], dx[c]);
                            }
                            db[c] = add2(db[c], gr);
                        }
                        *reinterpret_cast<Raw *>(static_cast<T *>(a.dx) + (int64_t)(t + i - (K - 1)) * width + col) = Quad<T>::pack(dx);
                    }
#pragma unroll
                    for (int i = 1; i < K; ++i) {
                        win.row[i] = rx[kBatch - K + i];
                        g[i][0] = gs[kBatch - 1 + i][0], g[i][1] = gs[kBatch - 1 + i][1];
                    }
                    t += kBatch;
                }
#pragma unroll
                for (int j = 0; j + 1 < K; ++j) g[j][0] = g[j + 1][0], g[j][1] = g[j + 1][1];
                g[K - 1][0] = g[K - 1][1] = both(0.f);
                if (t < end) {
                    win.push(Window<T, K>::of(a, t, col));
                    Quad<T>::unpack(*reinterpret_cast<const Raw *>(static_cast<const T *>(a.d_out) + (int64_t)t * width + col),
                                    g[K - 1]);
                    if constexpr (SILU) {
                        F2 u[2];
                        win.sum(f, u);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {  // silu' = s (1 + u (1 - s))
                            const F2 s = sigmoid2<T>(u[i]);
                            g[K - 1][i] = mul2(g[K - 1][i], mul2(s, fma2(u[i], fma2(s, both(-1.f), both(1.f)), both(1.f))));
                        }
                    }
                    if (t < s1) {
#pragma unroll
                        for (int j = 0; j < K; ++j) {
                            F2 x[2];
                            Quad<T>::unpack(win.row[j], x);
                            dw[j][0] = fma2(g[K - 1][0], x[0], dw[j][0]);
                            dw[j][1] = fma2(g[K - 1][1], x[1], dw[j][1]);
                        }
                        db[0] = add2(db[0], g[K - 1][0]);
                        db[1] = add2(db[1], g[K - 1][1]);
                    }
                }
                const int p = t++ - (K - 1);
                if (p < s0 && (s0 != start || !a.d_init)) continue;  // another run's row, or nobody's
                F2 d[2] = {both(0.f), both(0.f)};
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    d[0] = fma2(f.w[j][0], g[K - 1 - j][0], d[0]);
                    d[1] = fma2(f.w[j][1], g[K - 1 - j][1], d[1]);
                }
                if (a.d_final && p >= end - (K - 1)) {
                    F2 e[2];
                    Quad<T>::unpack(*reinterpret_cast<const Raw *>(static_cast<const T *>(a.d_final) +
                                                                 Window<T, K>::state_at(q, p - end + K - 1, width, col)),
                                    e);
                    d[0] = add2(d[0], e[0]);
                    d[1] = add2(d[1], e[1]);
                }
                T *to = p >= start ? static_cast<T *>(a.dx) + (int64_t)p * width + col
                                   : static_cast<T *>(a.d_init) + Window<T, K>::state_at(q, p - start + K - 1, width, col);
                *reinterpret_cast<Raw *>(to) = Quad<T>::pack(d);
            }
            s0 = s1;
        }
    }
    if (live && a.d_init)  // empty sequences hand the final state's gradient through
        each_empty(a.cu_seqlens, a.num_seqs, id, runs, lane, min(32, (width - blockIdx.x * 128) / 4), [&](int q) {
            copy_state<T, K>(static_cast<T *>(a.d_init), static_cast<const T *>(a.d_final), q, width, col);
        });
    griddep_launch_dependents();
#pragma unroll
    for (int j = 0; j <= K; ++j) {
        const float2 lo = f2_get(j < K ? dw[j < K ? j : 0][0] : db[0]), hi = f2_get(j < K ? dw[j < K ? j : 0][1] : db[1]);
        part[warp][j][lane] = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
    __syncthreads();
    if (!live) return;
    for (int j = warp; j <= K; j += kWarps) {
        float4 s = part[0][j][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 v = part[w][j][lane];
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        *reinterpret_cast<float4 *>(a.partials + ((int64_t)blockIdx.y * (K + 1) + j) * width + col) = s;
    }
}

// The weights' gradients from the CTAs' partial rows, in a fixed order: 32 columns of one tap (blockIdx.y; the bias
// last) per CTA, 32 interleaved runs of rows, then their sum.  Launched as a dependent of the gradient kernel.
__global__ void __launch_bounds__(1024) conv_weights_kernel(ConvArgs a, int width, int taps, int rows) {
    __shared__ float sums[32][33];
    const int c = threadIdx.x, col = blockIdx.x * 32 + c, j = blockIdx.y;
    griddep_wait();
    if (j == taps && !a.d_bias) return;
    const float *from = a.partials + (int64_t)j * width + col;
    float s = 0.f;
    if (col < width) {
#pragma unroll 8
        for (int r = threadIdx.y; r < rows; r += 32) s += from[(int64_t)r * (taps + 1) * width];
    }
    sums[threadIdx.y][c] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < width) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += sums[r][c];
        if (j == taps)
            a.d_bias[col] = t;
        else
            a.d_weight[(int64_t)col * taps + j] = t;
    }
}

// One token of each sequence.
template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs a, int width) {
    using Raw = typename Quad<T>::Raw;
    const int quads = width / 4;
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    const int64_t b = i / quads;
    if (b >= a.num_seqs) return;
    const int col = (int)(i - b * quads) * 4;
    const Filter<K> f(a, col);
    Window<T, K> win;
    T *state = static_cast<T *>(a.final_state);
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
        win.row[k] = *reinterpret_cast<const Raw *>(state + Window<T, K>::state_at((int)b, k, width, col));
    win.row[K - 1] = Window<T, K>::of(a, (int)b, col);
    F2 u[2];
    win.sum(f, u);
    if constexpr (SILU) {
        u[0] = mul2(u[0], sigmoid2<T>(u[0]));
        u[1] = mul2(u[1], sigmoid2<T>(u[1]));
    }
    *reinterpret_cast<Raw *>(static_cast<T *>(a.out) + b * width + col) = Quad<T>::pack(u);
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
        *reinterpret_cast<Raw *>(state + Window<T, K>::state_at((int)b, k, width, col)) = win.row[k + 1];
}

enum What { kForward, kBackward, kStep };

constexpr int kSms = 152;

// Tokens of a warp's run, and CTAs along the tokens.
void cut(int width, int64_t T, bool backward, int &run, int &ctas) {
    const int64_t columns = (width + 127) / 128, warps = (int64_t)kSms * 16;
    int64_t r = (T * columns + warps - 1) / warps;
    const int least = 8, most = backward ? 128 : 64;
    run = (int)(r < least ? least : r > most ? most : r);
    const int64_t n = (T + (int64_t)run * kWarps - 1) / ((int64_t)run * kWarps);
    ctas = n < 1 ? 1 : (int)n;
    while (ctas > 65535) {  // the grid's limit
        run *= 2;
        ctas = (int)((T + (int64_t)run * kWarps - 1) / ((int64_t)run * kWarps));
    }
}

template <typename T, int K, bool SILU>
cudaError_t launch_t(What what, const sse_conv_config_t &c, const ConvArgs &a, cudaStream_t s) {
    if (what == kStep) {
        const int64_t blocks = ((int64_t)a.num_seqs * (c.width / 4) + 127) / 128;
        if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
        conv_step_kernel<T, K, SILU><<<(unsigned)blocks, 128, 0, s>>>(a, c.width);
        return cudaGetLastError();
    }
    int run, ctas;
    cut(c.width, a.total_tokens, what == kBackward, run, ctas);
    const dim3 grid((c.width + 127) / 128, ctas);
    if (what == kForward) {
        conv_forward_kernel<T, K, SILU><<<grid, 32 * kWarps, Ring<T, 1>::kBytes, s>>>(a, c.width, run);
        return cudaGetLastError();
    }
    constexpr int kRing = Ring<T, 2>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(conv_backward_kernel<T, K, SILU>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing);
    if (e != cudaSuccess) return e;
    conv_backward_kernel<T, K, SILU><<<grid, 32 * kWarps, kRing, s>>>(a, c.width, run);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_dependent(conv_weights_kernel, dim3((c.width + 31) / 32, K + 1), dim3(32, 32), 0, s, a, c.width, K, ctas);
}

template <typename T> cudaError_t launch_taps(What what, const sse_conv_config_t &c, const ConvArgs &a, cudaStream_t s) {
    const bool silu = c.act == SSE_GATE_SILU;
    switch (c.taps) {
    case 2: return silu ? launch_t<T, 2, true>(what, c, a, s) : launch_t<T, 2, false>(what, c, a, s);
    case 3: return silu ? launch_t<T, 3, true>(what, c, a, s) : launch_t<T, 3, false>(what, c, a, s);
    default: return silu ? launch_t<T, 4, true>(what, c, a, s) : launch_t<T, 4, false>(what, c, a, s);
    }
}

cudaError_t launch(What what, const sse_conv_config_t &c, const ConvArgs &a, cudaStream_t s) {
    return c.dtype == SSE_BF16 ? launch_taps<__nv_bfloat16>(what, c, a, s) : launch_taps<float>(what, c, a, s);
}

}  // namespace

int64_t conv_partial_rows(const sse_conv_config_t &cfg, int64_t T) {
    int run, ctas;
    cut(cfg.width, T, true, run, ctas);
    return ctas;
}
cudaError_t launch_conv_forward(const sse_conv_config_t &cfg, const ConvArgs &a, cudaStream_t stream) {
    return launch(kForward, cfg, a, stream);
}
cudaError_t launch_conv_backward(const sse_conv_config_t &cfg, const ConvArgs &a, cudaStream_t stream) {
    return launch(kBackward, cfg, a, stream);
}
cudaError_t launch_conv_step(const sse_conv_config_t &cfg, const ConvArgs &a, cudaStream_t stream) {
    return launch(kStep, cfg, a, stream);
}

}  // namespace sse
