// selective.cu -- the selective state space scan: per channel c and state n, with
// D_t = softplus(delta_t + delta_bias) and a_t[n] = exp(D_t A[n]),
//   h_t[n] = a_t[n] h_{t-1}[n] + D_t B_t[n] x_t
//   y_t = sum_n C_t[n] h_t[n] + skip x_t,   out_t = y_t silu(gate_t)
// Gradients, with dy = d_out silu(gate) and g_t[n] = C_t[n] dy_t + a_{t+1}[n] g_{t+1}[n]:
//   d_gate = d_out y silu'(gate),  dx = skip dy + D sum_n B g
//   dD = x sum_n B g + sum_n A g a h_{t-1},  d_delta = dD softplus'
//   dB[n] = sum_c g D x,  dC[n] = sum_c dy h  (over the channels of the group)
//   dA = sum_t D g a h_{t-1},  d_skip = sum_t dy x,  d_delta_bias = sum_t d_delta
#include "selective.cuh"

namespace sse {
namespace {

// Lanes of a pair of channels, and at most so many states each.
constexpr int kL = 4, kNT = 4;


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

template <int L> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
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

// ---------------------------------------------------------------------------
// Forward.  A warp is a CTA; it has 16 channels of a group and one range of
// tokens, which it goes through in tiles of 16.  L = 4 lanes share a pair of
// channels, NT states each (lane = j * 8 + pair); SL slices of 4 NT states.
// Per tile:
//   1. steps D and D x, B and C in float32 to shared memory (16 bytes per pair
//      of channels: D0, D1, D x0, D x1), lanes over (token, four channels);
//   2. token by token, h = 2^(D A log2 e) h + (D x) B and this thread's part of
//      sum C h, its states in registers;
//   3. the parts' sum, skip and gate, lanes over (token, four channels) again.
// FULL: the whole forward.  Otherwise only what a later range starts from: the
// state at the range's end from nothing (or from the sequence that begins in
// it), and the sum of its steps, exp(A sum D) being the decay over the range.
// ---------------------------------------------------------------------------
template <typename T, int N, int L, bool FULL> struct Layout {
    static constexpr int kCols = 64 / L;
    static constexpr int kRow = kCols * sizeof(T), kBRow = N * sizeof(T);
    static constexpr int kTensors = FULL ? 3 : 2, kMats = FULL ? 2 : 1;
    static constexpr int kStage = kTile * (kTensors * kRow + kMats * kBRow);
    static constexpr int kStep = 2 * kStage;                      // float4 [16][kCols / 2]
    static constexpr int kB = kStep + kTile * kCols / 2 * 16;     // float [16][N], then C
    static constexpr int kY = kB + kMats * kTile * N * 4;         // float [16][kYRow]
    static constexpr int kYRow = 64 + (kCols < 32 ? kCols : 0);   // floats: [L][kCols], padded for the banks
    static constexpr int kH = kY + (FULL ? kTile * kYRow * 4 : 0);  // slices: float4 [SL][2][32]
    static constexpr int kBytes = kH + (N > 16 ? N * 64 : 0);
};

struct ForwardWork {  // what ranges hand on
    float *q, *steps;  // [ranges][width][N], [ranges][width]
};

template <typename T, int NT, int L, int SL, bool FULL>
__global__ void __launch_bounds__(32) selective_forward_kernel(SelectiveArgs a, SelectiveShape sh, ForwardWork wk) {
    constexpr int N = L * NT * SL, P = NT / 2;
    using Lay = Layout<T, N, L, FULL>;
    constexpr int kCols = Lay::kCols, kQuads = kCols / 4;
    using Raw = typename Quad<T>::Raw;
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x, j = lane / (32 / L), cl = lane % (32 / L), r = blockIdx.y;
    const Columns cols(sh, blockIdx.x, kCols);
    const Ranges rg(a, sh.ranges);
    int t0 = rg.start(r);
    const int t1 = rg.start(r + 1);
    const int pair = cols.c0 + 2 * cl;
    const bool live = 2 * cl < cols.left;
    const int64_t states = (int64_t)pair * N + j * NT;  // this thread's first state of its first channel, slice 0
    if constexpr (FULL) {
        if (a.final_state)  // empty sequences keep their state
            for (int q = r; q < a.num_seqs; q += sh.ranges)
                if (__ldg(a.cu_seqlens + q) >= __ldg(a.cu_seqlens + q + 1) && live)
                    for (int i = j; i < 2 * N; i += L) {
                        const int64_t at = ((int64_t)q * sh.width + pair) * N + i;
                        a.final_state[at] = a.init ? a.init[at] : 0.f;
                    }
    } else {
        const int from = rg.origin(t1);
        if (t1 >= rg.end || from == t1) return;  // the next range begins a sequence
        if (from > t0) t0 = from;
    }
    if (t0 >= t1) return;
    const int origin = rg.origin(t0);

    F2 hs[2][P], As[2][P];  // the states at hand, and A log2 e
    auto load_A = [&](int s) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            no_pairs(As[c]);
            if (live) read_pairs(a.A + states + (int64_t)c * N + s * L * NT, As[c]);
#pragma unroll
            for (int k = 0; k < P; ++k) As[c][k] = mul2(As[c][k], both(kLog2e));
        }
    };
    // this thread's states in an array of [.., width, N] at row i
    auto get = [&](const float *p, int64_t i, int s) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            no_pairs(hs[c]);
            if (p && live) read_pairs(p + i * sh.width * N + states + (int64_t)c * N + s * L * NT, hs[c]);
        }
    };
    auto put = [&](float *p, int64_t i, int s) {
        if (live)
#pragma unroll
            for (int c = 0; c < 2; ++c) write_pairs(p + i * sh.width * N + states + (int64_t)c * N + s * L * NT, hs[c]);
    };
    // a slice's states between tiles: registers with one slice, else shared memory (4 NT bytes of a thread, then the next's)
    float *kept = reinterpret_cast<float *>(smem + Lay::kH) + lane * 4;
    auto keep = [&](int s) {
        if constexpr (SL > 1) {
            static_assert(NT == 4, "a word per channel");
#pragma unroll
            for (int c = 0; c < 2; ++c) write_pairs(kept + (s * 2 + c) * 128, hs[c]);
        }
    };
    auto recall = [&](int s) {
        if constexpr (SL > 1) {
#pragma unroll
            for (int c = 0; c < 2; ++c) read_pairs(kept + (s * 2 + c) * 128, hs[c]);
            load_A(s);
        }
    };

    // the states that the range starts from
    if constexpr (FULL) {
        if (origin < t0) {
            int r0 = r - 1;  // the range that the sequence begins in
            for (int i = r - 1; i > 0; i -= 32) {
                const uint32_t m = __ballot_sync(0xffffffffu, i - lane > 0 && rg.start(i - lane) > origin);
                r0 -= __popc(m);
                if (m != 0xffffffffu) break;
            }
            for (int s = 0; s < SL; ++s) {
                load_A(s);
                get(wk.q, r0, s);
                for (int i = r0 + 1; i < r; ++i) {
                    F2 now[2][P];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < P; ++k) now[c][k] = hs[c][k];
                    get(wk.q, i, s);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const F2 d = both(live ? wk.steps[(int64_t)i * sh.width + pair + c] : 0.f);
#pragma unroll
                        for (int k = 0; k < P; ++k) hs[c][k] = fma2(ex2_ftz(mul2(d, As[c][k])), now[c][k], hs[c][k]);
                    }
                }
                keep(s);
            }
        } else {
            get(nullptr, 0, 0);
            for (int s = 0; s < SL; ++s) keep(s);
        }
    } else {
        get(nullptr, 0, 0);
        for (int s = 0; s < SL; ++s) keep(s);
    }
    if constexpr (SL == 1) load_A(0);

    const int row_first = t0 & ~(kTile - 1);
    const int esz = (int)sizeof(T), live_bytes = cols.left * esz;
    const uint32_t smem_at = (uint32_t)__cvta_generic_to_shared(smem);
    auto fetch = [&](int row0, int stage) {
        if (row0 < t1) {
            const uint32_t at = smem_at + stage * Lay::kStage;
            const int64_t c = (int64_t)cols.c0 * esz, n = (int64_t)cols.g * N * esz;
            copy_rows<Lay::kRow>(at, static_cast<const char *>(a.x) + c, a.x_stride * esz, live_bytes, row0, t0, t1, a.x, lane);
            copy_rows<Lay::kRow>(at + kTile * Lay::kRow, static_cast<const char *>(a.delta) + c, a.delta_stride * esz, live_bytes,
                                 row0, t0, t1, a.x, lane);
            const uint32_t mats = at + kTile * Lay::kTensors * Lay::kRow;
            copy_rows<Lay::kBRow>(mats, static_cast<const char *>(a.B) + n, a.b_stride * esz, Lay::kBRow, row0, t0, t1, a.x, lane);
            if constexpr (FULL) {
                if (a.gate)
                    copy_rows<Lay::kRow>(at + 2 * kTile * Lay::kRow, static_cast<const char *>(a.gate) + c, a.gate_stride * esz,
                                         live_bytes, row0, t0, t1, a.x, lane);
                copy_rows<Lay::kBRow>(mats + kTile * Lay::kBRow, static_cast<const char *>(a.C) + n, a.c_stride * esz,
                                      Lay::kBRow, row0, t0, t1, a.x, lane);
            }
        }
        copies_commit();
    };

    // parts 1 and 3: lane has four channels of every fourth token
    const int qd = lane % kQuads, tq = lane / kQuads;
    const bool quad_live = qd * 4 < cols.left;
    F2 bias[2], skip[2];
    load_quad(a.delta_bias, cols.c0 + qd * 4, quad_live, bias);
    load_quad(FULL ? a.skip : nullptr, cols.c0 + qd * 4, quad_live, skip);
    F2 steps = both(0.f);  // sums of this thread's channels' steps
    float4 *step = reinterpret_cast<float4 *>(smem + Lay::kStep);
    float *bs = reinterpret_cast<float *>(smem + Lay::kB), *cs = bs + kTile * N;
    float *ys = reinterpret_cast<float *>(smem + Lay::kY);
    Edges ed;
    fetch(row_first, 0);
    int stage = 0;
    for (int row0 = row_first; row0 < t1; row0 += kTile, stage ^= 1) {
        fetch(row0 + kTile, stage ^ 1);
        ed.find(rg, row0, t0, t1, lane);
        copies_wait<1>();
        const char *at = smem + stage * Lay::kStage;
#pragma unroll
        for (int k = 0; k < kTile; k += 32 / kQuads) {
            const int i = k + tq, t = row0 + i;
            F2 x[2], d[2];
            Quad<T>::unpack(*reinterpret_cast<const Raw *>(at + i * Lay::kRow + qd * 4 * esz), x);
            Quad<T>::unpack(*reinterpret_cast<const Raw *>(at + (kTile + i) * Lay::kRow + qd * 4 * esz), d);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                d[p] = softplus2(add2(d[p], bias[p]));
                if (t < t0 || t >= t1) d[p] = both(0.f);  // neither decay nor input
                x[p] = mul2(x[p], d[p]);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {  // banks: every other four lanes the other pair first
                const bool other = (p ^ (lane >> 2)) & 1;
                const float2 u = f2_get(other ? d[1] : d[0]), v = f2_get(other ? x[1] : x[0]);
                step[i * (kCols / 2) + qd * 2 + other] = make_float4(u.x, u.y, v.x, v.y);
            }
        }
        {
            const char *mats = at + kTile * Lay::kTensors * Lay::kRow;
#pragma unroll
            for (int k = lane; k < Lay::kMats * kTile * N / 4; k += 32) {
                F2 f[2];
                Quad<T>::unpack(*reinterpret_cast<const Raw *>(mats + k * 4 * esz), f);
                const float2 u = f2_get(f[0]), v = f2_get(f[1]);
                *reinterpret_cast<float4 *>(bs + k * 4) = make_float4(u.x, u.y, v.x, v.y);
            }
        }
        __syncwarp();
        for (int s = 0; s < SL; ++s) {
            recall(s);
            if constexpr (FULL)
                if (a.checkpoints && row0 >= t0) put(a.checkpoints, row0 / kTile, s);
            auto token = [&](int i) {  // returns this thread's part of y
                const float4 d = step[i * (kCols / 2) + cl];
                const float *bt = bs + i * N + s * L * NT + j * NT, *ct = cs + i * N + s * L * NT + j * NT;
                F2 B[P], y[2] = {both(0.f), both(0.f)};
                read_pairs(bt, B);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const F2 dc = both(c ? d.y : d.x), xc = both(c ? d.w : d.z);
#pragma unroll
                    for (int k = 0; k < P; ++k)
                        hs[c][k] = fma2(ex2_ftz(mul2(dc, As[c][k])), hs[c][k], mul2(xc, B[k]));
                }
                if constexpr (FULL) {
                    F2 C[P];
                    read_pairs(ct, C);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < P; ++k) y[c] = fma2(hs[c][k], C[k], y[c]);
                } else if (s == 0) {
                    steps = add2(steps, f2(d.x, d.y));
                }
                const float2 u = f2_get(y[0]), v = f2_get(y[1]);
                return make_float2(u.x + u.y, v.x + v.y);
            };
            auto leave = [&](int i, float2 part) {
                if constexpr (FULL) {
                    float2 *to = reinterpret_cast<float2 *>(ys + i * Lay::kYRow + j * kCols + cl * 2);
                    if (SL > 1 && s) part.x += to->x, part.y += to->y;
                    *to = part;
                }
            };
            if ((ed.starts | ed.ends) == 0) {
                // four tokens' loads before their stores
#pragma unroll 1
                for (int i = 0; i < kTile; i += 4) {
                    float2 part[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) part[u] = token(i + u);
#pragma unroll
                    for (int u = 0; u < 4; ++u) leave(i + u, part[u]);
                }
            } else {
                for (int i = 0; i < kTile; ++i) {
                    if ((ed.starts >> i) & 1u) get(a.init, __shfl_sync(0xffffffffu, ed.seq, i), s);
                    leave(i, token(i));
                    if constexpr (FULL) {
                        const int q = __shfl_sync(0xffffffffu, ed.seq, i);
                        if (((ed.ends >> i) & 1u) && a.final_state) put(a.final_state, q, s);
                    }
                }
            }
            keep(s);
        }
        __syncwarp();
        if constexpr (FULL) {
#pragma unroll
            for (int k = 0; k < kTile; k += 32 / kQuads) {
                const int i = k + tq, t = row0 + i;
                F2 y[2] = {both(0.f), both(0.f)}, x[2];
#pragma unroll
                for (int l = 0; l < L; ++l) {
                    const float4 u = *reinterpret_cast<const float4 *>(ys + i * Lay::kYRow + l * kCols + qd * 4);
                    y[0] = add2(y[0], f2(u.x, u.y));
                    y[1] = add2(y[1], f2(u.z, u.w));
                }
                Quad<T>::unpack(*reinterpret_cast<const Raw *>(at + i * Lay::kRow + qd * 4 * esz), x);
                y[0] = fma2(skip[0], x[0], y[0]);
                y[1] = fma2(skip[1], x[1], y[1]);
                if (a.gate) {
                    F2 z[2];
                    Quad<T>::unpack(*reinterpret_cast<const Raw *>(at + (2 * kTile + i) * Lay::kRow + qd * 4 * esz), z);
                    y[0] = mul2(y[0], mul2(z[0], sigmoid2<T>(z[0])));
                    y[1] = mul2(y[1], mul2(z[1], sigmoid2<T>(z[1])));
                }
                if (t >= t0 && t < t1 && quad_live)
                    *reinterpret_cast<Raw *>(static_cast<T *>(a.out) + (int64_t)t * sh.width + cols.c0 + qd * 4) = Quad<T>::pack(y);
            }
            __syncwarp();  // the stage is free
        }
    }
    if constexpr (!FULL) {
        for (int s = 0; s < SL; ++s) {
            recall(s);
            put(wk.q, r, s);
        }
        if (j == 0 && live) *reinterpret_cast<float2 *>(wk.steps + (int64_t)r * sh.width + pair) = f2_get(steps);
    }
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

enum What { kForward, kStep };

template <typename T, int N> cudaError_t launch_forward(const sse_selective_config_t &c, const SelectiveArgs &a, cudaStream_t s) {
    constexpr int L = kL, NT = N / L < kNT ? N / L : kNT, SL = N / (L * NT);
    const SelectiveShape sh = selective_shape(c, 64 / kL, a.total_tokens);
    ForwardWork wk;
    wk.q = reinterpret_cast<float *>(a.workspace);
    wk.steps = wk.q + (int64_t)sh.ranges * c.width * N;
    const dim3 grid(sh.tiles * c.groups, sh.ranges);
    const auto states = selective_forward_kernel<T, NT, L, SL, false>, full = selective_forward_kernel<T, NT, L, SL, true>;
    constexpr int kStates = Layout<T, N, L, false>::kBytes, kFull = Layout<T, N, L, true>::kBytes;
    if constexpr (kFull > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(full, cudaFuncAttributeMaxDynamicSharedMemorySize, kFull);
        if (e != cudaSuccess) return e;
    }
    static_assert(kStates <= 48 * 1024, "the default limit");
    if (sh.ranges > 1) states<<<grid, 32, kStates, s>>>(a, sh, wk);
    full<<<grid, 32, kFull, s>>>(a, sh, wk);
    return cudaGetLastError();
}

template <typename T, int L>
cudaError_t launch_t(What what, const sse_selective_config_t &c, const SelectiveArgs &a, cudaStream_t s) {
    if (what == kStep) {
        const int64_t blocks = ((int64_t)a.num_seqs * c.width * L + 255) / 256;
        if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
        selective_step_kernel<T, L><<<(unsigned)blocks, 256, 0, s>>>(a, c);
        return cudaGetLastError();
    }
    return launch_forward<T, 4 * L>(c, a, s);
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

size_t selective_forward_workspace(const sse_selective_config_t &c, int64_t T, int32_t) {
    const SelectiveShape s = selective_shape(c, 64 / kL, T);
    return s.ranges > 1 ? sizeof(float) * (size_t)s.ranges * c.width * (c.state + 1) : 0;
}
cudaError_t launch_selective_forward(const sse_selective_config_t &cfg, const SelectiveArgs &a, cudaStream_t stream) {
    return launch(kForward, cfg, a, stream);
}
cudaError_t launch_selective_step(const sse_selective_config_t &cfg, const SelectiveArgs &a, cudaStream_t stream) {
    return launch(kStep, cfg, a, stream);
}

}  // namespace sse
