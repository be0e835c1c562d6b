// selective.cu -- the selective state space scan: per channel c and state n, with
// D_t = softplus(delta_t + delta_bias) and a_t[n] = exp(D_t A[n]),
//   h_t[n] = a_t[n] h_{t-1}[n] + D_t B_t[n] x_t
//   y_t = sum_n C_t[n] h_t[n] + skip x_t,   out_t = y_t silu(gate_t)
// Gradients, with dy = d_out silu(gate) and g_t[n] = C_t[n] dy_t + a_{t+1}[n] g_{t+1}[n]:
//   d_gate = d_out y silu'(gate),  dx = skip dy + D sum_n B g
//   dD = x sum_n B g + sum_n A g a h_{t-1},  d_delta = dD softplus'
//   dB[n] = sum_c g D x,  dC[n] = sum_c dy h  (over the channels of the group)
//   dA = sum_t D g a h_{t-1},  d_skip = sum_t dy x,  d_delta_bias = sum_t d_delta
//
// The states never leave the SM, so HBM would allow a pass over 32768 x 2048 in 79 us
// (6.77 TB/s), but a token and channel of 8 bytes has 16 exponentials and about 110
// other operations.  For two states of 32 channels a warp issues four instructions of
// pairs (the exponent, D x B, the state, C h), two exponentials and a 16-byte load:
// 32 exponentials a clock and SM are 115 us, and the pairs, whose three distinct
// operands take the register ports three cycles, about 280.
// Measured on a GB300 in bf16, 16 states, gate and skip: 8 x 4096 x 2048 529 us, one
// sequence of 32768 514 (of either some 200 are the ranges' states), 16 x 2048 x 2048, whose
// sequences need no such states, 387, 24001 x 2048 in 16 ragged ones 399, a prompt of 500
// x 1024 27; checkpoints are 8 to 11 us of 32768 x 2048; issue 62 %, FMA pipe 51 %,
// exponentials 41 % busy.  Token by token with a
// lane per four states: 8 x 4096 x 2048 about 5 ms.
#include <type_traits>

#include "selective.cuh"

namespace sse {
namespace {

template <int L> __device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------------------
// Forward.  A warp is a CTA; it has 32 channels of a group, one to a lane with
// its states in registers (two slices of 32 where there are 64), and one range of
// tokens, which it goes through four tokens at a time.  Rows come to shared memory
// by asynchronous copies two tiles of 16 tokens ahead; B and C are turned to
// float32 there, and every lane reads the same 16 bytes.  The next four tokens'
// steps (pairs over the tokens) are made beside these four's states (pairs over
// the states), in one stretch of code without branches.
// kStates makes only what a later range starts from: the state at the range's end
// from nothing (or from the sequence that begins in it), and the sum of its steps,
// exp(A sum D) being the decay over the range.
//
// A channel per lane needs no shuffle and no second copy of the steps, and 64 registers
// hold states and A: four lanes to a channel pair took 607 us for 32768 x 2048 (531
// now).  Two warps to a CTA, a warp that only copies, and half of the states or of the
// channels to a lane were slower or the same.
// ---------------------------------------------------------------------------
constexpr int kCols = 32;           // channels of a warp
constexpr int kAlone = 1000;        // warps that sequences make by themselves, for a range each
constexpr int kQuarters = 4 * 152;  // of the SMs
constexpr int kBlock = 4;           // tokens at a time

// What a kernel makes: the states that later ranges start from, the forward without and with a gate.
enum { kStates, kPlain, kGated };

template <typename T, int N, int MODE> struct Layout {
    static constexpr int NT = N < 32 ? N : 32, SL = N / NT;
    static constexpr int kRow = kCols * sizeof(T), kBRow = N * sizeof(T);
    static constexpr int kTensors = MODE == kGated ? 3 : 2, kMats = MODE == kStates ? 1 : 2;
    static constexpr int kX = 0, kD = kTile * kRow, kZ = 2 * kD;  // a stage: x, delta, gate; B and C
    static constexpr int kMat = kTensors * kD;
    static constexpr int kStage = kMat + kMats * kTile * kBRow;
    static constexpr int kB = 3 * kStage;                     // float [16][N]: B, then C
    static constexpr int kKept = kB + kMats * kTile * N * 4;  // slices: states and A log2 e, float4 [SL][2][NT / 4][32]
    static constexpr int kBytes = kKept + (SL > 1 ? SL * 2 * NT * 128 : 0);
};

struct ForwardWork {  // what ranges hand on
    float *q, *steps;  // [ranges][width][N], [ranges][width]
};

template <typename T, int N, int MODE>
__global__ void __launch_bounds__(32, 1) selective_forward_kernel(SelectiveArgs a, SelectiveShape sh, ForwardWork wk) {
    using Lay = Layout<T, N, MODE>;
    using Raw = typename Two<T>::Raw;
    constexpr bool FULL = MODE != kStates;
    constexpr int NT = Lay::NT, SL = Lay::SL, P = NT / 2;
    extern __shared__ __align__(16) char smem[];
    const int lane = threadIdx.x, r = blockIdx.y;
    const Columns cols(sh, blockIdx.x, kCols);
    const Ranges rg(a, sh, [](const int32_t *cu, int S, int end) { return even_sequences(cu, S, end); });
    int t0 = rg.start(r);
    const int t1 = rg.start(r + 1);
    const bool live = lane < cols.left;
    const int ch = cols.c0 + (live ? lane : 0);
    const int64_t states = (int64_t)ch * N;  // this thread's first state
    if constexpr (FULL) {
        if (a.final_state)  // empty sequences keep their state
            each_empty(a.cu_seqlens, a.num_seqs, r, sh.ranges, lane, 32, [&](int q) {
                const int64_t at = (int64_t)q * sh.width * N + states;
                if (live) copy_words<N / 4, 1>(a.final_state + at, a.init ? a.init + at : nullptr);
            });
    } else {
        const int from = rg.origin(t1);
        if (t1 >= rg.end || from == t1) return;  // the next range begins a sequence
        if (from > t0) t0 = from;
    }
    if (t0 >= t1) return;
    const int origin = rg.origin(t0);

    F2 h[P], A[P];  // of the slice at hand; A log2 e
    auto load_A = [&](int s) {
        read_pairs(a.A + states + s * NT, A);
#pragma unroll
        for (int k = 0; k < P; ++k) A[k] = mul2(A[k], both(live ? kLog2e : 0.f));
    };
    // this thread's states in an array of [.., width, N] at row i
    auto get = [&](const float *p, int64_t i, int s) {
        if (p) {
            read_pairs(p + i * sh.width * N + states + s * NT, h);
        } else {
#pragma unroll
            for (int k = 0; k < P; ++k) h[k] = both(0.f);
        }
    };
    auto put = [&](float *p, int64_t i, int s) {
        if (live) write_pairs(p + i * sh.width * N + states + s * NT, h);
    };
    // a slice between blocks: registers with one slice, else shared memory
    float *kept = reinterpret_cast<float *>(smem + Lay::kKept) + lane * 4;
    auto keep = [&](int s, int which, const F2 (&f)[P]) {
#pragma unroll
        for (int k = 0; k < P; k += 2) {
            const F2 two[2] = {f[k], f[k + 1]};
            write_quad(kept + ((s * 2 + which) * (NT / 4) + k / 2) * 128, two);
        }
    };
    auto recall = [&](int s, int which, F2 (&f)[P]) {
#pragma unroll
        for (int k = 0; k < P; k += 2) {
            F2 two[2];
            read_quad(kept + ((s * 2 + which) * (NT / 4) + k / 2) * 128, two);
            f[k] = two[0], f[k + 1] = two[1];
        }
    };

    // the states that the range starts from
    int r0 = r;  // the range that the sequence at its start begins in
    if (FULL && origin < t0) {
        r0 = r - 1;
        for (int i = r - 1; i > 0; i -= 32) {
            const uint32_t m = __ballot_sync(0xffffffffu, i - lane > 0 && rg.start(i - lane) > origin);
            r0 -= __popc(m);
            if (m != 0xffffffffu) break;
        }
    }
    for (int s = 0; s < SL; ++s) {
        load_A(s);
        get(r0 < r ? wk.q : nullptr, r0, s);
        for (int i = r0 + 1; i < r; ++i) {
            F2 now[P];
            const F2 d = both(wk.steps[(int64_t)i * sh.width + ch]);
#pragma unroll
            for (int k = 0; k < P; ++k) now[k] = h[k];
            get(wk.q, i, s);
#pragma unroll
            for (int k = 0; k < P; ++k) h[k] = fma2(ex2_ftz(mul2(d, A[k])), now[k], h[k]);
        }
        if constexpr (SL > 1) {
            keep(s, 0, h);
            keep(s, 1, A);
        }
    }

    // A tile's rows, two tiles ahead.  Rows outside the range and channels past the group's end are zeros.
    const int esz = (int)sizeof(T), live_bytes = cols.left * esz;
    const uint32_t smem_at = (uint32_t)__cvta_generic_to_shared(smem);
    float *bs = reinterpret_cast<float *>(smem + Lay::kB), *cs = bs + kTile * N;
    auto fetch = [&](int row0, int stage) {
        if (row0 < t1) {
            const uint32_t at = smem_at + stage * Lay::kStage;
            const int64_t c = (int64_t)cols.c0 * esz, n = (int64_t)cols.g * N * esz;
            copy_rows<Lay::kRow>(at + Lay::kX, static_cast<const char *>(a.x) + c, a.x_stride * esz, live_bytes, row0, t0, t1,
                                 a.x, lane);
            copy_rows<Lay::kRow>(at + Lay::kD, static_cast<const char *>(a.delta) + c, a.delta_stride * esz, live_bytes, row0,
                                 t0, t1, a.x, lane);
            if constexpr (MODE == kGated)
                copy_rows<Lay::kRow>(at + Lay::kZ, static_cast<const char *>(a.gate) + c, a.gate_stride * esz, live_bytes, row0,
                                     t0, t1, a.x, lane);
            copy_rows<Lay::kBRow>(at + Lay::kMat, static_cast<const char *>(a.B) + n, a.b_stride * esz, Lay::kBRow, row0, t0,
                                  t1, a.x, lane);
            if constexpr (FULL)
                copy_rows<Lay::kBRow>(at + Lay::kMat + kTile * Lay::kBRow, static_cast<const char *>(a.C) + n,
                                      a.c_stride * esz, Lay::kBRow, row0, t0, t1, a.x, lane);
        }
        copies_commit();
    };
    const float bias = a.delta_bias ? a.delta_bias[ch] : 0.f, skip = FULL && a.skip ? a.skip[ch] : 0.f;
    // This channel's values of tokens i and i + 1 of a tile, as a pair.
    auto two = [&](const char *stage, int tensor, int i) {
        const Raw *at = reinterpret_cast<const Raw *>(stage + tensor) + lane;
        return Two<T>::unpack(at[i * kCols], at[(i + 1) * kCols]);
    };
    struct Steps {
        F2 d[kBlock / 2], dx[kBlock / 2];  // D and D x, pairs over the tokens
    };
    auto steps_of = [&](const char *stage, int i, int row, bool whole) {
        Steps s;
        F2 none;
#pragma unroll
        for (int u = 0; u < kBlock; u += 2) {
            F2 d = softplus2<false>(add2(two(stage, Lay::kD, i + u), both(bias)), none);
            if (!whole) {  // rows outside: neither decay nor input (their x is 0)
                const float2 f = f2_get(d);
                d = f2(row + u >= t0 && row + u < t1 ? f.x : 0.f, row + u + 1 >= t0 && row + u + 1 < t1 ? f.y : 0.f);
            }
            s.d[u / 2] = d;
            s.dx[u / 2] = mul2(d, two(stage, Lay::kX, i + u));
        }
        return s;
    };

    F2 steps = both(0.f);  // sums of this channel's steps
    Edges ed;
    const int first = t0 & ~(kBlock - 1), tile_first = first & ~(kTile - 1);
    fetch(tile_first, 0);
    fetch(tile_first + kTile, 1);
    copies_wait<1>();
    const char *here = smem, *ahead = smem + Lay::kStage;  // this tile's stage and the next one's
    int free_stage = 2;
    Steps st = steps_of(here, first - tile_first, first, false);
    for (int tile = tile_first; tile < t1; tile += kTile) {
        ed.find(rg, tile, t0, t1, lane);
        fetch(tile + 2 * kTile, free_stage);
        copies_wait<1>();  // the next tile is there, and the tile before has been read
        const typename Quad<T>::Raw *mats = reinterpret_cast<const typename Quad<T>::Raw *>(here + Lay::kMat);
#pragma unroll
        for (int k = lane; k < Lay::kMats * kTile * N / 4; k += 32) {
            F2 f[2];
            Quad<T>::unpack(mats[k], f);
            write_quad(bs + k * 4, f);
        }
        __syncwarp();
        if constexpr (FULL)
            if (a.checkpoints && tile >= t0)
                for (int s = 0; s < SL; ++s) {
                    if constexpr (SL > 1) recall(s, 0, h);
                    put(a.checkpoints, tile / kTile, s);
                }
        // PLAIN: no sequence begins or ends in the tile, and it and the next block are within the range
        auto block = [&](auto plain, int i0) {
            constexpr bool PLAIN = decltype(plain)::value;
            const int row = tile + i0, i1 = (i0 + kBlock) % kTile;
            const Steps st_next = steps_of(i1 ? here : ahead, i1, row + kBlock, PLAIN);
            F2 y[kBlock];
#pragma unroll
            for (int u = 0; u < kBlock; ++u) y[u] = both(0.f);
#pragma unroll
            for (int s = 0; s < SL; ++s) {
                if constexpr (SL > 1) {
                    recall(s, 0, h);
                    recall(s, 1, A);
                }
#pragma unroll
                for (int u = 0; u < kBlock; ++u) {
                    const int i = i0 + u;
                    const int q = PLAIN ? 0 : __shfl_sync(0xffffffffu, ed.seq, i);
                    if (!PLAIN && ((ed.starts >> i) & 1u)) get(a.init, q, s);
                    const float2 d = f2_get(st.d[u / 2]), dx = f2_get(st.dx[u / 2]);
                    const F2 dc = both(u & 1 ? d.y : d.x), xc = both(u & 1 ? dx.y : dx.x);
                    F2 B[P];
                    read_pairs(bs + i * N + s * NT, B);
#pragma unroll
                    for (int k = 0; k < P; ++k) h[k] = fma2(decay2(dc, A[k]), h[k], mul2(xc, B[k]));
                    if constexpr (FULL) {
                        F2 C[P];
                        read_pairs(cs + i * N + s * NT, C);
#pragma unroll
                        for (int k = 0; k < P; ++k) y[u] = fma2(h[k], C[k], y[u]);
                        if constexpr (!PLAIN)
                            if (((ed.ends >> i) & 1u) && a.final_state) put(a.final_state, q, s);
                    }
                }
                if constexpr (SL > 1) keep(s, 0, h);
            }
            if constexpr (FULL) {
#pragma unroll
                for (int u = 0; u < kBlock; u += 2) {
                    F2 o = fma2(both(skip), two(here, Lay::kX, i0 + u), f2(fold(y[u]), fold(y[u + 1])));
                    if constexpr (MODE == kGated) {
                        const F2 z = two(here, Lay::kZ, i0 + u);
                        o = mul2(o, mul2(z, sigmoid2<T>(z)));
                    }
                    T *to = static_cast<T *>(a.out) + (int64_t)(row + u) * sh.width + ch;
                    Two<T>::store(to, to + sh.width, o, live && (PLAIN || (row + u >= t0 && row + u < t1)),
                                  live && (PLAIN || (row + u + 1 >= t0 && row + u + 1 < t1)));
                }
            } else {
#pragma unroll
                for (int u = 0; u < kBlock / 2; ++u) steps = add2(steps, st.d[u]);
            }
            st = st_next;
        };
        if ((ed.starts | ed.ends) == 0 && tile >= t0 && tile + kTile + kBlock <= t1) {
#pragma unroll 1
            for (int i = 0; i < kTile; i += kBlock) block(std::true_type{}, i);
        } else {
#pragma unroll 1
            for (int i = max(first - tile, 0); i < kTile && tile + i < t1; i += kBlock) block(std::false_type{}, i);
        }
        __syncwarp();
        free_stage = free_stage == 2 ? 0 : free_stage + 1;
        here = ahead;
        ahead = smem + (free_stage == 0 ? 2 : free_stage - 1) * Lay::kStage;
    }
    if constexpr (!FULL) {
        for (int s = 0; s < SL; ++s) {
            if constexpr (SL > 1) recall(s, 0, h);
            put(wk.q, r, s);
        }
        if (live) wk.steps[(int64_t)r * sh.width + ch] = fold(steps);
    }
}

// One token of each sequence: L lanes for a pair of channels, four states of both each.  The states in and out are what it
// has to move; bound by their loads, one word of each a thread.  256 x 2048 with 16 states, more than L2 holds in turn, 18.1
// us (floor 10.6), the same state again and again 16.6 (one channel and library functions per thread 25), 8 states 10.4,
// 512 x 2048 with 64 133 (80).
template <typename T, int L>
__global__ void __launch_bounds__(256) selective_step_kernel(SelectiveArgs a, sse_selective_config_t cfg) {
    constexpr int N = 4 * L;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, pair = i / L;
    const int pairs = cfg.width / 2, n0 = (int)(i % L) * 4;
    int64_t b = pair / pairs;
    const bool live = b < a.num_seqs;
    if (!__any_sync(0xffffffffu, live)) return;
    if (!live) b = a.num_seqs - 1;
    const int c = (int)(live ? pair - b * pairs : 0) * 2, at = c / (cfg.width / cfg.groups) * N + n0;
    float *state = a.final_state + (b * cfg.width + c) * N + n0;
    F2 h[2][2], A[2][2], B[2], C[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        read_quad(state + k * N, h[k]);
        read_quad(a.A + (int64_t)(c + k) * N + n0, A[k]);
    }
    Quad<T>::unpack(*reinterpret_cast<const typename Quad<T>::Raw *>(static_cast<const T *>(a.B) + b * a.b_stride + at), B);
    Quad<T>::unpack(*reinterpret_cast<const typename Quad<T>::Raw *>(static_cast<const T *>(a.C) + b * a.c_stride + at), C);
    auto two = [](const void *p, int64_t at) {  // neighbouring channels
        const typename Two<T>::Raw *v = static_cast<const typename Two<T>::Raw *>(p) + at;
        return Two<T>::unpack(v[0], v[1]);
    };
    auto vector = [&](const float *p) {
        const float2 v = p ? *reinterpret_cast<const float2 *>(p + c) : make_float2(0.f, 0.f);
        return f2(v.x, v.y);
    };
    F2 none;
    const F2 x = two(a.x, b * a.x_stride + c);
    const F2 d = softplus2<false>(add2(two(a.delta, b * a.delta_stride + c), vector(a.delta_bias)), none), in = mul2(d, x);
    const float2 dv = f2_get(d), iv = f2_get(in);
    float y[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const F2 dk = both((k ? dv.y : dv.x) * kLog2e), ik = both(k ? iv.y : iv.x);
#pragma unroll
        for (int m = 0; m < 2; ++m) h[k][m] = fma2(decay2(dk, A[k][m]), h[k][m], mul2(ik, B[m]));
        y[k] = lanes_sum<L>(fold(fma2(h[k][0], C[0], mul2(h[k][1], C[1]))));
        if (live) write_quad(state + k * N, h[k]);
    }
    if (!live || n0) return;
    F2 o = fma2(vector(a.skip), x, f2(y[0], y[1]));
    if (a.gate) {
        const F2 z = two(a.gate, b * a.gate_stride + c);
        o = mul2(o, mul2(z, sigmoid2<T>(z)));
    }
    T *to = static_cast<T *>(a.out) + b * cfg.width + c;
    Two<T>::store(to, to + 1, o, true, true);
}

enum What { kForward, kStep };

// Warps of an SM quarter, by the registers that N states take: 4, 3, 2, 2.
SelectiveShape forward_shape(const sse_selective_config_t &c, int64_t T, int32_t S) {
    SelectiveShape s = selective_shape(c, kCols);
    const double held = c.state == 8 ? 4 : c.state == 16 ? 3 : 2;
    const Waves choices[] = {{2 * held, 400}, {held, 256}, {2, 96}, {1, 4 * kTile}};
    set_ranges(s, ranges_that_fill(s.tiles * c.groups, kQuarters, choices, T), kAlone, S);
    return s;
}

template <typename T, int N> cudaError_t launch_forward(const sse_selective_config_t &c, const SelectiveArgs &a, cudaStream_t s) {
    const SelectiveShape sh = forward_shape(c, a.total_tokens, a.num_seqs);
    ForwardWork wk;
    wk.q = reinterpret_cast<float *>(a.workspace);
    wk.steps = wk.q + (int64_t)sh.ranges * c.width * N;
    const dim3 grid(sh.tiles * c.groups, sh.ranges);
    const auto states = selective_forward_kernel<T, N, kStates>;
    const auto full = a.gate ? selective_forward_kernel<T, N, kGated> : selective_forward_kernel<T, N, kPlain>;
    constexpr int kGatedBytes = Layout<T, N, kGated>::kBytes;
    static_assert(Layout<T, N, kStates>::kBytes <= 48 * 1024 && Layout<T, N, kPlain>::kBytes <= kGatedBytes, "shared memory");
    if constexpr (kGatedBytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(full, cudaFuncAttributeMaxDynamicSharedMemorySize, kGatedBytes);
        if (e != cudaSuccess) return e;
    }
    if (sh.ranges > 1) states<<<grid, 32, Layout<T, N, kStates>::kBytes, s>>>(a, sh, wk);
    full<<<grid, 32, a.gate ? kGatedBytes : Layout<T, N, kPlain>::kBytes, s>>>(a, sh, wk);
    return cudaGetLastError();
}

template <typename T, int L>
cudaError_t launch_t(What what, const sse_selective_config_t &c, const SelectiveArgs &a, cudaStream_t s) {
    if (what == kStep) {
        const int64_t blocks = ((int64_t)a.num_seqs * (c.width / 2) * L + 255) / 256;
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

size_t selective_forward_workspace(const sse_selective_config_t &c, int64_t T, int32_t S) {
    const SelectiveShape s = forward_shape(c, T, S);
    return s.ranges > 1 ? sizeof(float) * (size_t)s.ranges * c.width * (c.state + 1) : 0;
}
cudaError_t launch_selective_forward(const sse_selective_config_t &cfg, const SelectiveArgs &a, cudaStream_t stream) {
    return launch(kForward, cfg, a, stream);
}
cudaError_t launch_selective_step(const sse_selective_config_t &cfg, const SelectiveArgs &a, cudaStream_t stream) {
    return launch(kStep, cfg, a, stream);
}

}  // namespace sse
