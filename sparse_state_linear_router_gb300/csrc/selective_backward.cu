// selective_backward.cu -- the gradients of the selective scan (formulas at the
// head of selective.cu).
//
// A warp has 16 channels of a group and one range of tokens, which it goes
// through backwards in tiles of 16.  Four lanes share a pair of channels, NT
// states each (lane = j * 8 + pair); SL slices of 4 NT states.  Per tile:
//   1. steps D and D x, dy, B and C in float32 to shared memory, lanes over
//      (token, four channels);
//   2. in halves of 8 tokens, the later one first: forwards from the checkpoint,
//      the decays and the states before the half's tokens in registers; then
//      backwards: g = C dy + e, e = a g, and this thread's parts of the sums over
//      states (y, sum B g, sum A g a h) and over channels (dB, dC);
//   3. the sums over states, lanes over (token, four channels), and with them
//      dx, d_delta, d_gate.
// The sums over channels go over the eight pairs of a warp by shuffles, over the
// four warps of a CTA through shared memory, and over the CTAs of a group in a
// second kernel: a float32 row of 2 N for each token and 64 channels.  Every sum
// has a fixed order.  B and C are in shared memory twice over, so that a pair over
// the channels takes a value as it is.
//
// Bound by instructions: about 48 of a warp for 64 (token, channel, state), 19 of them
// arithmetic of pairs and 9 the sums over channels, against 14 bytes and 16
// exponentials for a token and channel (159 us of HBM, 115 of exponentials for 8 x 4096
// x 2048 with 16 states).  Measured on a GB300, bf16: 1523 us there, 1567 as one
// sequence of 32768, 24001 x 2048 in 16 ragged sequences 1222, 64 x 512 x 512 421;
// issue 46 %, shared memory's pipe 56 %, FMA 41 %.  255 registers leave eight warps to
// an SM.  Spans of 4 tokens, whose 168 registers let twelve in, took 2623 us (1.75
// passes forwards instead of 1.5, and what did not fit in registers went to L2, shared
// memory having taken the L1); every step of a tile through shared memory 1655.
#include <type_traits>

#include "selective.cuh"

namespace sse {
namespace {

constexpr int kL = 4, kCols = 16;
constexpr int kAlone = 1000;  // warps that sequences make by themselves, for a range each
constexpr int kSpan = 8;      // tokens whose states are held in registers, and of an epilogue
constexpr int kPart = 1024;   // tokens of a sum for the weights

template <typename T, int N, bool FULL> struct Layout {
    static constexpr int NT = N == 8 ? 2 : 4, SL = N / (kL * NT);
    static constexpr int kWarps = FULL ? 4 : 1;
    static constexpr int kRow = kCols * sizeof(T), kBRow = N * sizeof(T);
    static constexpr int kMats = FULL ? 2 : 1;  // C, B
    // of a warp
    static constexpr int kCheck = kTile * (FULL ? 4 : 3) * kRow;  // delta, d_out, gate, x
    static constexpr int kStage = kCheck + (FULL ? kCols * N * 4 : 0);
    static constexpr int kStep = 2 * kStage;                    // float4 [16][8]: D0, D1, D x0, D x1
    static constexpr int kDy = kStep + kTile * kCols / 2 * 16;  // float [16][16]
    static constexpr int kSlope = kDy + kTile * kCols * 4;      // float [2][16][16]: softplus', d_out silu'(gate)
    static constexpr int kPart = kSlope + (FULL ? 2 * kTile * kCols * 4 : 0);  // float [3][8][4][16]: y, sum B g, sum A g a h
    static constexpr int kKept = kPart + (FULL ? 3 * kSpan * kL * kCols * 4 : 0);  // slices: e and dA, float4 [SL][2][2][32]
    static constexpr int kWarpBytes = kKept + (SL > 1 ? SL * 4 * 32 * 16 : 0);
    // of the CTA
    static constexpr int kMat = kTile * kBRow * kMats;
    static constexpr int kRaw = kWarps * kWarpBytes;            // C and B as stored, two stages
    static constexpr int kC = kRaw + 2 * kMat;                  // float [16][N][2]: C, then B, each value twice
    static constexpr int kSums = kC + kMats * kTile * N * 8;    // float [2][kWarps][8][32]
    static constexpr int kBytes = kSums + (FULL ? 2 * kWarps * kSpan * 32 * 4 : 0);
};

struct BackwardWork {
    float *q, *steps;   // what ranges hand on: [ranges][width][N], [ranges][width]
    float *tokens;      // [parts][T][groups][2 N]: dB and dC of 64 channels
    float *weights;     // [ranges][width][N + 2]: dA, d_skip, d_delta_bias
    int parts;          // CTAs of a group
};

// Not inline: the kernel's registers would be given out worse for it (8 x 4096 x 2048 1546 us instead of 1515).
__device__ __noinline__ bool even_sequences_called(const int32_t *cu, int S, int end) { return even_sequences(cu, S, end); }

// FULL: the gradients.  Otherwise what an earlier range starts from: e at the range's first token from nothing behind it
// (or from the sequence that ends in it), and the sum of its steps.
template <typename T, int N, bool FULL>
__global__ void __launch_bounds__(32 * Layout<T, N, FULL>::kWarps, FULL ? 2 : 1)
selective_backward_kernel(SelectiveArgs a, SelectiveShape sh, BackwardWork wk) {
    using Lay = Layout<T, N, FULL>;
    using Raw = typename Quad<T>::Raw;
    constexpr int NT = Lay::NT, SL = Lay::SL, kQuads = kCols / 4, kWarps = Lay::kWarps;
    extern __shared__ __align__(16) char all_smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, j = lane >> 3, cl = lane & 7, r = blockIdx.y;
    char *smem = all_smem + (FULL ? warp * Lay::kWarpBytes : 0);
    const int g = blockIdx.x / (FULL ? wk.parts : sh.tiles), part = blockIdx.x - g * (FULL ? wk.parts : sh.tiles);
    const int first = (FULL ? part * kWarps + warp : part) * kCols;
    const int left = max(0, min(kCols, sh.per - first)), c0 = g * sh.per + (left ? first : 0);
    const Ranges rg(a, sh, even_sequences_called);
    const int t0 = rg.start(r);
    int t1 = rg.start(r + 1);
    const int pair = c0 + 2 * cl;
    const bool live = 2 * cl < left;
    const int64_t states = (int64_t)pair * N + j * NT;
    if constexpr (FULL) {
        if (a.d_init)  // empty sequences hand the final state's gradient through
            each_empty(a.cu_seqlens, a.num_seqs, r, sh.ranges, lane, 32, [&](int q) {
                const int64_t at = ((int64_t)q * sh.width + pair) * N + 4 * j;
                if (live) copy_words<N / 8, kL>(a.d_init + at, a.d_final ? a.d_final + at : nullptr);
            });
    } else {
        if (t0 >= t1 || rg.origin(t0) == t0) return;  // the range begins a sequence
        t1 = min(t1, clamp_token(__ldg(a.cu_seqlens + sequence_of(rg.cu, rg.S, t0) + 1), rg.end));
    }

    // Of the slice at hand, pairs over the channels; A log2 e.  Every other two pairs of channels have the second two of
    // their states first, for the sums over channels.
    F2 e[NT], A[NT], dA[NT], h[NT];
    const int swap = NT == 4 ? lane >> 1 & 1 : 0;
    auto load_A = [&](int s) {
        no_states(A);
        if (live) read_states(a.A + states + s * kL * NT, N, swap, A);
#pragma unroll
        for (int k = 0; k < NT; ++k) A[k] = mul2(A[k], both(kLog2e));
    };
    // this thread's states in an array of [.., width, N] at row i
    auto get = [&](const float *p, int64_t i, int s, F2 (&to)[NT]) {
        no_states(to);
        if (p && live) read_states(p + i * sh.width * N + states + s * kL * NT, N, swap, to);
    };
    auto put = [&](float *p, int64_t i, int s, const F2 (&from)[NT]) {
        if (live) write_states(p + i * sh.width * N + states + s * kL * NT, N, swap, from);
    };
    // a slice's e between tiles and its dA: registers with one slice, else shared memory
    float *kept = reinterpret_cast<float *>(smem + Lay::kKept) + lane * 4;
    auto keep = [&](int s) {
        if constexpr (SL > 1) write_states(kept + s * 512, 128, 0, e);
    };
    auto recall = [&](int s) {
        if constexpr (SL > 1) {
            read_states(kept + s * 512, 128, 0, e);
            load_A(s);
        }
    };
    auto add_dA = [&](int s, const F2 (&half)[NT]) {
        if constexpr (SL > 1) read_states(kept + s * 512 + 256, 128, 0, dA);
#pragma unroll
        for (int k = 0; k < NT; ++k) dA[k] = add2(dA[k], half[k]);
        if constexpr (SL > 1) write_states(kept + s * 512 + 256, 128, 0, dA);
    };
    auto no_dA = [&](int s) {
        no_states(dA);
        if constexpr (SL > 1) write_states(kept + s * 512 + 256, 128, 0, dA);
    };
    auto decays = [&](F2 d, F2 (&to)[NT]) {
#pragma unroll
        for (int k = 0; k < NT; ++k) to[k] = decay2(d, A[k]);
    };

    // what the range takes over from those behind it
    int r_last = r;
    if (FULL && t0 < t1 && t1 < rg.end && rg.origin(t1) < t1) {
        const int stop = clamp_token(__ldg(a.cu_seqlens + sequence_of(rg.cu, rg.S, t1) + 1), rg.end);
        r_last = r + 1;
        for (int i = r + 2; i < rg.n; i += 32) {  // ranges that begin in front of the sequence's end
            const uint32_t m = __ballot_sync(0xffffffffu, i + lane < rg.n && rg.start(i + lane) < stop);
            r_last += __popc(m);
            if (m != 0xffffffffu) break;
        }
    }
    for (int s = 0; s < SL; ++s) {
        load_A(s);
        get(r_last > r ? wk.q : nullptr, r_last, s, e);
        for (int i = r_last - 1; i > r; --i) {
            F2 q[NT], dec[NT];
            float2 d = make_float2(0.f, 0.f);
            if (live) d = *reinterpret_cast<const float2 *>(wk.steps + (int64_t)i * sh.width + pair);
            get(wk.q, i, s, q);
            decays(f2(d.x, d.y), dec);
#pragma unroll
            for (int k = 0; k < NT; ++k) e[k] = fma2(dec[k], e[k], q[k]);
        }
        no_dA(s);
        keep(s);
    }

    const int esz = (int)sizeof(T), live_bytes = left * esz;
    const uint32_t smem_at = (uint32_t)__cvta_generic_to_shared(smem), cta_at = (uint32_t)__cvta_generic_to_shared(all_smem);
    constexpr int kR = kTile * Lay::kRow, kWords = kTile * Lay::kBRow / 16;  // 16-byte words of B or C in a tile
    auto fetch = [&](int row0, int stage) {
        if (row0 + kTile > t0 && row0 < t1 && row0 >= 0) {
            const uint32_t at = smem_at + stage * Lay::kStage;
            const int64_t c = (int64_t)c0 * esz, packed = (int64_t)sh.width * esz;
            copy_rows<Lay::kRow>(at, static_cast<const char *>(a.delta) + c, a.delta_stride * esz, live_bytes, row0, t0, t1,
                                 a.x, lane);
            copy_rows<Lay::kRow>(at + kR, static_cast<const char *>(a.d_out) + c, packed, live_bytes, row0, t0, t1, a.x, lane);
            if (a.gate)
                copy_rows<Lay::kRow>(at + 2 * kR, static_cast<const char *>(a.gate) + c, a.gate_stride * esz, live_bytes, row0,
                                     t0, t1, a.x, lane);
            if constexpr (FULL) {
                copy_rows<Lay::kRow>(at + 3 * kR, static_cast<const char *>(a.x) + c, a.x_stride * esz, live_bytes, row0, t0,
                                     t1, a.x, lane);
                const char *from = reinterpret_cast<const char *>(a.checkpoints + ((int64_t)(row0 / kTile) * sh.width + c0) * N);
#pragma unroll
                for (int k = lane; k < kCols * N / 4; k += 32) {
                    const bool ok = row0 >= t0 && k * 4 < left * N;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + Lay::kCheck + k * 16),
                                 "l"(ok ? static_cast<const void *>(from + k * 16) : a.x), "r"(ok ? 16 : 0) : "memory");
                }
            }
            for (int k = tid; k < Lay::kMats * kWords; k += 32 * kWarps) {  // each word by the thread that converts it
                const int m = k / kWords, i = (k % kWords) / (Lay::kBRow / 16), w = k % (Lay::kBRow / 16), t = row0 + i;
                const bool ok = t >= t0 && t < t1;
                const char *from = static_cast<const char *>(m ? a.B : a.C) +
                                   ((int64_t)t * (m ? a.b_stride : a.c_stride) + (int64_t)g * N) * esz + w * 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(cta_at + Lay::kRaw + stage * Lay::kMat + k * 16),
                             "l"(ok ? static_cast<const void *>(from) : a.x), "r"(ok ? 16 : 0) : "memory");
            }
        }
        copies_commit();
    };

    const int qd = lane % kQuads, tq = lane / kQuads;
    const bool quad_live = qd * 4 < left;
    F2 bias[2], skip[2], d_skip[2] = {both(0.f), both(0.f)}, d_bias[2] = {both(0.f), both(0.f)};
    load_quad(a.delta_bias, c0 + qd * 4, quad_live, bias);
    load_quad(FULL ? a.skip : nullptr, c0 + qd * 4, quad_live, skip);
    F2 steps = both(0.f);
    float4 *step = reinterpret_cast<float4 *>(smem + Lay::kStep);
    float *dys = reinterpret_cast<float *>(smem + Lay::kDy);
    float *cs = reinterpret_cast<float *>(all_smem + Lay::kC), *bs = cs + kTile * N * 2;
    float *slopes = reinterpret_cast<float *>(smem + Lay::kSlope);
    float *parts = reinterpret_cast<float *>(smem + Lay::kPart);
    float *sums = reinterpret_cast<float *>(all_smem + Lay::kSums);
    Edges ed;
    int stage = 0, turn = 0;
    const int row_last = (t1 - 1) & ~(kTile - 1);
    // The weights' sums go to the range's row every kPart tokens, which it then has the sum of: one chain of additions over
    // a long range would lose as many bits as its length has (131072 equal tokens in one range: d_A 2.3e-4 off, with the
    // parts 3e-6; it costs the other registers 1 % with 16 states).  `from`: the first token that is in them.  Every value
    // of the row is one thread's.
    auto leave_weights = [&](int from) {
        const bool more = (row_last & ~(kPart - 1)) > from;  // what was left behind `from`
        float *w = wk.weights + (int64_t)r * sh.width * (N + 2);
        for (int s = 0; s < SL; ++s) {
            float *to = w + (int64_t)pair * (N + 2) + s * kL * NT + j * NT;
            F2 was[NT];
            no_states(was);
            if (more && live) read_states(to, N + 2, swap, was);
            add_dA(s, was);
            if (live) write_states(to, N + 2, swap, dA);
            no_dA(s);
        }
        // the vectors' sums over the tokens of the eight lanes of a quad
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float2 u = f2_get(d_skip[p]), v = f2_get(d_bias[p]);
#pragma unroll
            for (int o = kQuads; o < 32; o <<= 1) {
                u.x += __shfl_xor_sync(0xffffffffu, u.x, o), u.y += __shfl_xor_sync(0xffffffffu, u.y, o);
                v.x += __shfl_xor_sync(0xffffffffu, v.x, o), v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
            }
            if (tq == 0 && quad_live) {
                float *to = w + (int64_t)(c0 + qd * 4 + 2 * p) * (N + 2) + N;
                if (more) u.x += to[0], v.x += to[1], u.y += to[N + 2], v.y += to[N + 3];
                to[0] = u.x, to[1] = v.x, to[N + 2] = u.y, to[N + 3] = v.y;
            }
            d_skip[p] = d_bias[p] = both(0.f);
        }
    };
    if (t0 < t1) fetch(row_last, 0);
    for (int row0 = row_last; t0 < t1 && row0 + kTile > t0; row0 -= kTile, stage ^= 1) {
        if constexpr (FULL)
            if ((row0 + kTile) % kPart == 0 && row0 < row_last) leave_weights(row0 + kTile);
        fetch(row0 - kTile, stage ^ 1);
        ed.find(rg, row0, t0, t1, lane);
        copies_wait<1>();
        const char *at = smem + stage * Lay::kStage;
        auto raw = [&](int tensor, int i, F2 (&to)[2]) {
            Quad<T>::unpack(*reinterpret_cast<const Raw *>(at + (tensor * kTile + i) * Lay::kRow + qd * 4 * esz), to);
        };
#pragma unroll
        for (int k = 0; k < kTile; k += 32 / kQuads) {
            const int i = k + tq, t = row0 + i;
            F2 x[2] = {both(0.f), both(0.f)}, d[2], dy[2], slope[2];
            raw(0, i, d);
            raw(1, i, dy);
            if constexpr (FULL) raw(3, i, x);
            if (a.gate) {
                F2 z[2];
                raw(2, i, z);
#pragma unroll
                for (int p = 0; p < 2; ++p) {  // silu' = s (1 + z (1 - s))
                    const F2 s = sigmoid2<T>(z[p]);
                    if constexpr (FULL)
                        slope[p] = mul2(dy[p], mul2(s, fma2(z[p], fma2(s, both(-1.f), both(1.f)), both(1.f))));
                    dy[p] = mul2(dy[p], mul2(z[p], s));
                }
                if constexpr (FULL) write_quad(slopes + (kTile + i) * kCols + qd * 4, slope);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                d[p] = softplus2<FULL>(add2(d[p], bias[p]), slope[p]);
                if (t < t0 || t >= t1) d[p] = both(0.f);  // neither decay nor input; dy is 0 there
                x[p] = mul2(x[p], d[p]);
            }
            if constexpr (FULL) write_quad(slopes + i * kCols + qd * 4, slope);
#pragma unroll
            for (int p = 0; p < 2; ++p) {  // banks: every other four lanes the other pair first
                const bool other = (p ^ (lane >> 2)) & 1;
                const float2 u = f2_get(other ? d[1] : d[0]), v = f2_get(other ? x[1] : x[0]);
                step[i * (kCols / 2) + qd * 2 + other] = make_float4(u.x, u.y, v.x, v.y);
            }
            write_quad(dys + i * kCols + qd * 4, dy);
        }
        for (int k = tid; k < Lay::kMats * kWords; k += 32 * kWarps) {
            const char *from = all_smem + Lay::kRaw + stage * Lay::kMat + k * 16;
            float4 *to = reinterpret_cast<float4 *>(cs + k * (16 / esz) * 2);
#pragma unroll
            for (int q = 0; q < 4 / esz; ++q) leave_twice<T>(to + 2 * q, reinterpret_cast<const Raw *>(from)[q]);
        }
        __syncthreads();  // B and C; they are written again behind the last barrier of this tile
        auto row_of = [&](const float *m, int i, int s, F2 (&to)[NT]) {  // this thread's states of B or C
            read_twice(m + (i * N + s * kL * NT + j * NT) * 2, swap, to);
        };
        if constexpr (!FULL) {
            for (int s = 0; s < SL; ++s) {
                recall(s);
                auto token = [&](int i) {
                    const float4 d = step[i * (kCols / 2) + cl];
                    const float2 dy = *reinterpret_cast<const float2 *>(dys + i * kCols + 2 * cl);
                    F2 C[NT], dec[NT];
                    row_of(cs, i, s, C);
                    decays(f2(d.x, d.y), dec);
#pragma unroll
                    for (int k = 0; k < NT; ++k) e[k] = mul2(dec[k], fma2(C[k], f2(dy.x, dy.y), e[k]));
                    if (s == 0) steps = add2(steps, f2(d.x, d.y));
                };
                if (ed.ends == 0) {
#pragma unroll 4
                    for (int i = kTile - 1; i >= 0; --i) token(i);
                } else {
                    for (int i = kTile - 1; i >= 0; --i) {
                        if ((ed.ends >> i) & 1u) get(a.d_final, __shfl_sync(0xffffffffu, ed.seq, i), s, e);
                        token(i);
                    }
                }
                keep(s);
            }
            __syncthreads();
        } else {
            // sums over states of the half's tokens, and what follows from them
            auto epilogue = [&](int from) {
                __syncwarp();
                const int i = from + tq, t = row0 + i;
                F2 sum[3][2];
#pragma unroll
                for (int m = 0; m < 3; ++m) {
                    sum[m][0] = sum[m][1] = both(0.f);
#pragma unroll
                    for (int l = 0; l < kL; ++l) {  // banks: see where they are left
                        const float4 u = *reinterpret_cast<const float4 *>(parts + ((m * kSpan + tq) * kL + (l ^ (tq & 1))) * kCols +
                                                                         qd * 4);
                        sum[m][0] = add2(sum[m][0], f2(u.x, u.y));
                        sum[m][1] = add2(sum[m][1], f2(u.z, u.w));
                    }
                }
                F2 x[2], dx[2], dd[2], dz[2], dy[2], slope[2], gate[2];
                raw(3, i, x);
                read_quad(dys + i * kCols + qd * 4, dy);
                read_quad(slopes + i * kCols + qd * 4, slope);
                read_quad(slopes + (kTile + i) * kCols + qd * 4, gate);
                const float2 d[2] = {*reinterpret_cast<const float2 *>(step + i * (kCols / 2) + qd * 2),
                                     *reinterpret_cast<const float2 *>(step + i * (kCols / 2) + qd * 2 + 1)};
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    dx[p] = fma2(skip[p], dy[p], mul2(f2(d[p].x, d[p].y), sum[1][p]));
                    dd[p] = mul2(fma2(x[p], sum[1][p], mul2(sum[2][p], both(0.693147181f))), slope[p]);  // the sum has A log2 e
                    dz[p] = mul2(gate[p], fma2(skip[p], x[p], sum[0][p]));
                }
                const bool in = t >= t0 && t < t1 && quad_live;
                const int64_t to = (int64_t)t * sh.width + c0 + qd * 4;
                if (a.gate && in) *reinterpret_cast<Raw *>(static_cast<T *>(a.d_gate) + to) = Quad<T>::pack(dz);
                if (in) {
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        d_skip[p] = fma2(dy[p], x[p], d_skip[p]);
                        d_bias[p] = add2(d_bias[p], dd[p]);
                    }
                    *reinterpret_cast<Raw *>(static_cast<T *>(a.dx) + to) = Quad<T>::pack(dx);
                    *reinterpret_cast<Raw *>(static_cast<T *>(a.d_delta) + to) = Quad<T>::pack(dd);
                }
                __syncwarp();
            };
            // The four warps' sums over channels of a half: each warp adds up a quarter of its tokens.
            auto reduce = [&](int from, int s) {
                __syncthreads();
                constexpr int kValues = 2 * kL * NT;
                const float *src = sums + turn * kWarps * kSpan * 32;
#pragma unroll
                for (int k = 0; k < kSpan / kWarps; ++k) {
                    const int i = warp * (kSpan / kWarps) + k, t = row0 + from + i;
                    float v = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) v += src[(w * kSpan + i) * 32 + lane];
                    // lane: dB (the first half of the values), then dC
                    if (lane < kValues && t >= t0 && t < t1)
                        wk.tokens[(((int64_t)part * a.total_tokens + t) * sh.groups + g) * 2 * N + lane / (kValues / 2) * N +
                                  s * kL * NT + lane % (kValues / 2)] = v;
                }
                turn ^= 1;
            };
            auto half = [&](auto edges, int from, int s) {
                constexpr bool EDGES = decltype(edges)::value;
                recall(s);
                read_states(reinterpret_cast<const float *>(at + Lay::kCheck) + 2 * cl * N + s * kL * NT + j * NT, N, swap, h);
                auto forward = [&](int i, F2 (&dec)[NT]) {
                    const float4 d = step[i * (kCols / 2) + cl];
                    F2 B[NT];
                    row_of(bs, i, s, B);
                    decays(f2(d.x, d.y), dec);
#pragma unroll
                    for (int k = 0; k < NT; ++k) h[k] = fma2(dec[k], h[k], mul2(f2(d.z, d.w), B[k]));
                };
                if (from) {  // to the middle of the tile
#pragma unroll 4
                    for (int i = 0; i < kSpan; ++i) {
                        F2 dec[NT];
                        if (EDGES && ((ed.starts >> i) & 1u)) get(a.init, __shfl_sync(0xffffffffu, ed.seq, i), s, h);
                        forward(i, dec);
                    }
                }
                F2 before[kSpan][NT], dec[kSpan][NT];
#pragma unroll
                for (int b = 0; b < kSpan; ++b) {
                    const int i = from + b;
                    if (EDGES && ((ed.starts >> i) & 1u)) get(a.init, __shfl_sync(0xffffffffu, ed.seq, i), s, h);
#pragma unroll
                    for (int k = 0; k < NT; ++k) before[b][k] = h[k];
                    forward(i, dec[b]);
                }
                // what a token takes from shared memory, loaded before the token behind it leaves its sums
                struct Operands {
                    float4 d;
                    float2 dy;
                    F2 B[NT], C[NT];
                };
                auto operands = [&](int i) {
                    Operands o;
                    o.d = step[i * (kCols / 2) + cl];
                    o.dy = *reinterpret_cast<const float2 *>(dys + i * kCols + 2 * cl);
                    row_of(bs, i, s, o.B);
                    row_of(cs, i, s, o.C);
                    return o;
                };
                Operands next = operands(from + kSpan - 1);
                F2 dA_half[NT];  // a sum of its own
                no_states(dA_half);
#pragma unroll
                for (int b = kSpan - 1; b >= 0; --b) {
                    const int i = from + b;
                    const Operands o = next;
                    if (b) next = operands(i - 1);
                    // A row of no token adds nothing to dA (its decay is 1 and its step 0, but an infinite or NaN state or
                    // gradient beside it is not) and passes e on; what it would leave for the other sums nobody reads.
                    if (EDGES && (row0 + i < t0 || row0 + i >= t1)) continue;
                    if (EDGES && ((ed.ends >> i) & 1u)) get(a.d_final, __shfl_sync(0xffffffffu, ed.seq, i), s, e);
                    const F2 d = f2(o.d.x, o.d.y), x = f2(o.d.z, o.d.w), dy = f2(o.dy.x, o.dy.y);
                    F2 sum[3] = {both(0.f), both(0.f), both(0.f)};
                    float vB[NT], vC[NT];
#pragma unroll
                    for (int k = 0; k < NT; ++k) {
                        const F2 u = mul2(dec[b][k], before[b][k]);
                        const F2 now = b + 1 == kSpan ? h[k] : EDGES ? fma2(x, o.B[k], u) : before[(b + 1) % kSpan][k];
                        const F2 gr = fma2(o.C[k], dy, e[k]);
                        e[k] = mul2(dec[b][k], gr);
                        const F2 w = mul2(gr, u);
                        sum[0] = fma2(o.C[k], now, sum[0]);
                        sum[1] = fma2(o.B[k], gr, sum[1]);
                        sum[2] = fma2(A[k], w, sum[2]);
                        dA_half[k] = fma2(d, w, dA_half[k]);
                        const float2 fB = f2_get(mul2(gr, x)), fC = f2_get(mul2(dy, now));
                        vB[k] = fB.x + fB.y;
                        vC[k] = fC.x + fC.y;
                    }
#pragma unroll
                    for (int m = 0; m < 3; ++m) {
                        // banks: an epilogue's eight lanes read two tokens, so odd tokens have neighbouring lanes' parts swapped
                        float2 *to = reinterpret_cast<float2 *>(parts + ((m * kSpan + b) * kL + (j ^ (b & 1))) * kCols + 2 * cl);
                        float2 v = f2_get(sum[m]);
                        if (SL > 1 && s) v.x += to->x, v.y += to->y;
                        *to = v;
                    }
                    // Over the eight pairs of channels: by bit 1 of the lane the first or second two states, which `swap` has
                    // put first; by bit 2 dB or dC; by bit 0 one of the two states.
                    if constexpr (NT == 4) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            vB[k] += __shfl_xor_sync(0xffffffffu, vB[k + 2], 2);
                            vC[k] += __shfl_xor_sync(0xffffffffu, vC[k + 2], 2);
                        }
                    }
                    const bool k2 = lane & 4, k0 = lane & 1;
                    const float v0 = (k2 ? vC[0] : vB[0]) + __shfl_xor_sync(0xffffffffu, k2 ? vB[0] : vC[0], 4);
                    const float v1 = (k2 ? vC[1] : vB[1]) + __shfl_xor_sync(0xffffffffu, k2 ? vB[1] : vC[1], 4);
                    float one = (k0 ? v1 : v0) + __shfl_xor_sync(0xffffffffu, k0 ? v0 : v1, 1);
                    if constexpr (NT == 2) one += __shfl_xor_sync(0xffffffffu, one, 2);
                    const int at_value = (lane >> 2 & 1) * kL * NT + j * NT + (swap << 1) + (lane & 1);
                    sums[((turn * kWarps + warp) * kSpan + b) * 32 + at_value] = one;
                    if (EDGES && ((ed.starts >> i) & 1u)) {
                        const int q = __shfl_sync(0xffffffffu, ed.seq, i);
                        if (a.d_init) put(a.d_init, q, s, e);
                    }
                }
                add_dA(s, dA_half);
                keep(s);
            };
#pragma unroll 1
            for (int from = kTile - kSpan; from >= 0; from -= kSpan) {
                for (int s = 0; s < SL; ++s) {
                    if ((ed.starts | ed.ends) == 0)
                        half(std::false_type{}, from, s);
                    else
                        half(std::true_type{}, from, s);
                    if (SL > 1 && s + 1 < SL) reduce(from, s);
                }
                epilogue(from);
                reduce(from, SL - 1);
            }
        }
    }
    if constexpr (FULL) {
        griddep_launch_dependents();
        leave_weights(t0);
    } else {
        for (int s = 0; s < SL; ++s) {
            recall(s);
            put(wk.q, r, s, e);
        }
        if (j == 0 && live) *reinterpret_cast<float2 *>(wk.steps + (int64_t)r * sh.width + pair) = f2_get(steps);
    }
}

// dB and dC from the CTAs' rows, four values per thread, in the first `tokens` CTAs; in those behind them the weights'
// gradients from the ranges' sums.  Launched as a dependent of the gradients' kernel.
template <typename T>
__global__ void __launch_bounds__(256) selective_sums_kernel(SelectiveArgs a, SelectiveShape sh, BackwardWork wk, int N, unsigned tokens) {
    griddep_wait();
    if (blockIdx.x >= tokens) {
        const int i = (blockIdx.x - tokens) * 256 + threadIdx.x, c = i / (N + 2), n = i % (N + 2);
        if (c >= sh.width) return;
        float s = 0.f;
#pragma unroll 8
        for (int r = 0; r < sh.ranges; ++r) s += wk.weights[(int64_t)r * sh.width * (N + 2) + i];
        if (n < N)
            a.d_A[(int64_t)c * N + n] = s;
        else if (n == N && a.d_skip)
            a.d_skip[c] = s;
        else if (n == N + 1 && a.d_delta_bias)
            a.d_delta_bias[c] = s;
        return;
    }
    const int groups = sh.groups, row = groups * N / 2;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, t = i / row;
    if (t >= clamp_token(__ldg(a.cu_seqlens + a.num_seqs), a.total_tokens)) return;
    const int at = (int)(i - t * row) * 4, g = at / (2 * N), n = at % (2 * N);
    const int64_t part = (int64_t)a.total_tokens * groups * 2 * N;
    const float *from = wk.tokens + (t * groups + g) * 2 * N + n;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 16
    for (int p = 0; p < wk.parts; ++p) {
        const float4 v = *reinterpret_cast<const float4 *>(from + p * part);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const F2 f[2] = {f2(s.x, s.y), f2(s.z, s.w)};
    *reinterpret_cast<typename Quad<T>::Raw *>(static_cast<T *>(n < N ? a.d_B : a.d_C) + (t * groups + g) * N + n % N) = Quad<T>::pack(f);
}

// CTAs that the GPU holds: two on an SM, one with 64 states, whose stages fill shared memory.
SelectiveShape backward_shape(const sse_selective_config_t &c, int64_t T, int32_t S) {
    SelectiveShape s = selective_shape(c, kCols);
    const int parts = (s.tiles + 3) / 4;
    const Waves choices[] = {{4, 400}, {2, 128}, {1, 4 * kTile}};
    set_ranges(s, ranges_that_fill((int64_t)parts * c.groups, c.state == 64 ? 152 : 304, choices, T), kAlone, S);
    return s;
}

// The workspace: what ranges hand on, the tokens' rows, the ranges' weights.
size_t carve(const sse_selective_config_t &c, const SelectiveShape &s, int64_t T, char *base, BackwardWork &wk) {
    const size_t N = c.state;
    size_t at = 0;
    auto take = [&](size_t floats) {
        float *p = reinterpret_cast<float *>(base + at);
        at += (floats * sizeof(float) + 255) & ~size_t(255);
        return p;
    };
    wk.parts = (s.tiles + 3) / 4;  // four warps a CTA
    wk.weights = take((size_t)s.ranges * c.width * (N + 2));
    wk.tokens = take((size_t)wk.parts * T * c.groups * 2 * N);
    wk.q = wk.steps = nullptr;
    if (s.ranges > 1) {
        wk.q = take((size_t)s.ranges * c.width * N);
        wk.steps = take((size_t)s.ranges * c.width);
    }
    return at;
}

template <typename T, int N> cudaError_t launch_t(const sse_selective_config_t &c, const SelectiveArgs &a, cudaStream_t s) {
    const SelectiveShape sh = backward_shape(c, a.total_tokens, a.num_seqs);
    BackwardWork wk;
    carve(c, sh, a.total_tokens, a.workspace, wk);
    const auto states = selective_backward_kernel<T, N, false>, full = selective_backward_kernel<T, N, true>;
    constexpr int kStates = Layout<T, N, false>::kBytes, kFull = Layout<T, N, true>::kBytes;
    static_assert(Layout<T, N, true>::kWarps == 4 && kStates <= 48 * 1024 && kFull <= 227 * 1024, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(full, cudaFuncAttributeMaxDynamicSharedMemorySize, kFull);
    if (e != cudaSuccess) return e;
    // (The gradients as a dependent of the states would have their CTAs placed beside those: 500 x 1024 51 -> 55 us.)
    if (sh.ranges > 1) states<<<dim3(sh.tiles * c.groups, sh.ranges), 32, kStates, s>>>(a, sh, wk);
    full<<<dim3(wk.parts * c.groups, sh.ranges), 32 * Layout<T, N, true>::kWarps, kFull, s>>>(a, sh, wk);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const unsigned tokens = (unsigned)(((int64_t)a.total_tokens * c.groups * N / 2 + 255) / 256);
    return launch_dependent(selective_sums_kernel<T>, dim3(tokens + (c.width * (N + 2) + 255) / 256), dim3(256), 0, s, a, sh, wk, N,
                            tokens);
}

template <typename T> cudaError_t launch_state(const sse_selective_config_t &c, const SelectiveArgs &a, cudaStream_t s) {
    switch (c.state) {
    case 8: return launch_t<T, 8>(c, a, s);
    case 16: return launch_t<T, 16>(c, a, s);
    case 32: return launch_t<T, 32>(c, a, s);
    default: return launch_t<T, 64>(c, a, s);
    }
}

}  // namespace

size_t selective_backward_workspace(const sse_selective_config_t &c, int64_t T, int32_t S) {
    BackwardWork wk;
    return carve(c, backward_shape(c, T, S), T, nullptr, wk);
}
cudaError_t launch_selective_backward(const sse_selective_config_t &cfg, const SelectiveArgs &a, cudaStream_t stream) {
    return cfg.dtype == SSE_BF16 ? launch_state<__nv_bfloat16>(cfg, a, stream) : launch_state<float>(cfg, a, stream);
}

}  // namespace sse
