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
//
// Measured on a GB300, bf16 (floors at 6.77 TB/s): forward with residual 16384 x 2304
// 51 us (44.6), 16384 x 2048 46 (39.7), 32768 x 1024 47, 4096 x 8192 48, without
// residual 16384 x 2048 29 (19.8), 65536 x 512 25, in float32 16384 x 2048 52 (39.7); backward
// with the residual's gradient 16384 x 2048 57 (39.7), 32768 x 1024 56, 4096 x 8192 73, 2048 x
// 16384 130, 8192 x 2048 in float32 51, 4096 x 8192 174 (79).
// Rows loaded when their turn came took 66 us for the first and 95 for the backward.
// The backward's rows wait in shared memory, so that what a row keeps
// over its sums is there and not in registers, and the columns' weights are in registers:
// 16 warps on an SM instead of 12 and no loads of weights, 66 -> 57 us (the first alone 68).
#include "quad.cuh"

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
// between the rows, so that one barrier a row is enough.  Every warp but the last has `whole` elements.
template <int N, int VPT, int E, int MAXW>
__device__ __forceinline__ void join(const LnShape &n, float4 &v, int warp, int lane, int turn, float4 *words) {
    if (n.warps == 1) return;
    constexpr float whole = 32 * VPT * E;
    const float last = (float)warp_elements(n, n.warps - 1, VPT, E);
    if (lane == 0) words[turn * 32 + warp] = v;
    __syncthreads();
    float mean = 0.f;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int w, const float4 &u) {
        const float d = u.x - mean;
        t.y += fmaf((w + 1 == n.warps ? last : whole) * d, d, u.y);
        if constexpr (N == 4) {
            t.z += u.z;
            t.w += fmaf(d, u.z, u.w);
        }
    };
    if constexpr (N == 4 && MAXW <= 4) {
        float4 u[MAXW];
#pragma unroll
        for (int w = 0; w < MAXW; ++w) {
            if (w >= n.warps) break;
            u[w] = words[turn * 32 + w];
            mean = fmaf(w + 1 == n.warps ? last : whole, u[w].x, mean);
        }
        mean *= n.inv_width;
#pragma unroll
        for (int w = 0; w < MAXW; ++w) {
            if (w >= n.warps) break;
            add(w, u[w]);
        }
    } else {
#pragma unroll 4
        for (int w = 0; w < n.warps; ++w) mean = fmaf(w + 1 == n.warps ? last : whole, words[turn * 32 + w].x, mean);
        mean *= n.inv_width;
#pragma unroll 4
        for (int w = 0; w < n.warps; ++w) add(w, words[turn * 32 + w]);
    }
    t.x = mean;
    v = t;
}

// A thread's words of a row: warp w, word i, lane l has word (w * VPT + i) * 32 + l.
template <typename T, int VPT> struct Words {
    uint4 u[VPT];
    __device__ __forceinline__ void load(const LnShape &n, const void *p, int64_t stride, int64_t row, int first, bool ok) {
        const T *at = static_cast<const T *>(p) + row * stride + first * Word<T>::kE;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            u[i] = ok && first + i * 32 < n.nv ? *reinterpret_cast<const uint4 *>(at + i * 32 * Word<T>::kE) : make_uint4(0, 0, 0, 0);
    }
};
// The words of the next DEPTH rows of TENSORS tensors in shared memory, each copied by the thread that reads it: no barrier.
template <typename T, int VPT, int TENSORS, int DEPTH> struct Ahead {
    static constexpr int kBytes = DEPTH * TENSORS * VPT * 16;  // of a thread
    uint32_t at;
    __device__ __forceinline__ Ahead(const void *ring) : at((uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * 16) {}
    __device__ __forceinline__ uint32_t word(int slot, int tensor, int i) const {
        return at + ((slot * TENSORS + tensor) * VPT + i) * blockDim.x * 16;
    }
    // Nothing for a row that is not there (nobody reads it), zeros where the row has no word.
    __device__ __forceinline__ void copy(const LnShape &n, int slot, int tensor, const void *p, int64_t stride, int64_t row, int first,
                                         bool ok) const {
        if (!ok) return;
        const T *from = static_cast<const T *>(p) + row * stride + first * Word<T>::kE;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const bool live = first + i * 32 < n.nv;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(word(slot, tensor, i)),
                         "l"(live ? static_cast<const void *>(from + i * 32 * Word<T>::kE) : p), "r"(live ? 16 : 0) : "memory");
        }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // Until the oldest row is there.
    static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
    __device__ __forceinline__ uint4 read(int slot, int tensor, int i) const {
        uint4 u;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "r"(word(slot, tensor, i)) : "memory");
        return u;
    }
};
// Word j of a float32 vector.
template <typename T> __device__ __forceinline__ void vector_word(const float *p, int j, F2 (&f)[Word<T>::kP]) {
#pragma unroll
    for (int k = 0; k < Word<T>::kP; k += 2) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p + j * Word<T>::kE + 2 * k));
        f[k] = f2(v.x, v.y);
        f[k + 1] = f2(v.z, v.w);
    }
}

// Threads of a row up to which the backward has its column sums in registers: 128 a thread.
constexpr int kInRegisters = 512;

// Threads of an SM that the forward's registers allow: 64 a thread for one word, 96 (float32 80) for two, else 128.
constexpr int forward_threads(int vpt, int bytes) { return vpt == 1 ? 1024 : vpt > 2 ? 512 : bytes == 2 ? 640 : 768; }

constexpr int kPart = 256;  // rows of a team in one sum

// Four column sums of a thread's own, added to what is there with `more`.
__device__ __forceinline__ void leave_quad(float *to, const F2 (&sum)[2], bool more) {
    F2 was[2] = {both(0.f), both(0.f)};
    if (more) read_quad(to, was);
    const F2 now[2] = {add2(sum[0], was[0]), add2(sum[1], was[1])};
    write_quad(to, now);
}

// Rows that the backward has on their way: two, or one where shared memory has the column sums.
constexpr int rows_ahead(int threads) { return threads > kInRegisters ? 1 : 2; }

// Rows of up to two words a thread have the columns' weights and bias in registers and two rows under way in shared memory
// (without residual: 65536 x 512 33 -> 25 us, 16384 x 2048 34.5 -> 29); wider ones load the vectors from L1 row by row and
// the next row to registers (4096 x 8192 48 us; through shared memory 53).
template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT, forward_threads(VPT, sizeof(T)) / MAXT) layer_norm_kernel(LayerNormArgs a, LnShape n) {
    constexpr int E = Word<T>::kE, P = Word<T>::kP;
    constexpr bool HELD = VPT <= 2;
    __shared__ float4 words[64];
    extern __shared__ __align__(16) float ring[];
    using Rows = Ahead<T, VPT, 2, 2>;
    const Rows ahead(ring);
    Words<T, VPT> x, r;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int warp = n.warps == 1 ? 0 : wid, j0 = warp * VPT * 32 + lane;
    const int64_t rows_on = n.warps == 1 ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const int64_t first = n.warps == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + wid : blockIdx.x;
    const float inv_mine = 1.f / (float)warp_elements(n, warp, VPT, E);
    auto fetch = [&](int slot, int64_t row) {
        const bool ok = row < a.T;
        if constexpr (HELD) {
            ahead.copy(n, slot, 0, a.x, a.x_stride, row, j0, ok);
            if (a.r) ahead.copy(n, slot, 1, a.r, a.r_stride, row, j0, ok);
            Rows::commit();
        } else {
            x.load(n, a.x, a.x_stride, row, j0, ok);
            if (a.r) r.load(n, a.r, a.r_stride, row, j0, ok);
        }
    };
    fetch(0, first);
    if constexpr (HELD) fetch(1, first + rows_on);
    F2 w[HELD ? VPT : 1][P], b[HELD ? VPT : 1][P];
    auto vectors = [&](int i, int j) {
        if (a.weight) vector_word<T>(a.weight, j, w[i]);
        if (a.bias) vector_word<T>(a.bias, j, b[i]);
    };
#pragma unroll
    for (int i = 0; i < (HELD ? VPT : 1); ++i) {
#pragma unroll
        for (int k = 0; k < P; ++k) w[i][k] = both(1.f), b[i][k] = both(0.f);
        if (HELD && j0 + i * 32 < n.nv) vectors(i, j0 + i * 32);
    }
    int turn = 0;
    for (int64_t row = first; row < a.T; row += rows_on) {
        F2 v[VPT][P];
        if constexpr (HELD) {
            Rows::wait();
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                x.u[i] = ahead.read(turn, 0, i);
                if (a.r) r.u[i] = ahead.read(turn, 1, i);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            Word<T>::unpack(x.u[i], v[i]);
            if (a.r) {
                F2 f[P];
                Word<T>::unpack(r.u[i], f);
#pragma unroll
                for (int k = 0; k < P; ++k) v[i][k] = add2(v[i][k], f[k]);
            }
        }
        fetch(turn, row + (HELD ? 2 : 1) * rows_on);
        F2 t = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int k = 0; k < P; ++k) t = add2(t, v[i][k]);
        float4 m = make_float4(warp_sum(fold(t)) * inv_mine, 0.f, 0.f, 0.f);
        t = both(0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (j0 + i * 32 < n.nv)
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const F2 d = add2(v[i][k], both(-m.x));
                    t = fma2(d, d, t);
                }
        m.y = warp_sum(fold(t));
        join<2, VPT, E, MAXT / 32>(n, m, warp, lane, turn, words);
        turn ^= 1;
        const float rstd = rsqrt_ftz(fmaf(m.y, n.inv_width, n.eps));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = j0 + i * 32, h = HELD ? i : 0;
            if (j >= n.nv) continue;
            const int64_t at = row * n.width + j * E;
            if (a.r_out) *reinterpret_cast<uint4 *>(static_cast<T *>(a.r_out) + at) = Word<T>::pack(v[i]);
            if (!HELD) vectors(0, j);
#pragma unroll
            for (int k = 0; k < P; ++k) v[i][k] = fma2(mul2(add2(v[i][k], both(-m.x)), both(rstd)), w[h][k], b[h][k]);
            *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + at) = Word<T>::pack(v[i]);
        }
    }
}

template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 128 ? 1 : VPT == 1 || sizeof(T) == 4 ? 5 : 4)
layer_norm_backward_kernel(LayerNormArgs a, LnShape n) {
    constexpr int E = Word<T>::kE, P = Word<T>::kP;
    __shared__ float4 words[64];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int warp = n.warps == 1 ? 0 : wid, j0 = warp * VPT * 32 + lane;
    const int64_t rows_on = n.warps == 1 ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const int64_t first = n.warps == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 5) + wid : blockIdx.x;
    const float inv_mine = 1.f / (float)warp_elements(n, warp, VPT, E);
    // column sums: in registers, or where there are too few, in words of shared memory of the thread's own
    constexpr bool SHARED = MAXT > kInRegisters;
    extern __shared__ __align__(16) float sums[];
    using Rows = Ahead<T, VPT, 3, rows_ahead(MAXT)>;
    const Rows ahead(sums + (SHARED ? VPT * P * 4 * blockDim.x : 0));
    F2 sum_w[SHARED ? 1 : VPT][P], sum_b[SHARED ? 1 : VPT][P];
    auto mine = [&](int which, int i, int k) { return sums + (((which * VPT + i) * (P / 2) + k / 2) * blockDim.x + threadIdx.x) * 4; };
    auto no_sums = [&] {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int k = 0; k < P; k += 2) {
                const F2 none[2] = {both(0.f), both(0.f)};
                if constexpr (SHARED) {
                    write_quad(mine(0, i, k), none);
                    write_quad(mine(1, i, k), none);
                } else {
                    sum_w[i][k] = sum_w[i][k + 1] = sum_b[i][k] = sum_b[i][k + 1] = both(0.f);
                }
            }
    };
    no_sums();
    int turn = 0;
    auto copy = [&](int slot, int64_t row) {
        ahead.copy(n, slot, 0, a.x, a.x_stride, row, j0, row < a.T);
        ahead.copy(n, slot, 1, a.d_out, n.width, row, j0, row < a.T);
        if (a.d_r_out) ahead.copy(n, slot, 2, a.d_r_out, n.width, row, j0, row < a.T);
        Rows::commit();
    };
    constexpr int kDepth = rows_ahead(MAXT);
    // the columns' weights, from L1 row by row where the column sums are not in registers either
    F2 w[SHARED ? 1 : VPT][P];
    auto weights = [&](int i, int j) {
        if (SHARED && a.weight) vector_word<T>(a.weight, j, w[0]);
    };
#pragma unroll
    for (int i = 0; i < (SHARED ? 1 : VPT); ++i) {
#pragma unroll
        for (int k = 0; k < P; ++k) w[i][k] = both(1.f);
        if (!SHARED && a.weight && j0 + i * 32 < n.nv) vector_word<T>(a.weight, j0 + i * 32, w[i]);
    }
#pragma unroll
    for (int k = 0; k < kDepth; ++k) copy(k, first + k * rows_on);
    int slot = 0;
    int64_t row = first;
    // This team's column sums go to its partial row of each every kPart rows, which it then has the sum of: one chain of
    // additions over a long batch would lose as many bits as its length has (2^19 equal rows of 8192 columns: d_weight
    // 5.8e-5 off, with the parts 2.5e-5, which its terms are).
    bool more = false;  // the partial rows have something already
    do {
        const int64_t stop = min(a.T, row + kPart * rows_on);
        for (; row < stop; row += rows_on) {
            F2 v[VPT][P];
            Rows::wait();
#pragma unroll
            for (int i = 0; i < VPT; ++i) Word<T>::unpack(ahead.read(slot, 0, i), v[i]);
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
                const int j = j0 + i * 32;
                if (j >= n.nv) continue;
                F2 d[P];
                weights(i, j);
                Word<T>::unpack(ahead.read(slot, 1, i), d);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const F2 c = add2(v[i][k], both(-m.x));
                    const F2 p = mul2(d[k], w[SHARED ? 0 : i][k]);
                    sq = fma2(c, c, sq);
                    sp = add2(sp, p);
                    sx = fma2(p, c, sx);
                }
            }
            m.y = warp_sum(fold(sq));
            m.z = warp_sum(fold(sp));
            m.w = warp_sum(fold(sx));
            join<4, VPT, E, MAXT / 32>(n, m, warp, lane, turn, words);
            turn ^= 1;
            const float rstd = rsqrt_ftz(fmaf(m.y, n.inv_width, n.eps));
            const float mean_p = m.z * n.inv_width, slope = m.w * n.inv_width * rstd * rstd;  // mean(p x_hat) rstd
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int j = j0 + i * 32;
                if (j >= n.nv) continue;
                F2 v[P], d[P], e[P];
                weights(i, j);
                Word<T>::unpack(ahead.read(slot, 0, i), v);
                Word<T>::unpack(ahead.read(slot, 1, i), d);
                if (a.d_r_out) Word<T>::unpack(ahead.read(slot, 2, i), e);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const F2 c = add2(v[k], both(-m.x));
                    v[k] = mul2(c, both(rstd));  // x_hat
                    if constexpr (!SHARED) {
                        sum_w[i][k] = fma2(d[k], v[k], sum_w[i][k]);
                        sum_b[i][k] = add2(sum_b[i][k], d[k]);
                    }
                    F2 p = mul2(d[k], w[SHARED ? 0 : i][k]);
                    p = mul2(fma2(c, both(-slope), add2(p, both(-mean_p))), both(rstd));
                    e[k] = a.d_r_out ? add2(p, e[k]) : p;
                }
                *reinterpret_cast<uint4 *>(static_cast<T *>(a.dx) + row * n.width + j * E) = Word<T>::pack(e);
                if constexpr (SHARED) {
#pragma unroll
                    for (int k = 0; k < P; k += 2) {
                        F2 w[2], b[2];
                        read_quad(mine(0, i, k), w);
                        read_quad(mine(1, i, k), b);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            w[q] = fma2(d[k + q], v[k + q], w[q]);
                            b[q] = add2(b[q], d[k + q]);
                        }
                        write_quad(mine(0, i, k), w);
                        write_quad(mine(1, i, k), b);
                    }
                }
            }
            copy(slot, row + kDepth * rows_on);
            slot = slot + 1 == kDepth ? 0 : slot + 1;
        }
        if (row >= a.T) griddep_launch_dependents();
        if (first < rows_on)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int j = j0 + i * 32;
                if (j >= n.nv) continue;
#pragma unroll
                for (int k = 0; k < P; k += 2) {
                    F2 w[2], b[2];
                    if constexpr (SHARED) {
                        read_quad(mine(0, i, k), w);
                        read_quad(mine(1, i, k), b);
                    } else {
                        w[0] = sum_w[i][k], w[1] = sum_w[i][k + 1], b[0] = sum_b[i][k], b[1] = sum_b[i][k + 1];
                    }
                    if (a.d_weight) leave_quad(a.partials + first * n.width + j * E + 2 * k, w, more);
                    if (a.d_bias) leave_quad(a.partials + (rows_on + first) * n.width + j * E + 2 * k, b, more);
                }
            }
        no_sums();
        more = true;
    } while (row < a.T);
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

// Up to `most` words per thread.  Rows of one warp share a CTA of four.  With a residual 384 threads of an SM (512 in
// larger CTAs) are enough for HBM, and more in the way of each other (16384 x 2048: 45 us with 384, 48 with 512, 50 with 640;
// 16384 x 2304 51 with 480, 56 with 640); without, 29 us with 640 and 35 with 384.
LnPlan plan(const sse_layer_norm_config_t &c, int64_t T, bool backward, bool residual) {
    LnPlan p{};
    p.n.width = c.width;
    p.n.nv = c.width / (c.dtype == SSE_BF16 ? 8 : 4);
    p.n.eps = c.eps;
    const int most = backward || p.n.nv <= 512 ? 2 : 4;
    p.n.inv_width = 1.f / c.width;
    p.n.warps = (p.n.nv + 32 * most - 1) / (32 * most);
    p.vpt = (p.n.nv + 32 * p.n.warps - 1) / (32 * p.n.warps);
    p.n.warps = (p.n.nv + 32 * p.vpt - 1) / (32 * p.vpt);
    p.teams = p.n.warps == 1 ? 4 : 1;
    p.threads = 32 * p.n.warps * p.teams;
    // as many as an SM holds; backward: 96 registers a thread for rows of few words, 128, 64 with more than 512 threads
    const bool small = p.threads <= 128 && (p.vpt == 1 || c.dtype == SSE_F32);
    const int hold_threads = !backward ? forward_threads(p.vpt, c.dtype == SSE_BF16 ? 2 : 4) : small ? 640 : p.threads <= 512 ? 512 : 1024;
    int per_sm = hold_threads / p.threads;
    if (per_sm < 1) per_sm = 1;
    const int enough = (p.threads <= 128 ? 384 : 512) / p.threads;
    if (!backward && residual && p.vpt <= 2 && per_sm > enough) per_sm = enough;
    const int64_t need = (T + p.teams - 1) / p.teams, hold = (int64_t)kSms * per_sm;
    p.grid = (int)(need < hold ? need : hold);
    return p;
}

template <typename T, int VPT, int MAXT> cudaError_t launch_forward_t(const LnPlan &p, const LayerNormArgs &a, cudaStream_t s) {
    const auto kernel = layer_norm_kernel<T, VPT, MAXT>;
    constexpr int kBytes = VPT <= 2 ? Ahead<T, VPT, 2, 2>::kBytes : 0;  // of a thread
    if constexpr (kBytes * MAXT > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes * MAXT);
        if (e != cudaSuccess) return e;
    }
    kernel<<<p.grid, p.threads, kBytes * p.threads, s>>>(a, p.n);
    return cudaGetLastError();
}
template <typename T> cudaError_t launch_forward(const LnPlan &p, const LayerNormArgs &a, cudaStream_t s) {
    if (p.vpt == 1) return launch_forward_t<T, 1, 128>(p, a, s);
    if (p.vpt > 2) return launch_forward_t<T, 4, 512>(p, a, s);
    return p.threads <= 128 ? launch_forward_t<T, 2, 128>(p, a, s) : launch_forward_t<T, 2, 320>(p, a, s);
}

template <typename T, int VPT, int MAXT> cudaError_t launch_backward_t(const LnPlan &p, const LayerNormArgs &a, cudaStream_t s) {
    const auto kernel = layer_norm_backward_kernel<T, VPT, MAXT>;
    constexpr int kSums = MAXT > kInRegisters ? VPT * 16 / (int)sizeof(T) / 2 * 16 : 0;
    constexpr int kBytes = kSums + Ahead<T, VPT, 3, rows_ahead(MAXT)>::kBytes;  // of a thread
    static_assert(kBytes * MAXT + 1024 <= 227 * 1024, "shared memory");
    if constexpr (kBytes * MAXT > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes * MAXT);
        if (e != cudaSuccess) return e;
    }
    kernel<<<p.grid, p.threads, kBytes * p.threads, s>>>(a, p.n);
    return cudaGetLastError();
}
template <typename T> cudaError_t launch_backward(const LnPlan &p, const LayerNormArgs &a, cudaStream_t s) {
    if (p.vpt == 1) return launch_backward_t<T, 1, 128>(p, a, s);
    if (p.threads <= 128) return launch_backward_t<T, 2, 128>(p, a, s);
    if (p.threads <= kInRegisters) return launch_backward_t<T, 2, kInRegisters>(p, a, s);
    return launch_backward_t<T, 2, 1024>(p, a, s);
}

}  // namespace

int64_t layer_norm_partial_rows(const sse_layer_norm_config_t &cfg, int64_t T) {
    const LnPlan p = plan(cfg, T, true, true);
    return (int64_t)p.grid * p.teams;
}

cudaError_t launch_layer_norm(const sse_layer_norm_config_t &cfg, const LayerNormArgs &a, cudaStream_t stream) {
    const LnPlan p = plan(cfg, a.T, false, a.r != nullptr);
    return cfg.dtype == SSE_BF16 ? launch_forward<__nv_bfloat16>(p, a, stream) : launch_forward<float>(p, a, stream);
}

cudaError_t launch_layer_norm_backward(const sse_layer_norm_config_t &cfg, const LayerNormArgs &a, cudaStream_t stream) {
    const LnPlan p = plan(cfg, a.T, true, true);
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
