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
// A team of threads covers a row, two 16-byte words per thread (one for rows up
// to 512 bytes), and goes from row to row; each thread copies its own words of
// the rows ahead to shared memory asynchronously (no barrier: nobody else reads
// them), so the next rows' loads are in flight while this one is summed.  Sums
// over the row go through shuffles and one word per warp of shared memory; sums
// over a group of columns through shuffles where the group is a power of two of
// lanes, else through shared memory: up to 32 words by every thread for its own,
// beyond by a warp per group.  Arithmetic is on float32 pairs.  Measured on a
// GB300, bf16, against the bytes at 6.77 TB/s: per-head norm and gate of 32768 x
// 2048 67 us (floor 59.5); norm, scale, residual and next norm of 16384 x 2304 53
// us (44.6); backward of head norm, gate, residual and next norm of 32768 x 2048
// 182 us (158.6); the norm before alone, 32768 x 2048, 52 us (39.6).  Groups of 96
// and 192 columns: 16384 x 2304 67 and 71 us (44.6), backward 131 and 138 (66.9);
// of 512: 16384 x 2048 with a gate 63 (49.6) and 121 (79.3).  float32, 16384 x
// 2048, norm over the row, gate, residual and next norm: 120 us (99.1) and 165
// (158.6).  Rows of 16384 columns have 64 registers per thread and spill: 4096 of
// them 123 us (79.3) and 331 (118.9).  One word per thread left the same backward
// (every part, 32768 x 2048) at 254 us: the control flow of a row (600 instructions
// per word then, 510 now) is shared by two words.  Bound now by issue at 16 warps
// per SM (60 % of the slots) as much as by HBM.
#include "f32x2.cuh"
#include "sse_internal.cuh"

namespace sse {
namespace {

constexpr int kSms = 152;
constexpr size_t kRoom = 220 * 1024;  // shared memory of an SM that the CTAs of a call may take together

// How the sum of squares of the norm after the block is shared.
enum { kGroupNone, kGroupRow, kGroupShuffle, kGroupShared, kGroupWide };

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
    static __device__ __forceinline__ void store(char *at, const F2 (&f)[kP]) {
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
        *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ F2 both(float x) { return f2(x, x); }

// 1 / (1 + exp(-z)).  For bf16 gates from the approximate exponential and reciprocal: the product's rounding is |z|
// 2^-24 of exp(-z), next to the gates' own steps of 2^-8 nothing.  In float32 that would be up to 2^-18 of a gate that
// is almost closed, so exp is expf there.  The reciprocal is one unit in the last place off (the quotient in its place:
// 16384 x 2048, head norm 110 against 120 us and backward 172 against 192, but groups of 256 165 against 148, 8192
// columns 125 against 118, and the norm before alone, which has no gate, 54 against 52).
template <typename T> __device__ __forceinline__ F2 sigmoid2(F2 z) {
    if constexpr (sizeof(T) == 4) {
        const float2 v = f2_get(z);
        float x, y;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(1.f + expf(-v.x)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + expf(-v.y)));
        return f2(x, y);
    }
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
template <typename T, bool GRAD, int P> __device__ __forceinline__ void act(int gate, F2 (&z)[P], F2 (&d)[P]) {
    if (gate == SSE_GATE_SILU) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const F2 s = sigmoid2<T>(z[i]);
            if (GRAD) d[i] = mul2(s, fma2(z[i], fma2(s, both(-1.f), both(1.f)), both(1.f)));
            z[i] = mul2(z[i], s);
        }
    } else if (gate == SSE_GATE_SIGMOID) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            z[i] = sigmoid2<T>(z[i]);
            if (GRAD) d[i] = mul2(z[i], fma2(z[i], both(-1.f), both(1.f)));
        }
    } else if (GRAD) {
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = both(1.f);
    }
}

// At most 2^-22.9 off, in float32 rows too: once per row or group, next to the 2^-24 of every product behind it.
__device__ __forceinline__ float rsqrt_ftz(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
    float *vec_words;   // [rows][words of a row]: kGroupShared and kGroupWide
    int turn;
    __device__ __forceinline__ Team(uint4 *smem, uint32_t sums_at, uint32_t words_at) {
        warp_words = reinterpret_cast<float *>(reinterpret_cast<char *>(smem) + sums_at);
        vec_words = reinterpret_cast<float *>(reinterpret_cast<char *>(smem) + words_at);
        turn = 0;
        for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 4 * 32 * (int)blockDim.y; i += blockDim.x * blockDim.y)
            warp_words[i] = 0.f;
        __syncthreads();
    }
    __device__ __forceinline__ float gather(const float *w) const {
        float4 v = *reinterpret_cast<const float4 *>(w);
        float s = (v.x + v.y) + (v.z + v.w);
        for (int k = 4; k < (int)blockDim.x >> 5; k += 4) {
            v = *reinterpret_cast<const float4 *>(w + k);
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
// WIDE: the kernels for groups of more than 32 words, kGroupWide, and no others
// (in one kernel with the rest it took registers of those: the norm before alone
// of 16384 x 2304 bf16 42 against 38 us).
template <bool WIDE, int VPT>
__device__ __forceinline__ void group_sum(Team &tm, int mode, int gw, int nv, float (&v)[VPT]) {
    if constexpr (WIDE) {
        // A warp adds up a group, 32 words at a time, into the place of its first word: no sum has more than 32 terms
        // one after the other.
        float *w = tm.vec_words + threadIdx.y * nv;
        __syncthreads();  // the sums of the call before have been read
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (j < nv) w[j] = v[i];
        }
        __syncthreads();
        for (int j0 = ((int)threadIdx.x >> 5) * gw; j0 < nv; j0 += ((int)blockDim.x >> 5) * gw) {
            float s = 0.f;
            for (int k = threadIdx.x & 31; k < gw; k += 32) s += w[j0 + k];
            s = warp_sum(s);
            if ((threadIdx.x & 31) == 0) w[j0] = s;  // which only this lane has read
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int j = threadIdx.x + i * blockDim.x;
            if (j < nv) v[i] = w[j / gw * gw];
        }
    } else if (mode == kGroupRow) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) s += v[i];
        float t[1] = {s};
        tm.row_sum<1>(t);
#pragma unroll
        for (int i = 0; i < VPT; ++i) v[i] = t[0];
    } else if (mode == kGroupShuffle) {  // a power of two of neighbouring lanes
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < gw)
#pragma unroll
                for (int i = 0; i < VPT; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    } else {  // up to 32 words: each thread adds up its words' groups
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
    // The launch's layout, here so that it takes no registers.
    int stages;                                // rows of a thread's ring
    uint32_t stage_bytes, vec;                 // bytes of a stage of the ring; between a thread's words of a row
    uint32_t slot[5], word;                    // a tensor's place in a stage (absent ones share one of zeros), its words
    uint32_t coef_at, sums_at, words_at;       // shared memory: coefficients, Team's words
    int64_t stride[5], packed;                 // bytes of a row in each fetched tensor and in a packed one
    int gate;
    float eps, rs, bs;
    float inv_width, inv_group;
};

// A thread's ring of rows: TENSORS x VPT words per row, each thread's own.  The
// slot of a row is free again when its words have been taken to registers.
// Words past the row's end, rows past the last one and absent tensors read as
// zeros.
template <int TENSORS, int VPT> struct Ring {
    uint32_t at;  // this thread's first word
    const void *const (&base)[TENSORS];  // null: absent

    __device__ __forceinline__ Ring(const NormShape &n, const void *const (&tensors)[TENSORS]) : base(tensors) {
        extern __shared__ uint4 smem[];
        at = (uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.y * blockDim.x + threadIdx.x) * 16;
        for (int s = 0; s < n.stages; ++s)  // the words that no fetch writes
#pragma unroll
            for (int t = 0; t < TENSORS; ++t)
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (!base[t] || !col_ok(n, i)) clear(at + s * n.stage_bytes + n.slot[t] + i * n.word);
    }
    static __device__ __forceinline__ bool col_ok(const NormShape &n, int i) {
        return (int)threadIdx.x + i * (int)blockDim.x < n.nv;
    }
    static __device__ __forceinline__ void clear(uint32_t dst) {
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
    }
    // Tensors T0 to T1 of one row, as one group of copies.
    template <int T0, int T1> __device__ __forceinline__ void fetch(const NormShape &n, int stage, int64_t row, bool row_ok) {
        const uint32_t dst = at + stage * n.stage_bytes;
#pragma unroll
        for (int t = T0; t < T1; ++t) {
            if (!base[t]) continue;
            if (row_ok) {
                const char *src = static_cast<const char *>(base[t]) + row * n.stride[t] + threadIdx.x * 16;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %2, 0;\n@p cp.async.cg.shared.global [%0], [%1], 16;\n}"
                                 ::"r"(dst + n.slot[t] + i * n.word), "l"(src + i * n.vec), "r"((uint32_t)col_ok(n, i))
                                 : "memory");
            } else {
#pragma unroll
                for (int i = 0; i < VPT; ++i) clear(dst + n.slot[t] + i * n.word);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ uint4 take(const NormShape &n, int stage, int t, int i) const {
        uint4 u;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "r"(at + stage * n.stage_bytes + n.slot[t] + i * n.word) : "memory");
        return u;
    }
};
// This thread's word of a row of a packed output.
__device__ __forceinline__ char *word_of(void *base, const NormShape &n, int64_t row, int i) {
    return static_cast<char *>(base) + row * n.packed + threadIdx.x * 16 + i * n.vec;
}
// Waits for the oldest of `stages` rows' groups, GROUPS to a row.
template <int GROUPS> __device__ __forceinline__ void fetches_wait(int stages) {
    if (stages == 3)
        asm volatile("cp.async.wait_group %0;" ::"n"(3 * GROUPS - 1) : "memory");
    else if (stages == 2)
        asm volatile("cp.async.wait_group %0;" ::"n"(2 * GROUPS - 1) : "memory");
    else
        asm volatile("cp.async.wait_group %0;" ::"n"(GROUPS - 1) : "memory");
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

template <typename T, int VPT, int MAXT, bool WIDE>
__global__ void __launch_bounds__(MAXT, VPT == 1 ? 8 : 1) norm_forward_kernel(BlockNormArgs a, NormShape n) {
    constexpr int P = Row<T>::kP;
    extern __shared__ uint4 smem[];
    const bool has_o = a.o != nullptr, has_z = a.z != nullptr, has_r = a.r != nullptr;
    const int64_t on = (int64_t)gridDim.x * blockDim.y, row0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    // rows of this team, and of the CTA's first (the others have as many or one less)
    const int mine = row0 < a.T ? (int)((a.T - 1 - row0) / on) + 1 : 0;
    const int most = (int)((a.T - 1 - (int64_t)blockIdx.x * blockDim.y) / on) + 1;
    const void *const tensors[3] = {a.o, a.z, a.r};
    Ring<3, VPT> ring(n, tensors);
    for (int k = 0; k < n.stages; ++k) ring.template fetch<0, 3>(n, k, row0 + k * on, k < mine);
    F2 coef[VPT][P], wb[VPT][P];
    load_coef<T, VPT>(a, n, coef, wb);
    Team tm(smem, n.sums_at, n.words_at);
    int stage = 0;
    int64_t row = row0;
    for (int k = 0; k < most; ++k, row += on) {
        const bool live = k < mine;
        F2 u[VPT][P];
        uint4 uz[VPT], ur[VPT];
        fetches_wait<1>(n.stages);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            Row<T>::unpack(ring.take(n, stage, 0, i), u[i]);
            uz[i] = ring.take(n, stage, 1, i);
            ur[i] = ring.take(n, stage, 2, i);
        }
        ring.template fetch<0, 3>(n, stage, row + n.stages * on, k + n.stages < mine);
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
            group_sum<WIDE>(tm, n.mode, n.gw, n.nv, ss);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const F2 rstd = both(rsqrt_ftz(fmaf(ss[i], n.inv_group, n.eps)));
#pragma unroll
                for (int k = 0; k < P; ++k) u[i][k] = mul2(u[i][k], rstd);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int k = 0; k < P; ++k) u[i][k] = mul2(u[i][k], coef[i][k]);
            if (has_z) {
                F2 z[P], none[P];
                Row<T>::unpack(uz[i], z);
                act<T, false>(n.gate, z, none);
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
            if (a.r_out && live && ring.col_ok(n, i))
                Row<T>::store(word_of(a.r_out, n, row, i), u[i]);
        }
        if (a.next) {
            F2 t = both(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int k = 0; k < P; ++k) t = fma2(u[i][k], u[i][k], t);
            float sum[1] = {fold(t)};
            tm.row_sum<1>(sum);
            const F2 rstd = both(rsqrt_ftz(fmaf(sum[0], n.inv_width, n.eps)));
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
#pragma unroll
                for (int k = 0; k < P; ++k) u[i][k] = mul2(mul2(u[i][k], rstd), wb[i][k]);
                if (live && ring.col_ok(n, i)) Row<T>::store(word_of(a.next, n, row, i), u[i]);
            }
        }
    }
}

// The backward's coefficients: registers hold the column sums instead.  Both
// vectors in shared memory, a word's 16-byte pieces nv apart (no bank conflicts);
// the widest rows (SMEM false) leave no room for them beside the ring, and read
// them from global memory.
template <typename T, bool SMEM> struct Coefs {
    static constexpr int E = Row<T>::kE, P = Row<T>::kP;
    const float4 *smem;  // [2][E / 4][nv]: coef, w_before
    int nv;
    __device__ __forceinline__ void fill(const BlockNormArgs &a, const NormShape &n, float4 *at) {
        smem = at;
        nv = n.nv;
        if (!SMEM) return;
        const int threads = blockDim.x * blockDim.y;
        for (int q = threadIdx.y * blockDim.x + threadIdx.x; q < n.nv * (E / 4); q += threads) {
            const int j = q / (E / 4), h = q % (E / 4);
            float4 c, b;
            load(a, n, j, h, c, b);
            at[h * n.nv + j] = c;
            at[(E / 4 + h) * n.nv + j] = b;
        }
    }
    static __device__ __forceinline__ void load(const BlockNormArgs &a, const NormShape &n, int j, int h, float4 &c,
                                                float4 &b) {
        const int at = j * E + 4 * h;
        c = make_float4(n.bs, n.bs, n.bs, n.bs);
        b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.w_after) {
            const float4 w = __ldg(reinterpret_cast<const float4 *>(a.w_after + at));
            c.x *= w.x; c.y *= w.y; c.z *= w.z; c.w *= w.w;
        }
        if (a.channel) {
            const float4 w = __ldg(reinterpret_cast<const float4 *>(a.channel + at));
            c.x *= w.x; c.y *= w.y; c.z *= w.z; c.w *= w.w;
        }
        if (a.w_before) b = __ldg(reinterpret_cast<const float4 *>(a.w_before + at));
    }
    // which: 0 coef, 1 w_before
    __device__ __forceinline__ void get(const BlockNormArgs &a, const NormShape &n, int which, int j, F2 (&f)[P]) const {
        if (j >= nv) j = nv - 1;  // a word past the row meets zeros
#pragma unroll
        for (int h = 0; h < E / 4; ++h) {
            float4 v;
            if constexpr (SMEM) {
                v = smem[(which * (E / 4) + h) * nv + j];
            } else {
                float4 c, b;
                load(a, n, j, h, c, b);
                v = which ? b : c;
            }
            f[2 * h] = f2(v.x, v.y);
            f[2 * h + 1] = f2(v.z, v.w);
        }
    }
};

template <typename T, int VPT, int MAXT, bool WIDE>
__global__ void __launch_bounds__(MAXT, VPT == 1 ? 5 : 1) norm_backward_kernel(BlockNormArgs a, NormShape n) {
    constexpr int E = Row<T>::kE, P = Row<T>::kP;
    extern __shared__ uint4 smem[];
    const bool has_o = a.o != nullptr, has_z = a.z != nullptr, has_n = a.d_next != nullptr;
    const int64_t on = (int64_t)gridDim.x * blockDim.y, row0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    // rows of this team, and of the CTA's first (the others have as many or one less)
    const int mine = row0 < a.T ? (int)((a.T - 1 - row0) / on) + 1 : 0;
    const int most = (int)((a.T - 1 - (int64_t)blockIdx.x * blockDim.y) / on) + 1;
    // the first three make dr', and their place in the ring is free again while the last two are at work
    const void *const tensors[5] = {a.d_r_out, has_n ? a.r : nullptr, a.d_next, a.o, a.z};
    Ring<5, VPT> ring(n, tensors);
    for (int k = 0; k < n.stages; ++k) {
        ring.template fetch<0, 3>(n, k, row0 + k * on, k < mine);
        ring.template fetch<3, 5>(n, k, row0 + k * on, k < mine);
    }
    Coefs<T, MAXT <= 512> co;
    co.fill(a, n, reinterpret_cast<float4 *>(reinterpret_cast<char *>(smem) + n.coef_at));
    Team tm(smem, n.sums_at, n.words_at);
    F2 sum_c[VPT][P], sum_b[VPT][P];  // C_j and dw_before of the thread's columns
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < P; ++k) sum_c[i][k] = sum_b[i][k] = both(0.f);
    int stage = 0;
    int64_t row = row0;
    for (int k = 0; k < most; ++k, row += on) {
        const bool live = k < mine;
        F2 d[VPT][P];
        fetches_wait<2>(n.stages);
        float rstd_row = 0.f, minus_mean = 0.f;
        if (has_n) {
            F2 ss = both(0.f), dot = both(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                F2 r[P], g[P], w[P];
                Row<T>::unpack(ring.take(n, stage, 1, i), r);
                Row<T>::unpack(ring.take(n, stage, 2, i), g);
                co.get(a, n, 1, threadIdx.x + i * blockDim.x, w);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    ss = fma2(r[k], r[k], ss);
                    dot = fma2(mul2(g[k], w[k]), r[k], dot);
                }
            }
            float sums[2] = {fold(ss), fold(dot)};
            tm.row_sum<2>(sums);
            rstd_row = rsqrt_ftz(fmaf(sums[0], n.inv_width, n.eps));
            minus_mean = -(sums[1] * rstd_row * n.inv_width);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            Row<T>::unpack(ring.take(n, stage, 0, i), d[i]);
            if (has_n) {
                F2 r[P], g[P], w[P];
                Row<T>::unpack(ring.take(n, stage, 1, i), r);
                Row<T>::unpack(ring.take(n, stage, 2, i), g);
                co.get(a, n, 1, threadIdx.x + i * blockDim.x, w);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    const F2 hat = mul2(r[k], both(rstd_row));
                    sum_b[i][k] = fma2(g[k], hat, sum_b[i][k]);
                    d[i][k] = fma2(both(rstd_row), fma2(hat, both(minus_mean), mul2(g[k], w[k])), d[i][k]);
                }
            }
            if (a.d_r && live && ring.col_ok(n, i)) {
                F2 v[P];
#pragma unroll
                for (int k = 0; k < P; ++k) v[k] = mul2(both(n.rs), d[i][k]);
                Row<T>::store(word_of(a.d_r, n, row, i), v);
            }
        }
        ring.template fetch<0, 3>(n, stage, row + n.stages * on, k + n.stages < mine);
        fetches_wait<2>(n.stages);
        if (has_o) {
            float rstd[VPT], dot[VPT];
            if (n.mode != kGroupNone) {
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    F2 o[P], t = both(0.f);
                    Row<T>::unpack(ring.take(n, stage, 3, i), o);
#pragma unroll
                    for (int k = 0; k < P; ++k) t = fma2(o[k], o[k], t);
                    rstd[i] = fold(t);
                }
                group_sum<WIDE>(tm, n.mode, n.gw, n.nv, rstd);
#pragma unroll
                for (int i = 0; i < VPT; ++i) rstd[i] = rsqrt_ftz(fmaf(rstd[i], n.inv_group, n.eps));
            } else {
#pragma unroll
                for (int i = 0; i < VPT; ++i) rstd[i] = 1.f;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                F2 o[P], c[P];
                Row<T>::unpack(ring.take(n, stage, 3, i), o);
                co.get(a, n, 0, threadIdx.x + i * blockDim.x, c);
#pragma unroll
                for (int k = 0; k < P; ++k) o[k] = mul2(o[k], both(rstd[i]));
                if (has_z) {
                    F2 av[P], da[P];
                    Row<T>::unpack(ring.take(n, stage, 4, i), av);
                    act<T, true>(n.gate, av, da);
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        da[k] = mul2(mul2(mul2(d[i][k], c[k]), o[k]), da[k]);
                        d[i][k] = mul2(d[i][k], av[k]);
                    }
                    if (live && ring.col_ok(n, i)) Row<T>::store(word_of(a.d_z, n, row, i), da);
                }
                F2 t = both(0.f);
#pragma unroll
                for (int k = 0; k < P; ++k) {
                    sum_c[i][k] = fma2(d[i][k], o[k], sum_c[i][k]);
                    d[i][k] = mul2(d[i][k], c[k]);
                    t = fma2(d[i][k], o[k], t);
                }
                dot[i] = fold(t);
            }
            if (n.mode != kGroupNone) {
                group_sum<WIDE>(tm, n.mode, n.gw, n.nv, dot);
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    // d = rstd (d - o_hat mean), o_hat = o rstd
                    const F2 f = both(-dot[i] * n.inv_group * rstd[i]);
                    F2 o[P];
                    Row<T>::unpack(ring.take(n, stage, 3, i), o);
#pragma unroll
                    for (int k = 0; k < P; ++k) d[i][k] = mul2(both(rstd[i]), fma2(o[k], f, d[i][k]));
                }
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (live && ring.col_ok(n, i)) Row<T>::store(word_of(a.d_o, n, row, i), d[i]);
        }
        ring.template fetch<3, 5>(n, stage, row + n.stages * on, k + n.stages < mine);
        stage = stage + 1 == n.stages ? 0 : stage + 1;
    }
    griddep_launch_dependents();
    // column sums of this team: one partial row of each
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int j = threadIdx.x + i * blockDim.x;
        if (j < n.nv) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
                if (a.d_w_after || a.d_channel)
                    *reinterpret_cast<float2 *>(a.partials + row0 * n.width + j * E + 2 * k) = f2_get(sum_c[i][k]);
                if (a.d_w_before)
                    *reinterpret_cast<float2 *>(a.partials + (on + row0) * n.width + j * E + 2 * k) = f2_get(sum_b[i][k]);
            }
        }
    }
}

// The weights' gradients from the partial rows, in a fixed order: 32 columns of
// one array (blockIdx.y: C_j, dw_before) per CTA, 32 interleaved runs of rows,
// then their sum.  Launched as a dependent of the gradient kernel.
__global__ void __launch_bounds__(1024) norm_weight_grads_kernel(BlockNormArgs a, NormShape n, int rows) {
    __shared__ float part[32][33];
    const int c = threadIdx.x, col = blockIdx.x * 32 + c;
    const bool before = blockIdx.y != 0;
    griddep_wait();
    if (before ? !a.d_w_before : !a.d_w_after && !a.d_channel) return;
    const float *from = a.partials + (before ? (int64_t)rows * n.width : 0) + col;
    float s = 0.f;
    if (col < n.width) {
#pragma unroll 8
        for (int r = threadIdx.y; r < rows; r += 32) s += from[(int64_t)r * n.width];
    }
    part[threadIdx.y][c] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < n.width) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += part[r][c];
        if (before) {
            a.d_w_before[col] = t;
        } else {
            const float w = a.w_after ? a.w_after[col] : 1.f, ch = a.channel ? a.channel[col] : 1.f;
            if (a.d_w_after) a.d_w_after[col] = n.bs * ch * t;
            if (a.d_channel) a.d_channel[col] = n.bs * w * t;
        }
    }
}

struct NormPlan {
    NormShape n;
    int vpt, threads, rows;  // words per thread, threads of a row, rows per CTA
    int per_sm;              // CTAs on an SM
    uint32_t row_bytes, coef_bytes, sum_bytes;  // shared memory: a row in the ring, the coefficients, the sums' words
    size_t smem;
};

int most_per_sm(const NormPlan &p, bool backward) {
    const int n = (p.vpt == 2 ? 512 : backward ? 640 : 1024) / (p.threads * p.rows);
    return n < 1 ? 1 : n;
}

NormPlan plan_norm(const sse_norm_config_t &c, const BlockNormArgs &a, bool backward) {
    NormPlan p{};
    const bool after = a.w_after != nullptr;
    const int E = c.dtype == SSE_BF16 ? 8 : 4;
    const int group = c.group ? c.group : c.width;
    p.n.width = c.width;
    p.n.nv = c.width / E;
    p.n.gw = group / E;
    const bool pow2 = (p.n.gw & (p.n.gw - 1)) == 0;
    p.n.mode = !after ? kGroupNone : group == c.width ? kGroupRow : p.n.gw > 32 ? kGroupWide : pow2 ? kGroupShuffle : kGroupShared;
    p.n.gate = c.gate;
    p.n.eps = c.eps;
    p.n.rs = c.residual_scale;
    p.n.bs = c.branch_scale;
    p.n.inv_width = 1.f / c.width;
    p.n.inv_group = 1.f / group;
    // Two words per thread: the control flow of a row is shared by both.
    p.vpt = p.n.nv <= 32 ? 1 : 2;
    p.threads = ((p.n.nv + p.vpt - 1) / p.vpt + 31) / 32 * 32;
    p.rows = p.threads >= 128 ? 1 : 128 / p.threads;
    p.coef_bytes = backward && p.threads <= 512 ? 2 * c.width * (uint32_t)sizeof(float) : 0;
    p.sum_bytes = sizeof(float) * 4 * 32 * p.rows;
    // a stage of the ring: the tensors that the call has, and words of zeros for the others
    const void *const fwd[5] = {a.o, a.z, a.r}, *const bwd[5] = {a.d_r_out, a.d_next ? a.r : nullptr, a.d_next, a.o, a.z};
    p.n.word = p.threads * p.rows * 16;
    uint32_t present = 0;
    for (int t = 0; t < (backward ? 5 : 3); ++t)
        if ((backward ? bwd : fwd)[t]) p.n.slot[t] = present++ * p.vpt * p.n.word;
    for (int t = 0; t < (backward ? 5 : 3); ++t)
        if (!(backward ? bwd : fwd)[t]) p.n.slot[t] = present * p.vpt * p.n.word;
    p.row_bytes = (present + (present < (backward ? 5 : 3))) * p.vpt * p.n.word;
    const size_t fixed = p.coef_bytes + p.sum_bytes + (p.n.mode >= kGroupShared ? sizeof(float) * p.rows * p.n.nv : 0);
    // As many CTAs on an SM as its registers and shared memory hold (up to 128 registers per thread with two words, 64
    // and 96 with one), then up to three rows of each.
    p.per_sm = most_per_sm(p, backward);
    while (p.per_sm > 1 && p.per_sm * (p.row_bytes + fixed) > kRoom) --p.per_sm;
    p.n.stages = 3;
    while (p.n.stages > 1 && p.per_sm * (p.n.stages * p.row_bytes + fixed) > kRoom) --p.n.stages;
    p.smem = p.n.stages * p.row_bytes + fixed;
    return p;
}

int norm_grid(const NormPlan &p, int64_t T) {
    const int64_t need = (T + p.rows - 1) / p.rows, most = (int64_t)kSms * p.per_sm;
    return (int)(need < most ? need : most);
}

template <typename T, int VPT, int MAXT, bool WIDE>
cudaError_t launch_t(NormPlan p, const BlockNormArgs &a, bool backward, cudaStream_t stream) {
    const auto kernel = backward ? norm_backward_kernel<T, VPT, MAXT, WIDE> : norm_forward_kernel<T, VPT, MAXT, WIDE>;
    if (p.smem > 48 * 1024) {
        // The limit belongs to the kernel and not to the call, whose size differs from that of another host thread's:
        // every call sets the same one.
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRoom);
        if (e != cudaSuccess) return e;
    }
    const int64_t width = p.n.width, fwd[5] = {a.o_stride, a.z_stride, a.r_stride, 0, 0},
                  bwd[5] = {width, a.r_stride, width, a.o_stride, a.z_stride};
    for (int t = 0; t < 5; ++t) p.n.stride[t] = (backward ? bwd : fwd)[t] * (int64_t)sizeof(T);
    p.n.packed = width * (int64_t)sizeof(T);
    p.n.stage_bytes = p.row_bytes;
    p.n.vec = p.threads * 16;
    p.n.coef_at = p.n.stages * p.row_bytes;
    p.n.sums_at = p.n.coef_at + p.coef_bytes;
    p.n.words_at = p.n.sums_at + p.sum_bytes;
    kernel<<<norm_grid(p, a.T), dim3(p.threads, p.rows), p.smem, stream>>>(a, p.n);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rows(const NormPlan &p, const BlockNormArgs &a, bool backward, cudaStream_t stream) {
    if (p.vpt == 1) return launch_t<T, 1, 128, false>(p, a, backward, stream);  // 32 words at most
    const bool wide = p.n.mode == kGroupWide;
    if (p.threads <= 512)
        return wide ? launch_t<T, 2, 512, true>(p, a, backward, stream) : launch_t<T, 2, 512, false>(p, a, backward, stream);
    return wide ? launch_t<T, 2, 1024, true>(p, a, backward, stream) : launch_t<T, 2, 1024, false>(p, a, backward, stream);
}

}  // namespace

int64_t block_norm_partial_rows(const sse_norm_config_t &cfg, int64_t T) {
    // at most: a call's own plan has as many CTAs on an SM or fewer
    NormPlan p = plan_norm(cfg, BlockNormArgs{}, true);
    p.per_sm = most_per_sm(p, true);
    return (int64_t)norm_grid(p, T) * p.rows;
}

cudaError_t launch_block_norm(const sse_norm_config_t &cfg, const BlockNormArgs &a, cudaStream_t stream) {
    const NormPlan p = plan_norm(cfg, a, false);
    return cfg.dtype == SSE_BF16 ? launch_rows<__nv_bfloat16>(p, a, false, stream)
                                 : launch_rows<float>(p, a, false, stream);
}

cudaError_t launch_block_norm_backward(const sse_norm_config_t &cfg, const BlockNormArgs &a, cudaStream_t stream) {
    const NormPlan p = plan_norm(cfg, a, true);
    if (a.T > 0) {
        const cudaError_t e = cfg.dtype == SSE_BF16 ? launch_rows<__nv_bfloat16>(p, a, true, stream)
                                                    : launch_rows<float>(p, a, true, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.d_w_after || a.d_channel || a.d_w_before) {
        const int rows = norm_grid(p, a.T) * p.rows;
        return launch_dependent(norm_weight_grads_kernel, dim3((cfg.width + 31) / 32, 2), dim3(32, 32), 0, stream, a, p.n,
                                rows);
    }
    return cudaSuccess;
}

}  // namespace sse
