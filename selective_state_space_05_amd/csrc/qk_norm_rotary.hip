// qk_norm_rotary.hip -- norm of queries and keys for each head with their rotation
// by position in the same pass, forward and backward.
//
//   n = x r w,  r = 1 / sqrt(mean(x^2) + eps)
//   y_j = n_j cos a_j - n_{j+R/2} sin a_j,  y_{j+R/2} = n_{j+R/2} cos a_j + n_j sin a_j
//   a_j = position base^(-2j/R) for j < R/2;  values from R on are not rotated
// and, with dn the gradient turned back and e = dn w,
//   dx = r (e - x r^2 mean(e x)),   dw = sum over tokens and heads of dn x r
//
// Bound by memory: every value is read once and written once.  A group of lanes
// holds a head, each lane the two vectors of one or two slots, which the rotation
// pairs with each other, so nothing but the sums of squares and of products passes
// between lanes; the next head is under way meanwhile.  A workgroup has a run of
// tokens of q or of k, so that weights and their gradients' sums stay in registers.  A
// token's sines and cosines are formed once for all its heads, into LDS: the angle in
// turns in float64, where 2^20 positions keep their digits, its fraction in float32 with a
// turn by what that left (sines are off by 0.32 of a rounding of 1 in the root mean square,
// without that turn by 0.55).
// Measured in bfloat16 at 8192 tokens of 20 + 20 heads of 128: forward 31 us (5.4 TB/s),
// backward 49 us (5.1 TB/s) and 4.6 us for the weights' sums; 8 tokens 4 us.  Widths or
// rotated parts that are no multiple of two vectors go element by element: 8192 tokens of
// 20 + 20 heads of 120 in whole calls 82 us in bfloat16 (1.9 TB/s), 58 us in float32, where
// they are whole vectors (5.4 TB/s).
#include <algorithm>
#include <type_traits>

#include "device_math.h"
#include "internal.h"

namespace mssm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kMaxHalf = MSSM_MAX_HEAD_DIM / 2;

// VEC consecutive elements as they lie in memory, at any element's address.
template <typename T, int VEC> struct Vec;
template <> struct Vec<float, 4> {
    typedef u32x4 Any __attribute__((aligned(4)));
    u32x4 v;
    __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const Any *>(p); }
    __device__ __forceinline__ float get(int k) const { return __uint_as_float(v[k]); }
    __device__ __forceinline__ static void store(float *p, const float *f) {
        *reinterpret_cast<Any *>(p) = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                            __float_as_uint(f[3])};
    }
};
template <> struct Vec<uint16_t, 8> {
    typedef u32x4 Any __attribute__((aligned(2)));
    u32x4 v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const Any *>(p); }
    __device__ __forceinline__ float get(int k) const {
        return __uint_as_float(k % 2 ? v[k / 2] & 0xffff0000u : v[k / 2] << 16);
    }
    __device__ __forceinline__ static void store(uint16_t *p, const float *f) {
        typedef __bf16 b8 __attribute__((ext_vector_type(8)));
        b8 b;
#pragma unroll
        for (int k = 0; k < 8; ++k) b[k] = static_cast<__bf16>(f[k]);
        *reinterpret_cast<Any *>(p) = __builtin_bit_cast(u32x4, b);
    }
};
template <typename T> struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ float get(int) const { return Io<T>::load(&v, 0); }
    __device__ __forceinline__ static void store(T *p, const float *f) { Io<T>::store(p, 0, *f); }
};

// q or k: its workgroups have `run` tokens each, `tile` of them at a time.
struct Side {
    const void *x, *dy;
    void *y;
    const float *weight;
    float *part;             // backward: column sums of every workgroup, (dim) each; may be null
    int heads, run, blocks;
};

struct HeadNorm {
    Side q, k;
    const int64_t *positions;
    int64_t tokens;
    int dim, rotary, tile;
    double log2_base;
    float eps;
};

// Slot s of a head: the first elements of its two vectors, and the index of its first
// angle (-1: not rotated).  A head's last slot may lack its second vector (VEC 1).
template <int VEC>
struct Slot {
    int a, b, angle;
    bool has_a, has_b;
    __device__ __forceinline__ Slot(int s, int dim, int rotary) {
        const int half = rotary / 2;
        if (s * VEC < half) {
            a = s * VEC;
            b = half + a;
            angle = a;
        } else {
            a = rotary + 2 * (s * VEC - half);
            b = a + VEC;
            angle = -1;
        }
        has_a = a < dim;
        has_b = b < dim;
    }
};

// Sum over the G lanes of a group, the same in all of them.
template <int G>
__device__ __forceinline__ float group_sum(float x) {
    const auto dpp = [](float v, auto ctrl) {
        return __builtin_bit_cast(
            float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    x += dpp(x, std::integral_constant<int, 0xb1>());                             // quad_perm 1 0 3 2
    x += dpp(x, std::integral_constant<int, 0x4e>());                             // quad_perm 2 3 0 1
    if constexpr (G >= 8) x += dpp(x, std::integral_constant<int, 0x141>());      // halves of 8 mirrored
    if constexpr (G >= 16) x += dpp(x, std::integral_constant<int, 0x140>());     // rows of 16 mirrored
    if constexpr (G >= 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if constexpr (G >= 64) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return x;
}

// 1 / sqrt(mean(x^2) + eps) of a head, whose sum of squares is `ss`.  Where float32 cannot
// hold that sum (values from 1e18 on, or with no eps to speak of below 3e-14, where squares
// near the least normal number), of values that a power of two brings into its range.
template <int G, int N>
__device__ __forceinline__ float rstd_of(float ss, const float (&x)[N], float dim, float eps) {
    const float m = ss / dim + eps;
    if (m > 0x1p-90f && m < 0x1p120f) return 1.0f / sqrtf(m);
    const float by = m > 1.0f ? 0x1p-70f : 0x1p70f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum = fmaf(x[i] * by, x[i] * by, sum);
    return by / sqrtf(group_sum<G>(sum) / dim + eps * by * by);
}

// G lanes a head, SLOTS slots a lane.
template <typename T, int VEC, int G, int SLOTS, bool BWD>
__global__ __launch_bounds__(kThreads, 4) void head_norm_kernel(const HeadNorm N) {
    constexpr int GROUPS = kThreads / G;
    typedef Vec<T, VEC> V;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int half = N.rotary / 2;
    double *const rate = reinterpret_cast<double *>(smem);
    float2 *const turn = reinterpret_cast<float2 *>(rate + kMaxHalf);   // (tile, half): cos, sin
    for (int j = threadIdx.x; j < half; j += kThreads)                 // turns a position
        rate[j] = exp2(-N.log2_base * (2 * j) / N.rotary) * 0.15915494309189535;
    const bool of_k = static_cast<int>(blockIdx.x) >= N.q.blocks;
    const Side &S = of_k ? N.k : N.q;
    const int block = of_k ? blockIdx.x - N.q.blocks : blockIdx.x, heads = S.heads;
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    float w[SLOTS][2][VEC], dw[SLOTS][2][VEC];
    int at[SLOTS][2];                // elements of a head; -1: none
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const Slot<VEC> slot(lane + s * G, N.dim, N.rotary);
        at[s][0] = slot.has_a ? slot.a : -1;
        at[s][1] = slot.has_b ? slot.b : -1;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                w[s][i][j] = S.weight && at[s][i] >= 0 ? S.weight[at[s][i] + j] : 1.0f;
                dw[s][i][j] = 0.0f;
            }
    }
    const int64_t begin = static_cast<int64_t>(block) * S.run, end = min(begin + S.run, N.tokens);
    V x[SLOTS][2], g[SLOTS][2];
    auto load = [&](int64_t row) {   // of token row / heads
        const T *const px = static_cast<const T *>(S.x) + row * N.dim, *const pg = static_cast<const T *>(S.dy) + row * N.dim;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[s][i] = V{};
                g[s][i] = V{};
                if (at[s][i] >= 0) {
                    x[s][i].load(px + at[s][i]);
                    if (BWD) g[s][i].load(pg + at[s][i]);
                }
            }
    };
    if (begin * heads + group < end * heads) load(begin * heads + group);
    for (int64_t t0 = begin; t0 < end; t0 += N.tile) {
        const int count = static_cast<int>(min(static_cast<int64_t>(N.tile), end - t0));
        __syncthreads();
        for (int id = threadIdx.x; id < count * half; id += kThreads) {
            const double a = static_cast<double>(N.positions[t0 + id / half]) * rate[id % half];
            // the fraction's rounding to float32, up to 2^-26 turns, is turned back to first order
            const double turns = a - rint(a);
            const float f = static_cast<float>(turns), left = static_cast<float>((turns - f) * 6.283185307179586);
            float s, c;
            sincospif(2.0f * f, &s, &c);
            turn[id] = float2{fmaf(-s, left, c), fmaf(c, left, s)};
        }
        __syncthreads();
        for (int id = group; id < count * heads; id += GROUPS) {
            const int64_t row = t0 * heads + id;
            float xf[SLOTS][2][VEC], gf[SLOTS][2][VEC], ss = 0.0f;
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        xf[s][i][j] = x[s][i].get(j);
                        gf[s][i][j] = BWD ? g[s][i].get(j) : 0.0f;
                        ss = fmaf(xf[s][i][j], xf[s][i][j], ss);
                    }
            // the group's next head, of this tile or of the next one
            const int64_t next = id + GROUPS < count * heads ? row + GROUPS : (t0 + count) * heads + group;
            if (next < end * heads) load(next);
            const float r = rstd_of<G>(group_sum<G>(ss), reinterpret_cast<const float(&)[SLOTS * 2 * VEC]>(xf), N.dim, N.eps);
            const float2 *const my = turn + id / heads * half;
            float ex = 0.0f;
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                const int angle = (lane + s * G) * VEC;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float2 cs = angle < half ? my[angle + j] : float2{1.0f, 0.0f};
                    float &xa = xf[s][0][j], &xb = xf[s][1][j];
                    if (BWD) {
                        const float ga = gf[s][0][j], gb = gf[s][1][j];
                        const float na = fmaf(gb, cs.y, ga * cs.x), nb = fmaf(-ga, cs.y, gb * cs.x);
                        dw[s][0][j] = fmaf(na * r, xa, dw[s][0][j]);
                        dw[s][1][j] = fmaf(nb * r, xb, dw[s][1][j]);
                        gf[s][0][j] = na * w[s][0][j];
                        gf[s][1][j] = nb * w[s][1][j];
                        ex = fmaf(gf[s][0][j], xa, ex);
                        ex = fmaf(gf[s][1][j], xb, ex);
                    } else {
                        const float na = xa * r * w[s][0][j], nb = xb * r * w[s][1][j];
                        xa = fmaf(-nb, cs.y, na * cs.x);
                        xb = fmaf(na, cs.y, nb * cs.x);
                    }
                }
            }
            if (BWD) {
                const float c = group_sum<G>(ex) / N.dim * r * r;
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) xf[s][i][j] = r * fmaf(-xf[s][i][j], c, gf[s][i][j]);
            }
            T *const y = static_cast<T *>(S.y) + row * N.dim;
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (at[s][i] >= 0) V::store(y + at[s][i], xf[s][i]);
        }
    }
    if (BWD && S.part) {
        // the groups' column sums, added in the order of the groups
        float *const sum = reinterpret_cast<float *>(smem);   // (GROUPS, dim)
        __syncthreads();
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (at[s][i] >= 0) sum[group * N.dim + at[s][i] + j] = dw[s][i][j];
        __syncthreads();
        for (int d = threadIdx.x; d < N.dim; d += kThreads) {
            float v = 0.0f;
#pragma unroll 8
            for (int i = 0; i < GROUPS; ++i) v += sum[i * N.dim + d];
            S.part[static_cast<int64_t>(block) * N.dim + d] = v;
        }
    }
}

// Adds the workgroups' column sums of q (blockIdx.y 0) and k: 32 columns by 32 slices of
// the workgroups, then the slices in order.
__global__ __launch_bounds__(1024) void head_norm_sum_kernel(const float *__restrict__ q, int q_parts, float *__restrict__ dq,
                                                             const float *__restrict__ k, int k_parts, float *__restrict__ dk,
                                                             int dim) {
    __shared__ float sum[32][33];
    const float *const part = blockIdx.y ? k : q;
    const int parts = blockIdx.y ? k_parts : q_parts, c = threadIdx.x % 32, slice = threadIdx.x / 32;
    float *const to = blockIdx.y ? dk : dq;
    const int d = blockIdx.x * 32 + c;
    float v = 0.0f;
    if (d < dim)
#pragma unroll 4
        for (int i = slice; i < parts; i += 32) v += part[static_cast<int64_t>(i) * dim + d];
    sum[slice][c] = v;
    __syncthreads();
    if (slice || d >= dim || !to) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sum[i][c];
    to[d] = v;
}

constexpr int64_t kBlocks = 1024;   // four a compute unit, of q and k together; they run at once
constexpr int kTile = 16;           // tokens that a workgroup has the angles of at most

// Tokens of a workgroup of q or k, in proportion to their heads.
int64_t run_of(const HeadNormArgs &a, int64_t heads) {
    const int64_t blocks = std::max<int64_t>(1, kBlocks * heads / std::max<int64_t>(1, a.q_heads + a.k_heads));
    return (a.tokens + blocks - 1) / blocks;
}
int64_t blocks_of(const HeadNormArgs &a, int64_t heads) {
    return heads && a.tokens ? (a.tokens + run_of(a, heads) - 1) / run_of(a, heads) : 0;
}

template <typename T, bool BWD>
hipError_t launch(const HeadNormArgs &a, float *part, hipStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const int q_blocks = static_cast<int>(blocks_of(a, a.q_heads)), k_blocks = static_cast<int>(blocks_of(a, a.k_heads));
    const int q_run = static_cast<int>(run_of(a, a.q_heads)), k_run = static_cast<int>(run_of(a, a.k_heads));
    const int tile = std::min(kTile, std::max(q_blocks ? q_run : 1, k_blocks ? k_run : 1));
    const HeadNorm n{{a.q, a.dq, a.q_out, a.q_weight, part, static_cast<int>(a.q_heads), q_run, q_blocks},
                     {a.k, a.dk, a.k_out, a.k_weight, part ? part + q_blocks * a.dim : nullptr, static_cast<int>(a.k_heads),
                      k_run, k_blocks},
                     a.positions, a.tokens, static_cast<int>(a.dim), static_cast<int>(a.rotary), tile, log2(a.base), a.eps};
    const dim3 grid(static_cast<uint32_t>(q_blocks + k_blocks));
    auto go = [&](auto kernel, int groups) {
        size_t lds = kMaxHalf * sizeof(double) + tile * (a.rotary / 2) * sizeof(float2);
        if (BWD) lds = std::max(lds, groups * a.dim * sizeof(float));
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), lds, stream, n);
    };
    // whole vectors where both halves of the rotated and of the other values hold them
    const bool vec = a.rotary % (2 * V) == 0 && a.dim % (2 * V) == 0;
    const int64_t slots = vec ? a.dim / (2 * V) : (a.dim + 1) / 2;
    if (vec && slots <= 4) go(head_norm_kernel<T, V, 4, 1, BWD>, kThreads / 4);
    else if (vec && slots <= 8) go(head_norm_kernel<T, V, 8, 1, BWD>, kThreads / 8);
    else if (vec && slots <= 16) go(head_norm_kernel<T, V, 16, 1, BWD>, kThreads / 16);
    else if (vec) go(head_norm_kernel<T, V, 32, 1, BWD>, kThreads / 32);
    else if (slots <= 16) go(head_norm_kernel<T, 1, 16, 1, BWD>, kThreads / 16);
    else if (slots <= 64) go(head_norm_kernel<T, 1, 64, 1, BWD>, kThreads / 64);
    else go(head_norm_kernel<T, 1, 64, 2, BWD>, kThreads / 64);
    return hipGetLastError();
}

}  // namespace

size_t qk_norm_rotary_bwd_workspace(const HeadNormArgs &a) {
    return static_cast<size_t>(blocks_of(a, a.q_heads) + blocks_of(a, a.k_heads)) * a.dim * sizeof(float);
}

hipError_t launch_qk_norm_rotary_fwd(const HeadNormArgs &a, hipStream_t stream) {
    return a.io == IO_F32 ? launch<float, false>(a, nullptr, stream) : launch<uint16_t, false>(a, nullptr, stream);
}

hipError_t launch_qk_norm_rotary_bwd(const HeadNormArgs &a, void *workspace, hipStream_t stream) {
    const bool sums = a.dq_weight || a.dk_weight;
    void *ws = workspace;
    if (sums && !ws)
        if (const hipError_t e = scratch_alloc(&ws, qk_norm_rotary_bwd_workspace(a), stream)) return e;
    float *part = sums ? static_cast<float *>(ws) : nullptr;
    hipError_t e = a.io == IO_F32 ? launch<float, true>(a, part, stream) : launch<uint16_t, true>(a, part, stream);
    if (part && e == hipSuccess) {
        const int q_blocks = static_cast<int>(blocks_of(a, a.q_heads)), k_blocks = static_cast<int>(blocks_of(a, a.k_heads));
        hipLaunchKernelGGL(head_norm_sum_kernel, dim3(static_cast<uint32_t>((a.dim + 31) / 32), 2), dim3(1024), 0, stream, part,
                           q_blocks, a.dq_weight, part + q_blocks * a.dim, k_blocks, a.dk_weight, static_cast<int>(a.dim));
        e = hipGetLastError();
    }
    if (part && !workspace) {
        const hipError_t f = scratch_free(ws, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

}  // namespace mssm
