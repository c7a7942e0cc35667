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
// pairs with each other, so nothing but the sum of squares passes between lanes.
// A token's sines and cosines are formed once for all its heads, into LDS: the
// angle in turns in float64, where 2^20 positions keep their digits, its fraction
// in float32.
#include <algorithm>

#include "device_math.h"
#include "internal.h"

namespace mssm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kMaxHalf = MSSM_MAX_HEAD_DIM / 2;

// VEC consecutive elements as floats, at any element's address.
template <int VEC>
__device__ __forceinline__ void load(const float *p, float (&f)[VEC]) {
    if constexpr (VEC == 4) {
        typedef f32x4 Any __attribute__((aligned(4)));
        const f32x4 v = *reinterpret_cast<const Any *>(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
        f[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void load(const uint16_t *p, float (&f)[VEC]) {
    if constexpr (VEC == 8) {
        typedef u32x4 Any __attribute__((aligned(2)));
        const u32x4 v = *reinterpret_cast<const Any *>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(j % 2 ? v[j / 2] & 0xffff0000u : v[j / 2] << 16);
    } else {
        f[0] = bf16_to_f32(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void store(float *p, const float (&f)[VEC]) {
    if constexpr (VEC == 4) {
        typedef f32x4 Any __attribute__((aligned(4)));
        *reinterpret_cast<Any *>(p) = f32x4{f[0], f[1], f[2], f[3]};
    } else {
        *p = f[0];
    }
}
template <int VEC>
__device__ __forceinline__ void store(uint16_t *p, const float (&f)[VEC]) {
    if constexpr (VEC == 8) {
        typedef u32x4 Any __attribute__((aligned(2)));
        typedef __bf16 b8 __attribute__((ext_vector_type(8)));
        b8 b;
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = static_cast<__bf16>(f[j]);
        *reinterpret_cast<Any *>(p) = __builtin_bit_cast(u32x4, b);
    } else {
        *p = f32_to_bf16(f[0]);
    }
}

struct HeadNorm {
    const void *q, *k, *dq, *dk;
    void *q_out, *k_out;
    const float *q_weight, *k_weight;
    const int64_t *positions;
    float *part;             // backward: column sums of every workgroup, (2, dim) each; may be null
    int64_t tokens;
    int q_heads, k_heads, dim, rotary, tile;   // tile: tokens a workgroup takes at a time
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

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int d = 1; d < G; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// G lanes a head, SLOTS slots a lane.
template <typename T, int VEC, int G, int SLOTS, bool BWD>
__global__ __launch_bounds__(kThreads) void head_norm_kernel(const HeadNorm N) {
    constexpr int GROUPS = kThreads / G;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const int half = N.rotary / 2;
    double *const rate = reinterpret_cast<double *>(smem);
    float2 *const turn = reinterpret_cast<float2 *>(rate + kMaxHalf);   // (tile, half): cos, sin
    for (int j = threadIdx.x; j < half; j += kThreads)                 // turns a position
        rate[j] = exp2(-N.log2_base * (2 * j) / N.rotary) * 0.15915494309189535;
    const int lane = threadIdx.x % G, group = threadIdx.x / G;
    float dw[2][SLOTS][2 * VEC];
    if (BWD)
        for (int which = 0; which < 2; ++which)
            for (int s = 0; s < SLOTS; ++s)
                for (int j = 0; j < 2 * VEC; ++j) dw[which][s][j] = 0.0f;

    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * N.tile; t0 < N.tokens;
         t0 += static_cast<int64_t>(gridDim.x) * N.tile) {
        const int count = static_cast<int>(min(static_cast<int64_t>(N.tile), N.tokens - t0));
        __syncthreads();
        for (int id = threadIdx.x; id < count * half; id += kThreads) {
            const double x = static_cast<double>(N.positions[t0 + id / half]) * rate[id % half];
            float s, c;
            sincospif(2.0f * static_cast<float>(x - rint(x)), &s, &c);
            turn[id] = float2{c, s};
        }
        __syncthreads();
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int heads = which ? N.k_heads : N.q_heads;
            const T *const x0 = static_cast<const T *>(which ? N.k : N.q) + t0 * heads * N.dim;
            const T *const d0 = static_cast<const T *>(which ? N.dk : N.dq) + t0 * heads * N.dim;
            T *const y0 = static_cast<T *>(which ? N.k_out : N.q_out) + t0 * heads * N.dim;
            const float *const weight = which ? N.k_weight : N.q_weight;
            float w[SLOTS][2 * VEC];
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                const Slot<VEC> at(lane + s * G, N.dim, N.rotary);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    w[s][j] = weight && at.has_a ? weight[at.a + j] : 1.0f;
                    w[s][VEC + j] = weight && at.has_b ? weight[at.b + j] : 1.0f;
                }
            }
            for (int id = group; id < count * heads; id += GROUPS) {
                const int64_t off = static_cast<int64_t>(id) * N.dim;
                const float2 *const my = turn + id / heads * half;
                float x[SLOTS][2][VEC] = {}, g[SLOTS][2][VEC] = {}, ss = 0.0f;
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    const Slot<VEC> at(lane + s * G, N.dim, N.rotary);
                    if (at.has_a) load(x0 + off + at.a, x[s][0]);
                    if (at.has_b) load(x0 + off + at.b, x[s][1]);
                    if (BWD) {
                        if (at.has_a) load(d0 + off + at.a, g[s][0]);
                        if (at.has_b) load(d0 + off + at.b, g[s][1]);
                    }
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        ss = fmaf(x[s][0][j], x[s][0][j], ss);
                        ss = fmaf(x[s][1][j], x[s][1][j], ss);
                    }
                }
                const float r = 1.0f / sqrtf(group_sum<G>(ss) / N.dim + N.eps);
                float ex = 0.0f;
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    const Slot<VEC> at(lane + s * G, N.dim, N.rotary);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float2 cs = at.angle < 0 ? float2{1.0f, 0.0f} : my[at.angle + j];
                        float &xa = x[s][0][j], &xb = x[s][1][j];
                        if (BWD) {
                            const float ga = g[s][0][j], gb = g[s][1][j];
                            const float na = fmaf(gb, cs.y, ga * cs.x), nb = fmaf(-ga, cs.y, gb * cs.x);
                            dw[which][s][j] = fmaf(na * r, xa, dw[which][s][j]);
                            dw[which][s][VEC + j] = fmaf(nb * r, xb, dw[which][s][VEC + j]);
                            g[s][0][j] = na * w[s][j];
                            g[s][1][j] = nb * w[s][VEC + j];
                            ex = fmaf(g[s][0][j], xa, ex);
                            ex = fmaf(g[s][1][j], xb, ex);
                        } else {
                            const float na = xa * r * w[s][j], nb = xb * r * w[s][VEC + j];
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
                        for (int j = 0; j < VEC; ++j) {
                            x[s][0][j] = r * fmaf(-x[s][0][j], c, g[s][0][j]);
                            x[s][1][j] = r * fmaf(-x[s][1][j], c, g[s][1][j]);
                        }
                }
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    const Slot<VEC> at(lane + s * G, N.dim, N.rotary);
                    if (at.has_a) store(y0 + off + at.a, x[s][0]);
                    if (at.has_b) store(y0 + off + at.b, x[s][1]);
                }
            }
        }
    }
    if (BWD && N.part) {
        // the groups' column sums, added in the order of the groups
        float *const sum = reinterpret_cast<float *>(smem);   // (GROUPS, dim)
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
            for (int s = 0; s < SLOTS; ++s) {
                const Slot<VEC> at(lane + s * G, N.dim, N.rotary);
                for (int j = 0; j < VEC; ++j) {
                    if (at.has_a) sum[group * N.dim + at.a + j] = dw[which][s][j];
                    if (at.has_b) sum[group * N.dim + at.b + j] = dw[which][s][VEC + j];
                }
            }
            __syncthreads();
            for (int d = threadIdx.x; d < N.dim; d += kThreads) {
                float v = 0.0f;
                for (int i = 0; i < GROUPS; ++i) v += sum[i * N.dim + d];
                N.part[(static_cast<int64_t>(blockIdx.x) * 2 + which) * N.dim + d] = v;
            }
        }
    }
}

// Adds the workgroups' column sums: a workgroup a column of dq_weight or dk_weight.
__global__ __launch_bounds__(kThreads) void head_norm_sum_kernel(const float *__restrict__ part, int parts,
                                                                 float *__restrict__ dq, float *__restrict__ dk, int dim) {
    __shared__ float sum[kThreads];
    const int d = blockIdx.x;
    float *const to = d < dim ? dq : dk;
    float v = 0.0f;
    for (int i = threadIdx.x; i < parts; i += kThreads) v += part[static_cast<int64_t>(i) * 2 * dim + d];
    sum[threadIdx.x] = v;
    for (int n = kThreads / 2; n > 0; n /= 2) {
        __syncthreads();
        if (threadIdx.x < n) sum[threadIdx.x] += sum[threadIdx.x + n];
    }
    if (threadIdx.x == 0 && to) to[d % dim] = sum[0];
}

int64_t blocks_of(const HeadNormArgs &a, int64_t tile) {
    return std::min<int64_t>((a.tokens + tile - 1) / tile, 1024);
}
int64_t tile_of(const HeadNormArgs &a) { return a.tokens >= 4096 ? 4 : 1; }

template <typename T, bool BWD>
hipError_t launch(const HeadNormArgs &a, float *part, hipStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const int64_t tile = tile_of(a);
    HeadNorm n{a.q, a.k, a.dq, a.dk, a.q_out, a.k_out, a.q_weight, a.k_weight, a.positions, part, a.tokens,
               static_cast<int>(a.q_heads), static_cast<int>(a.k_heads), static_cast<int>(a.dim),
               static_cast<int>(a.rotary), static_cast<int>(tile), log2(a.base), a.eps};
    const dim3 grid(static_cast<uint32_t>(blocks_of(a, tile)));
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
    return static_cast<size_t>(blocks_of(a, tile_of(a))) * 2 * a.dim * sizeof(float);
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
        hipLaunchKernelGGL(head_norm_sum_kernel, dim3(static_cast<uint32_t>(2 * a.dim)), dim3(kThreads), 0, stream, part,
                           static_cast<int>(blocks_of(a, tile_of(a))), a.dq_weight, a.dk_weight, static_cast<int>(a.dim));
        e = hipGetLastError();
    }
    if (part && !workspace) {
        const hipError_t f = scratch_free(ws, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

}  // namespace mssm
