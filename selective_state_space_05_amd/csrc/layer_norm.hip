// layer_norm.hip -- layer norm over rows, forward and backward.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps)
//   y    = (x - mean) rstd w + b
// and, with xhat = (x - mean) rstd and e = dy w,
//   dx   = rstd (e - mean(e) - xhat mean(e xhat))
//   dw   = sum over rows of dy xhat,  db = sum over rows of dy
//
// Both are bound by memory: every operand is read once and every result
// written once, so a row has to stay on chip between its sums and its result.
// It stays in registers: a group of G lanes holds a row as K vectors of 16
// bytes per lane, forms the sums with lane swaps (and, for rows of several
// waves, one exchange through LDS per sum), and the next row of the group is
// already under way meanwhile.  The weights, and in the backward the column
// sums dw and db, are held in registers too, in the lanes of their columns;
// the column sums leave once per workgroup and a second launch adds them up.
// All sums are float32, in an order that depends on the sizes alone.  Measured in
// bfloat16 at 8192 x 2560: forward 15.4 us (5.5 TB/s), backward 29.6 us (4.3 TB/s,
// of which the second launch takes 4 us); 64 rows forward 3.7 us.
//
// Rows begin at any element: the vectors are loaded and stored unaligned, and
// the last vector of a row is moved back to end with the row, its elements
// that the lane before holds too being masked out of the sums.
#include <algorithm>
#include <type_traits>

#include "device_math.h"
#include "internal.h"

namespace mssm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// VEC consecutive elements as they lie in memory.
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

// How rows lie over lanes: K vectors of VEC elements for each of G lanes.  The
// first FULL of them hold a whole vector in every lane, whatever the row's
// length for which this shape is taken.
template <int VEC_, int K_, int FULL_, int G_>
struct Shape {
    static constexpr int VEC = VEC_, K = K_, FULL = FULL_, G = G_;
    static constexpr int kWaves = (G + 63) / 64;   // of a row
};

// Position of a lane's vector k in its row, and how many of the vector's
// elements the lane before it holds (VEC or more: all).
template <typename S>
struct Place {
    int at, skip;
    __device__ __forceinline__ Place(int k, int lane, int dim) {
        const int want = (k * S::G + lane) * S::VEC;
        at = k < S::FULL ? want : min(want, dim - S::VEC);
        skip = want - at;
    }
};

// Which of the workgroup's rows a thread's lanes hold; known to be one for a wave.
template <typename S>
__device__ __forceinline__ int group_of() {
    const int g = threadIdx.x / S::G;
    return S::G < 64 ? g : __builtin_amdgcn_readfirstlane(g);
}

// Sums of N values over a row's lanes, the same in all of them.  sh: N floats per
// wave of the row, not written again until the lanes have met at another barrier.
template <typename S, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float *sh) {
    constexpr int G = S::G;
    auto dpp = [](float x, auto ctrl) {
        return __builtin_bit_cast(
            float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x = v[i];
        x += dpp(x, std::integral_constant<int, 0xb1>());    // quad_perm 1 0 3 2
        x += dpp(x, std::integral_constant<int, 0x4e>());    // quad_perm 2 3 0 1
        x += dpp(x, std::integral_constant<int, 0x141>());   // halves of 8 mirrored
        if constexpr (G >= 16) x += dpp(x, std::integral_constant<int, 0x140>());   // rows of 16 mirrored
        if constexpr (G >= 32) {
            const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
            x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        }
        if constexpr (G >= 64) {
            const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
            x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        }
        v[i] = x;
        if constexpr (S::kWaves > 1)
            if (threadIdx.x % 64 == 0) sh[i * S::kWaves + threadIdx.x / 64] = x;
    }
    if constexpr (S::kWaves > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = sh[i * S::kWaves];
#pragma unroll
            for (int w = 1; w < S::kWaves; ++w) v[i] += sh[i * S::kWaves + w];
        }
    }
}
template <typename S>
__device__ __forceinline__ float row_sum(float v, float *sh) {
    float x[1] = {v};
    row_sums<S, 1>(x, sh);
    return x[0];
}

// Values of the lane's columns, `other` where there is no vector.
template <typename S>
__device__ __forceinline__ void load_columns(const float *__restrict__ p, float other, int lane, int dim,
                                             float (&f)[S::K][S::VEC]) {
#pragma unroll
    for (int k = 0; k < S::K; ++k) {
        const Place<S> place(k, lane, dim);
#pragma unroll
        for (int e = 0; e < S::VEC; ++e) f[k][e] = p ? p[place.at + e] : other;
    }
}

template <typename T, typename S>
__device__ __forceinline__ void load_row(const T *__restrict__ p, int lane, int dim, Vec<T, S::VEC> (&v)[S::K]) {
#pragma unroll
    for (int k = 0; k < S::K; ++k) v[k].load(p + Place<S>(k, lane, dim).at);
}

// ---- forward -----------------------------------------------------------------

template <typename T, typename S>
struct NormFwd {
    static constexpr int kThreads = S::G > 256 ? S::G : 256;
    static constexpr int kRows = kThreads / S::G;   // of a workgroup at once
    struct Held {
        Vec<T, S::VEC> x[S::K];
    };
    const T *__restrict__ x;
    const float *__restrict__ weight, *__restrict__ bias;
    float eps;
    T *__restrict__ y;
    float *__restrict__ mean, *__restrict__ rstd;
    int64_t rows;
    int dim;

    __device__ __forceinline__ void load(int64_t row, int lane, Held &h) const {
        load_row<T, S>(x + (row < rows ? row : rows - 1) * dim, lane, dim, h.x);
    }
    __device__ __forceinline__ void finish(int64_t row, int lane, const Held &h, const float (&w)[S::K][S::VEC],
                                           const float (&b)[S::K][S::VEC], float *sh) const {
        float part[S::K];
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            part[k] = 0.0f;
            const Place<S> place(k, lane, dim);
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) part[k] += k < S::FULL || e >= place.skip ? h.x[k].get(e) : 0.0f;
        }
        float s = part[0];
#pragma unroll
        for (int k = 1; k < S::K; ++k) s += part[k];
        const float mu = row_sum<S>(s, sh) / dim;
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            part[k] = 0.0f;
            const Place<S> place(k, lane, dim);
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) {
                const float c = k < S::FULL || e >= place.skip ? h.x[k].get(e) - mu : 0.0f;
                part[k] = fmaf(c, c, part[k]);
            }
        }
        s = part[0];
#pragma unroll
        for (int k = 1; k < S::K; ++k) s += part[k];
        const float r = 1.0f / sqrtf(row_sum<S>(s, sh + S::kWaves) / dim + eps);
        if (row >= rows) return;
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            const Place<S> place(k, lane, dim);
            float f[S::VEC];
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) f[e] = fmaf((h.x[k].get(e) - mu) * r, w[k][e], b[k][e]);
            if (k < S::FULL || place.skip < S::VEC) Vec<T, S::VEC>::store(y + row * dim + place.at, f);
        }
        if (lane == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = r;
        }
    }
};

template <typename T, typename S>
__global__ __launch_bounds__((NormFwd<T, S>::kThreads)) void norm_fwd_kernel(NormFwd<T, S> n) {
    __shared__ float sh[2 * S::kWaves];
    const int lane = threadIdx.x % S::G, group = group_of<S>();
    const int64_t step = static_cast<int64_t>(gridDim.x) * n.kRows;
    int64_t base = static_cast<int64_t>(blockIdx.x) * n.kRows;
    typename NormFwd<T, S>::Held a, b;
    n.load(base + group, lane, a);
    float w[S::K][S::VEC], c[S::K][S::VEC];
    load_columns<S>(n.weight, 1.0f, lane, n.dim, w);
    load_columns<S>(n.bias, 0.0f, lane, n.dim, c);
    for (;;) {
        n.load(base + step + group, lane, b);
        n.finish(base + group, lane, a, w, c, sh);
        base += step;
        if (base >= n.rows) return;
        n.load(base + step + group, lane, a);
        n.finish(base + group, lane, b, w, c, sh);
        base += step;
        if (base >= n.rows) return;
    }
}

// ---- backward ----------------------------------------------------------------

// Columns in LDS as the lanes hold them: four floats per lane side by side (one,
// where a lane's vector is one).
template <typename S>
struct Columns {
    static constexpr int Q = S::VEC < 4 ? S::VEC : 4, kFloats = S::K * S::VEC * S::G;
    typedef float Four __attribute__((ext_vector_type(Q)));
    __device__ __forceinline__ static Four &at(float *lds, int k, int q, int lane) {
        return reinterpret_cast<Four *>(lds)[(k * (S::VEC / Q) + q) * S::G + lane];
    }
    __device__ __forceinline__ static void get(const float *lds, int k, int lane, float (&f)[S::VEC]) {
#pragma unroll
        for (int q = 0; q < S::VEC / Q; ++q) {
            const Four v = at(const_cast<float *>(lds), k, q, lane);
#pragma unroll
            for (int e = 0; e < Q; ++e) f[q * Q + e] = v[e];
        }
    }
    __device__ __forceinline__ static void put(float *lds, int k, int lane, const float (&f)[S::VEC]) {
#pragma unroll
        for (int q = 0; q < S::VEC / Q; ++q) {
            Four v;
#pragma unroll
            for (int e = 0; e < Q; ++e) v[e] = f[q * Q + e];
            at(lds, k, q, lane) = v;
        }
    }
};

template <typename T, typename S>
struct NormBwd {
    static constexpr int kThreads = S::G > 64 ? S::G : 512;
    static constexpr int kRows = kThreads / S::G;   // of a workgroup at once
    struct Held {
        Vec<T, S::VEC> x[S::K], dy[S::K];
        float mu, r;
    };
    const T *__restrict__ dy;
    const T *__restrict__ x;
    const float *__restrict__ mean, *__restrict__ rstd, *__restrict__ weight;
    T *__restrict__ dx;
    float *__restrict__ part;   // (workgroups, 2 dim): dw, db of a workgroup's rows; may be null
    int64_t rows;
    int dim;

    __device__ __forceinline__ void load(int64_t row, int lane, Held &h) const {
        row = row < rows ? row : rows - 1;   // the last one again where none is left
        int none = 0;
        asm("" : "+v"(none));   // as vector loads: a scalar one would be waited for with the next LDS read
        h.mu = mean[row + none];
        h.r = rstd[row + none];
        load_row<T, S>(x + row * dim, lane, dim, h.x);
        load_row<T, S>(dy + row * dim, lane, dim, h.dy);
    }
    // Finishes a row and, with RELOAD, loads the next into the registers that it leaves.
    template <bool RELOAD>
    __device__ __forceinline__ void finish(int64_t row, int64_t step, int lane, Held &h, const float *weights,
                                           float (&dw)[S::K][S::VEC], float (&db)[S::K][S::VEC], float *sh) const {
        // the weights are read anew for every row: held, they would not leave room for the next row
        asm volatile("" ::: "memory");
        float p0[S::K], p1[S::K];
        const bool there = S::G >= 64 || row < rows;
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            p0[k] = p1[k] = 0.0f;
            const Place<S> place(k, lane, dim);
            float w[S::VEC];
            Columns<S>::get(weights, k, lane, w);
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) {
                const float xh = (h.x[k].get(e) - h.mu) * h.r, g = h.dy[k].get(e), gw = g * w[e];
                const bool own = k < S::FULL || e >= place.skip;
                p0[k] += own ? gw : 0.0f;
                p1[k] = own ? fmaf(gw, xh, p1[k]) : p1[k];
                dw[k][e] = there ? fmaf(g, xh, dw[k][e]) : dw[k][e];
                db[k][e] += there ? g : 0.0f;
            }
            __builtin_amdgcn_sched_barrier(0);   // one vector after the other: fewer registers
        }
        float s[2] = {p0[0], p1[0]};
#pragma unroll
        for (int k = 1; k < S::K; ++k) s[0] += p0[k], s[1] += p1[k];
        row_sums<S, 2>(s, sh);
        const float m0 = s[0] / dim, m1 = s[1] / dim;
        // from here on x and dy are unpacked again, not kept as floats meanwhile
#pragma unroll
        for (int k = 0; k < S::K; ++k) asm volatile("" : "+v"(h.x[k].v), "+v"(h.dy[k].v));
        asm volatile("" ::: "memory");
        const int64_t next = row + step < rows ? row + step : rows - 1;   // the last one again where none is left
        int none = 0;
        asm("" : "+v"(none));   // as vector loads: a scalar one would be waited for with the next LDS read
        const float mu = h.mu, r = h.r;
        if (RELOAD) {
            h.mu = mean[next + none];
            h.r = rstd[next + none];
        }
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
            const Place<S> place(k, lane, dim);
            float f[S::VEC], w[S::VEC];
            Columns<S>::get(weights, k, lane, w);
#pragma unroll
            for (int e = 0; e < S::VEC; ++e) {
                const float xh = (h.x[k].get(e) - mu) * r;
                f[e] = r * (h.dy[k].get(e) * w[e] - m0 - xh * m1);
            }
            if (there && (k < S::FULL || place.skip < S::VEC)) Vec<T, S::VEC>::store(dx + row * dim + place.at, f);
            if (RELOAD) {
                h.x[k].load(x + next * dim + place.at);
                h.dy[k].load(dy + next * dim + place.at);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // Adds the column sums of the workgroup's rows and writes them out.
    __device__ __forceinline__ void write_sums(int lane, float (&f)[S::K][S::VEC], float *out, float *lds) const {
        using C = Columns<S>;
        constexpr int kHolders = kThreads / 64 / S::kWaves;   // waves that hold the same columns
        float *mine = lds + group_of<S>() / (S::G < 64 ? 64 / S::G : 1) * C::kFloats;
#pragma unroll
        for (int k = 0; k < S::K; ++k) {
#pragma unroll
            for (int e = 0; e < S::VEC; ++e)
#pragma unroll
                for (int m = S::G; m < 64; m *= 2) f[k][e] += __shfl_xor(f[k][e], m);
            if (threadIdx.x % 64 < S::G) C::put(mine, k, lane, f[k]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < C::kFloats; i += kThreads) {
            float v = lds[i];
#pragma unroll
            for (int h = 1; h < kHolders; ++h) v += lds[h * C::kFloats + i];
            const int slot = i / C::Q, k = slot / (S::VEC / C::Q * S::G), q = slot / S::G % (S::VEC / C::Q);
            const Place<S> place(k, slot % S::G, dim);
            const int e = q * C::Q + i % C::Q;
            if (e >= place.skip) out[place.at + e] = v;
        }
    }
};

template <typename T, typename S>
__global__ __launch_bounds__((NormBwd<T, S>::kThreads)) void norm_bwd_kernel(NormBwd<T, S> n) {
    extern __shared__ __align__(16) float lds[];   // weights; then the waves' column sums
    __shared__ float sh[4 * S::kWaves];
    const int lane = threadIdx.x % S::G, group = group_of<S>();
    // a workgroup's groups take rows far apart, so that few rows still reach every workgroup
    const int64_t step = static_cast<int64_t>(gridDim.x) * n.kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) + static_cast<int64_t>(gridDim.x) * group;
    constexpr int kSlots = (S::K * S::G + n.kThreads - 1) / n.kThreads;
    float w[kSlots][S::VEC];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        const int i = s * n.kThreads + threadIdx.x;
        const Place<S> place(i / S::G, i % S::G, n.dim);
#pragma unroll
        for (int e = 0; e < S::VEC; ++e) w[s][e] = n.weight && i < S::K * S::G ? n.weight[place.at + e] : 1.0f;
    }
    typename NormBwd<T, S>::Held a;
    n.load(row, lane, a);
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        const int i = s * n.kThreads + threadIdx.x;
        if (i < S::K * S::G) Columns<S>::put(lds, i / S::G, i % S::G, w[s]);
    }
    __syncthreads();
    // what the first lane group of the wave has left decides for the wave
    const int64_t lead = row - static_cast<int64_t>(gridDim.x) * (S::G < 64 ? threadIdx.x % 64 / S::G : 0);
    int left = __builtin_amdgcn_readfirstlane(static_cast<int>(n.rows - lead));
    const int stride = static_cast<int>(step);
    float dw[S::K][S::VEC] = {}, db[S::K][S::VEC] = {};
    if constexpr (S::G == 256) {
        // the waves of a row wait for one another: the next row comes in meanwhile
        // (4096 x 8192 in bfloat16 51 us against 59 us; 16 waves have no registers for it)
        typename NormBwd<T, S>::Held b;
        while (left > 0) {
            n.load(row + step, lane, b);
            n.template finish<false>(row, step, lane, a, lds, dw, db, sh);
            row += step;
            if ((left -= stride) <= 0) break;
            n.load(row + step, lane, a);
            n.template finish<false>(row, step, lane, b, lds, dw, db, sh + 2 * S::kWaves);
            row += step;
            left -= stride;
        }
    } else {
        for (int k = 0; left > 0; left -= stride, row += step, k ^= 1)
            n.template finish<true>(row, step, lane, a, lds, dw, db, sh + 2 * S::kWaves * k);
    }
    if (!n.part) return;
    __syncthreads();
    float *out = n.part + static_cast<int64_t>(blockIdx.x) * 2 * n.dim;
    n.write_sums(lane, dw, out, lds);
    __syncthreads();
    n.write_sums(lane, db, out + n.dim, lds);
}

// Adds the workgroups' column sums: 64 columns a workgroup, 16 slices.
constexpr int kSumSlices = 16;
__global__ __launch_bounds__(64 * kSumSlices) void norm_sum_kernel(const float *__restrict__ part, int parts,
                                                                   float *dweight, float *dbias, int dim) {
    __shared__ float sh[kSumSlices][64];
    const int lane = threadIdx.x % 64, slice = threadIdx.x / 64;
    const int64_t d = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 64 + lane;
    float v = 0.0f;
    if (d < 2 * static_cast<int64_t>(dim)) {
        constexpr int kAhead = 8;   // loads under way at a time
        for (int s = slice; s < parts; s += kAhead * kSumSlices) {
            float f[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                f[u] = part[static_cast<int64_t>(min(s + u * kSumSlices, parts - 1)) * 2 * dim + d];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) v += s + u * kSumSlices < parts ? f[u] : 0.0f;
        }
    }
    sh[slice][lane] = v;
    __syncthreads();
    if (slice > 0 || d >= 2 * static_cast<int64_t>(dim)) return;
#pragma unroll
    for (int s = 1; s < kSumSlices; ++s) v += sh[s][lane];
    float *out = d < dim ? dweight : dbias;
    if (out) out[d < dim ? d : d - dim] = v;
}

// ---- rows that no group holds --------------------------------------------------
//
// A workgroup goes over the row once per sum and once for the result.

constexpr int kWideThreads = 1024;
using Wide = Shape<1, 1, 0, kWideThreads>;

template <typename T>
__global__ __launch_bounds__(kWideThreads) void norm_wide_fwd_kernel(const T *__restrict__ x,
                                                                     const float *__restrict__ weight,
                                                                     const float *__restrict__ bias, float eps,
                                                                     T *__restrict__ y, float *__restrict__ mean,
                                                                     float *__restrict__ rstd, int dim) {
    __shared__ float sh[2 * Wide::kWaves];
    const int64_t row = blockIdx.x;
    x += row * dim;
    y += row * dim;
    float s = 0.0f;
    for (int64_t d = threadIdx.x; d < dim; d += kWideThreads) s += Io<T>::load(x, d);
    const float mu = row_sum<Wide>(s, sh) / dim;
    float v = 0.0f;
    for (int64_t d = threadIdx.x; d < dim; d += kWideThreads) {
        const float c = Io<T>::load(x, d) - mu;
        v = fmaf(c, c, v);
    }
    const float r = 1.0f / sqrtf(row_sum<Wide>(v, sh + Wide::kWaves) / dim + eps);
    for (int64_t d = threadIdx.x; d < dim; d += kWideThreads) {
        const float w = weight ? weight[d] : 1.0f, b = bias ? bias[d] : 0.0f;
        Io<T>::store(y, d, fmaf((Io<T>::load(x, d) - mu) * r, w, b));
    }
    if (threadIdx.x == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = r;
    }
}

template <typename T>
__global__ __launch_bounds__(kWideThreads) void norm_wide_dx_kernel(
    const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
    const float *__restrict__ rstd, const float *__restrict__ weight, T *__restrict__ dx, int dim) {
    __shared__ float sh[2 * Wide::kWaves];
    const int64_t row = blockIdx.x;
    x += row * dim;
    dy += row * dim;
    dx += row * dim;
    const float mu = mean[row], r = rstd[row];
    float s0 = 0.0f, s1 = 0.0f;
    for (int64_t d = threadIdx.x; d < dim; d += kWideThreads) {
        const float e = Io<T>::load(dy, d) * (weight ? weight[d] : 1.0f);
        s0 += e;
        s1 = fmaf(e, (Io<T>::load(x, d) - mu) * r, s1);
    }
    const float m0 = row_sum<Wide>(s0, sh) / dim, m1 = row_sum<Wide>(s1, sh + Wide::kWaves) / dim;
    for (int64_t d = threadIdx.x; d < dim; d += kWideThreads) {
        const float e = Io<T>::load(dy, d) * (weight ? weight[d] : 1.0f);
        const float xh = (Io<T>::load(x, d) - mu) * r;
        Io<T>::store(dx, d, r * (e - m0 - xh * m1));
    }
}

// Column sums of every gridDim.y-th row.
template <typename T>
__global__ __launch_bounds__(256) void norm_wide_part_kernel(
    const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
    const float *__restrict__ rstd, float *__restrict__ part, int64_t rows, int dim) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (d >= dim) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        const float g = Io<T>::load(dy, row * dim + d);
        dw = fmaf(g, (Io<T>::load(x, row * dim + d) - mean[row]) * rstd[row], dw);
        db += g;
    }
    float *p = part + static_cast<int64_t>(blockIdx.y) * 2 * dim;
    p[d] = dw;
    p[dim + d] = db;
}

// ---- launches ------------------------------------------------------------------

// The longest rows that registers hold.  The backward of 16 waves a row has no
// registers for 24 elements a lane with their column sums (1500 x 24000 in
// bfloat16 141 us, going over the rows again 125 us; forward 29 us and 84 us).
constexpr int64_t kMostHeldFwd = 24576, kMostHeldBwd = 16384;

// Calls f with the shape for rows of `dim` elements; false if there is none.
// A lane holds 8 elements, or as many as keep a row within one wave up to 40
// (the float32 backward, two vectors for one, 32: 8192 x 2560 47 us against 58 us),
// above that within 4 waves, above that within 16 waves up to 16 or, forward, 24
// (a workgroup of 16 waves leaves each half the registers).  Below 8 elements a
// lane holds one.
template <typename T, bool BWD, typename F>
bool with_shape(int64_t dim, F f) {
    constexpr int V = 16 / sizeof(T), U = 8 / V;   // elements of a vector, vectors of 8 elements
    constexpr bool kLong = !(BWD && sizeof(T) == 4);
    if (dim < 8) f(Shape<1, 1, 0, 8>());
    else if (dim <= 64) f(Shape<V, U, 0, 8>());
    else if (dim <= 128) f(Shape<V, U, 0, 16>());
    else if (dim <= 256) f(Shape<V, U, 0, 32>());
    else if (dim <= 512) f(Shape<V, U, 0, 64>());
    else if (dim <= 1024) f(Shape<V, 2 * U, U, 64>());
    else if (dim <= 1536) f(Shape<V, 3 * U, 2 * U, 64>());
    else if (dim <= 2048) f(Shape<V, 4 * U, 3 * U, 64>());
    else if (dim <= (kLong ? 2560 : 2048)) {
        if constexpr (kLong) f(Shape<V, 5 * U, 4 * U, 64>());
    }
    else if (dim <= 4096) f(Shape<V, 2 * U, U, 256>());
    else if (dim <= 6144) f(Shape<V, 3 * U, 2 * U, 256>());
    else if (dim <= 8192) f(Shape<V, 4 * U, 3 * U, 256>());
    else if (dim <= 10240) f(Shape<V, 5 * U, 4 * U, 256>());
    else if (dim <= kMostHeldBwd) f(Shape<V, 2 * U, U, 1024>());
    else {
        if constexpr (!BWD)
            if (dim <= kMostHeldFwd) {
                f(Shape<V, 3 * U, 2 * U, 1024>());
                return true;
            }
        return false;
    }
    return true;
}

template <typename T>
hipError_t fwd(const NormArgs &a, hipStream_t stream) {
    const int dim = static_cast<int>(a.dim);
    const bool held = with_shape<T, false>(a.dim, [&](auto shape) {
        using S = decltype(shape);
        using N = NormFwd<T, S>;
        const N n{static_cast<const T *>(a.x), a.weight, a.bias, a.eps, static_cast<T *>(a.y), a.mean, a.rstd, a.rows, dim};
        // As many workgroups as run at once, each with the same number of rows in turn:
        // 4 waves on a SIMD, 2 where a lane holds 40 elements.  Weights are then read
        // once for several rows: 8192 x 2560 in bfloat16 takes 15.4 us with 2 rows a
        // wave and more, 20 us with one.
        constexpr int64_t most = (S::K * S::VEC > 32 ? 2048 : 4096) * 64 / N::kThreads;
        const int64_t blocks = (a.rows + N::kRows - 1) / N::kRows, each = (blocks + most - 1) / most;
        hipLaunchKernelGGL((norm_fwd_kernel<T, S>), dim3(static_cast<uint32_t>((blocks + each - 1) / each)),
                           dim3(N::kThreads), 0, stream, n);
    });
    if (!held)
        hipLaunchKernelGGL(norm_wide_fwd_kernel<T>, dim3(static_cast<uint32_t>(a.rows)), dim3(kWideThreads), 0, stream,
                           static_cast<const T *>(a.x), a.weight, a.bias, a.eps, static_cast<T *>(a.y), a.mean,
                           a.rstd, dim);
    return hipGetLastError();
}

// Partial column sums of the backward, one per workgroup, one workgroup per
// compute unit: with two, the column sums cost more than the second hides
// (8192 x 2560 in bfloat16: 43 us against 33 us).  Slices of wide rows.
int64_t parts_of(const NormArgs &a) { return std::min<int64_t>(a.rows, a.dim > kMostHeldBwd ? 64 : 256); }

template <typename T>
hipError_t bwd(const NormArgs &a, void *workspace, hipStream_t stream) {
    const int dim = static_cast<int>(a.dim), parts = static_cast<int>(parts_of(a));
    const bool sums = a.dweight || a.dbias;
    void *ws = workspace;
    if (sums && !ws)
        if (const hipError_t e = scratch_alloc(&ws, layer_norm_bwd_workspace(a), stream)) return e;
    float *part = sums ? static_cast<float *>(ws) : nullptr;
    const T *dy = static_cast<const T *>(a.dy), *x = static_cast<const T *>(a.x);
    T *dx = static_cast<T *>(a.dx);
    hipError_t e = hipSuccess;
    const bool held = with_shape<T, true>(a.dim, [&](auto shape) {
        using S = decltype(shape);
        using N = NormBwd<T, S>;
        const N n{dy, x, a.mean, a.rstd, a.weight, dx, part, a.rows, dim};
        constexpr int lds = N::kThreads / 64 / S::kWaves * Columns<S>::kFloats * 4;
        if (lds > 65536)
            e = hipFuncSetAttribute(reinterpret_cast<const void *>(norm_bwd_kernel<T, S>),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e == hipSuccess)
            hipLaunchKernelGGL((norm_bwd_kernel<T, S>), dim3(parts), dim3(N::kThreads), lds, stream, n);
    });
    if (!held) {
        hipLaunchKernelGGL(norm_wide_dx_kernel<T>, dim3(static_cast<uint32_t>(a.rows)), dim3(kWideThreads), 0, stream,
                           dy, x, a.mean, a.rstd, a.weight, dx, dim);
        if (part)
            hipLaunchKernelGGL(norm_wide_part_kernel<T>, dim3(static_cast<uint32_t>((a.dim + 255) / 256), parts),
                               dim3(256), 0, stream, dy, x, a.mean, a.rstd, part, a.rows, dim);
    }
    if (part && e == hipSuccess) {
        // one dimension of a grid holds less than 2^32 threads
        const int64_t blocks = (2 * a.dim + 63) / 64, x = std::min<int64_t>(blocks, int64_t(1) << 20);
        hipLaunchKernelGGL(norm_sum_kernel, dim3(static_cast<uint32_t>(x), static_cast<uint32_t>((blocks + x - 1) / x)),
                           dim3(64 * kSumSlices), 0, stream, part, parts, a.dweight, a.dbias, dim);
    }
    if (e == hipSuccess) e = hipGetLastError();
    if (part && !workspace) {
        const hipError_t f = scratch_free(ws, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

}  // namespace

size_t layer_norm_bwd_workspace(const NormArgs &a) { return static_cast<size_t>(parts_of(a)) * 2 * a.dim * sizeof(float); }

hipError_t launch_layer_norm_fwd(const NormArgs &a, hipStream_t stream) {
    return a.io == IO_F32 ? fwd<float>(a, stream) : fwd<uint16_t>(a, stream);
}

hipError_t launch_layer_norm_bwd(const NormArgs &a, void *workspace, hipStream_t stream) {
    return a.io == IO_F32 ? bwd<float>(a, workspace, stream) : bwd<uint16_t>(a, workspace, stream);
}

}  // namespace mssm
