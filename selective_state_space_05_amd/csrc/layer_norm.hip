// layer_norm.hip -- layer norm over rows, forward and backward.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps)
//   y    = (x - mean) rstd w + b
// and, with xhat = (x - mean) rstd and e = dy w,
//   dx   = rstd (e - mean(e) - xhat mean(e xhat))
//   dw   = sum over rows of dy xhat,  db = sum over rows of dy
//
// One workgroup per row; sums in float32.
#include "device_math.h"
#include "internal.h"

namespace mssm {
namespace {

constexpr int kThreads = 256;

// Sum over the workgroup, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float *sh) {
#pragma unroll
    for (int m = 32; m >= 1; m /= 2) v += __shfl_xor(v, m);
    __syncthreads();
    if (threadIdx.x % 64 == 0) sh[threadIdx.x / 64] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) s += sh[w];
    return s;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(const T *__restrict__ x,
                                                            const float *__restrict__ weight,
                                                            const float *__restrict__ bias, float eps,
                                                            T *__restrict__ y, float *__restrict__ mean,
                                                            float *__restrict__ rstd, int dim) {
    __shared__ float sh[kThreads / 64];
    const int64_t row = blockIdx.x;
    x += row * dim;
    y += row * dim;
    float s = 0.0f;
    for (int d = threadIdx.x; d < dim; d += kThreads) s += Io<T>::load(x, d);
    const float mu = block_sum(s, sh) / dim;
    float v = 0.0f;
    for (int d = threadIdx.x; d < dim; d += kThreads) {
        const float c = Io<T>::load(x, d) - mu;
        v = fmaf(c, c, v);
    }
    const float r = 1.0f / sqrtf(block_sum(v, sh) / dim + eps);
    for (int d = threadIdx.x; d < dim; d += kThreads) {
        const float w = weight ? weight[d] : 1.0f, b = bias ? bias[d] : 0.0f;
        Io<T>::store(y, d, fmaf((Io<T>::load(x, d) - mu) * r, w, b));
    }
    if (threadIdx.x == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = r;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void norm_bwd_dx_kernel(
    const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
    const float *__restrict__ rstd, const float *__restrict__ weight, T *__restrict__ dx, int dim) {
    __shared__ float sh[kThreads / 64];
    const int64_t row = blockIdx.x;
    x += row * dim;
    dy += row * dim;
    dx += row * dim;
    const float mu = mean[row], r = rstd[row];
    float s0 = 0.0f, s1 = 0.0f;
    for (int d = threadIdx.x; d < dim; d += kThreads) {
        const float e = Io<T>::load(dy, d) * (weight ? weight[d] : 1.0f);
        s0 += e;
        s1 = fmaf(e, (Io<T>::load(x, d) - mu) * r, s1);
    }
    const float m0 = block_sum(s0, sh) / dim, m1 = block_sum(s1, sh) / dim;
    for (int d = threadIdx.x; d < dim; d += kThreads) {
        const float e = Io<T>::load(dy, d) * (weight ? weight[d] : 1.0f);
        const float xh = (Io<T>::load(x, d) - mu) * r;
        Io<T>::store(dx, d, r * (e - m0 - xh * m1));
    }
}

// Column sums over a slice of the rows: part[slice][0..dim) = dw terms,
// [dim..2 dim) = db terms.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_bwd_part_kernel(
    const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
    const float *__restrict__ rstd, float *__restrict__ part, int64_t rows, int dim) {
    const int d = blockIdx.x * kThreads + threadIdx.x;
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

__global__ __launch_bounds__(kThreads) void norm_bwd_sum_kernel(const float *__restrict__ part, int slices,
                                                                float *dweight, float *dbias, int dim) {
    const int d = blockIdx.x * kThreads + threadIdx.x;
    if (d >= dim) return;
    float dw = 0.0f, db = 0.0f;
    for (int s = 0; s < slices; ++s) {
        const float *p = part + static_cast<int64_t>(s) * 2 * dim;
        dw += p[d];
        db += p[dim + d];
    }
    if (dweight) dweight[d] = dw;
    if (dbias) dbias[d] = db;
}

template <typename T>
hipError_t fwd(const NormArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL(norm_fwd_kernel<T>, dim3(static_cast<uint32_t>(a.rows)), dim3(kThreads), 0, stream,
                       static_cast<const T *>(a.x), a.weight, a.bias, a.eps, static_cast<T *>(a.y), a.mean,
                       a.rstd, static_cast<int>(a.dim));
    return hipGetLastError();
}

int64_t slices_of(const NormArgs &a) { return a.rows < 64 ? a.rows : 64; }

template <typename T>
hipError_t bwd(const NormArgs &a, void *workspace, hipStream_t stream) {
    const int dim = static_cast<int>(a.dim);
    hipLaunchKernelGGL(norm_bwd_dx_kernel<T>, dim3(static_cast<uint32_t>(a.rows)), dim3(kThreads), 0, stream,
                       static_cast<const T *>(a.dy), static_cast<const T *>(a.x), a.mean, a.rstd, a.weight,
                       static_cast<T *>(a.dx), dim);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!a.dweight && !a.dbias)) return e;
    const int slices = static_cast<int>(slices_of(a));
    void *part = workspace;
    if (!part) e = scratch_alloc(&part, layer_norm_bwd_workspace(a), stream);
    if (e != hipSuccess) return e;
    const uint32_t cols = static_cast<uint32_t>((a.dim + kThreads - 1) / kThreads);
    hipLaunchKernelGGL(norm_bwd_part_kernel<T>, dim3(cols, slices), dim3(kThreads), 0, stream,
                       static_cast<const T *>(a.dy), static_cast<const T *>(a.x), a.mean, a.rstd,
                       static_cast<float *>(part), a.rows, dim);
    hipLaunchKernelGGL(norm_bwd_sum_kernel, dim3(cols), dim3(kThreads), 0, stream,
                       static_cast<const float *>(part), slices, a.dweight, a.dbias, dim);
    e = hipGetLastError();
    if (!workspace) {
        const hipError_t f = scratch_free(part, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

}  // namespace

size_t layer_norm_bwd_workspace(const NormArgs &a) { return static_cast<size_t>(slices_of(a)) * 2 * a.dim * sizeof(float); }

hipError_t launch_layer_norm_fwd(const NormArgs &a, hipStream_t stream) {
    return a.io == IO_F32 ? fwd<float>(a, stream) : fwd<uint16_t>(a, stream);
}

hipError_t launch_layer_norm_bwd(const NormArgs &a, void *workspace, hipStream_t stream) {
    return a.io == IO_F32 ? bwd<float>(a, workspace, stream) : bwd<uint16_t>(a, workspace, stream);
}

}  // namespace mssm
