// gated_recurrence.hip -- the elementwise gated linear recurrence, forward and
// backward.
//
//   log a_t = -c softplus(lam) sigmoid(r_t)
//   h_t     = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,   y_t = h_t
//
// One lane per (batch, channel) row walks the sequence; the gradient walks it
// from the end with g_t = dy_t + a_{t+1} g_{t+1}.
#include "device_math.h"
#include "internal.h"

namespace mssm {
namespace {

constexpr int kThreads = 64;

// 1 / (1 + 2^(-x log2 e)).
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-x * kLog2e));
}

// e^x - 1 for x <= 0.  Above -0.35 the Taylor series (x^8 / 8! < 6e-9
// relative), below it 2^y - 1, where the subtraction loses at most a factor 3.4.
__device__ __forceinline__ float expm1_neg(float x) {
    float p = 1.0f / 5040.0f;
    p = fmaf(p, x, 1.0f / 720.0f);
    p = fmaf(p, x, 1.0f / 120.0f);
    p = fmaf(p, x, 1.0f / 24.0f);
    p = fmaf(p, x, 1.0f / 6.0f);
    p = fmaf(p, x, 0.5f);
    p = fmaf(p * x, x, x);
    return x > -0.35f ? p : fast_exp2(x * kLog2e) - 1.0f;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void recurrence_fwd_kernel(const T *__restrict__ x,
                                                                  const T *__restrict__ r,
                                                                  const T *__restrict__ i,
                                                                  const float *__restrict__ lam, float scale,
                                                                  const float *h0, T *__restrict__ y,
                                                                  float *h_last, int64_t rows, int64_t L,
                                                                  int64_t dim) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (row >= rows) return;
    const int64_t b = row / dim, d = row - b * dim;
    const float rate = -scale * softplus_libm(lam[d]);
    float h = h0 ? h0[row] : 0.0f;
    int64_t at = b * L * dim + d;
    for (int64_t t = 0; t < L; ++t, at += dim) {
        const float p = expm1_neg(rate * sigmoid(Io<T>::load(r, at)));
        const float m = sqrtf(-p * (2.0f + p));
        h = fmaf(1.0f + p, h, m * sigmoid(Io<T>::load(i, at)) * Io<T>::load(x, at));
        Io<T>::store(y, at, h);
    }
    if (h_last) h_last[row] = h;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void recurrence_bwd_kernel(
    const T *__restrict__ x, const T *__restrict__ r, const T *__restrict__ i,
    const float *__restrict__ lam, float scale, const float *__restrict__ h0, const T *__restrict__ y,
    const T *__restrict__ dy, const float *__restrict__ dh_last, T *__restrict__ dx, T *__restrict__ dr,
    T *__restrict__ di, float *__restrict__ part, float *__restrict__ dh0, int64_t rows, int64_t L,
    int64_t dim) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (row >= rows) return;
    const int64_t b = row / dim, d = row - b * dim;
    const float rate = -scale * softplus_libm(lam[d]);
    const float start = h0 ? h0[row] : 0.0f;
    float carry = dh_last ? dh_last[row] : 0.0f;   // a_{t+1} g_{t+1}
    float sum = 0.0f;
    for (int64_t t = L - 1; t >= 0; --t) {
        const int64_t at = (b * L + t) * dim + d;
        const float sr = sigmoid(Io<T>::load(r, at)), si = sigmoid(Io<T>::load(i, at));
        const float xv = Io<T>::load(x, at);
        const float la = rate * sr;
        const float p = expm1_neg(la), a = 1.0f + p;
        const float m = sqrtf(-p * (2.0f + p));
        const float q = m > 0.0f ? la / m : 0.0f;      // -> 0 with la
        const float before = t > 0 ? Io<T>::load(y, at - dim) : start;
        const float g = Io<T>::load(dy, at) + carry;
        const float ga = g * a;
        const float w = ga * (before * la - a * (si * xv) * q);
        Io<T>::store(dx, at, g * m * si);
        Io<T>::store(di, at, g * m * si * xv * (1.0f - si));
        Io<T>::store(dr, at, w * (1.0f - sr));
        sum += w;
        carry = ga;
    }
    if (part) part[row] = sum;
    if (dh0) dh0[row] = carry;
}

// dlam = sum of w over batches and steps, times sigmoid(lam) / softplus(lam)
// (which tends to 1 as lam falls).
__global__ __launch_bounds__(kThreads) void recurrence_dlam_kernel(const float *__restrict__ part,
                                                                   const float *__restrict__ lam,
                                                                   float *__restrict__ dlam, int64_t parts,
                                                                   int64_t dim) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (d >= dim) return;
    float s = 0.0f;
    for (int64_t k = 0; k < parts; ++k) s += part[k * dim + d];
    const float sp = softplus_libm(lam[d]), sg = 1.0f / (1.0f + expf(-lam[d]));
    dlam[d] = s * (sp > 0.0f ? sg / sp : 1.0f);
}

template <typename T>
hipError_t fwd(const RecurrenceArgs &a, hipStream_t stream) {
    const int64_t rows = a.batch * a.dim;
    hipLaunchKernelGGL(recurrence_fwd_kernel<T>, dim3(static_cast<uint32_t>((rows + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, stream, static_cast<const T *>(a.x), static_cast<const T *>(a.r),
                       static_cast<const T *>(a.i), a.lam, a.scale, a.h0, static_cast<T *>(a.y), a.h_last,
                       rows, a.L, a.dim);
    return hipGetLastError();
}

template <typename T>
hipError_t bwd(const RecurrenceArgs &a, hipStream_t stream) {
    const int64_t rows = a.batch * a.dim;
    void *part = nullptr;
    hipError_t e = hipSuccess;
    if (a.dlam) e = scratch_alloc(&part, static_cast<size_t>(rows) * sizeof(float), stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(recurrence_bwd_kernel<T>, dim3(static_cast<uint32_t>((rows + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, stream, static_cast<const T *>(a.x), static_cast<const T *>(a.r),
                       static_cast<const T *>(a.i), a.lam, a.scale, a.h0, static_cast<const T *>(a.y),
                       static_cast<const T *>(a.dy), a.dh_last, static_cast<T *>(a.dx),
                       static_cast<T *>(a.dr), static_cast<T *>(a.di), static_cast<float *>(part), a.dh0,
                       rows, a.L, a.dim);
    e = hipGetLastError();
    if (e == hipSuccess && a.dlam) {
        hipLaunchKernelGGL(recurrence_dlam_kernel, dim3(static_cast<uint32_t>((a.dim + kThreads - 1) / kThreads)),
                           dim3(kThreads), 0, stream, static_cast<const float *>(part), a.lam, a.dlam, a.batch,
                           a.dim);
        e = hipGetLastError();
    }
    if (part) {
        const hipError_t f = scratch_free(part, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

}  // namespace

bool gated_recurrence_supported(const RecurrenceArgs &a) {
    return a.batch * a.dim < (int64_t(1) << 31);   // one lane a row, 64 a workgroup
}

hipError_t launch_gated_recurrence_fwd(const RecurrenceArgs &a, hipStream_t stream) {
    return a.io == IO_F32 ? fwd<float>(a, stream) : fwd<uint16_t>(a, stream);
}

hipError_t launch_gated_recurrence_bwd(const RecurrenceArgs &a, hipStream_t stream) {
    return a.io == IO_F32 ? bwd<float>(a, stream) : bwd<uint16_t>(a, stream);
}

}  // namespace mssm
