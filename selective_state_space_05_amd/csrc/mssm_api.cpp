// mssm_api.cpp -- the C ABI of libmssm (declared in include/mssm.h):
// argument validation, kernel-variant choice and launch on the caller's
// stream.  Validation runs before any HIP call, so every error path can be
// exercised without a GPU.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <string>

#include "internal.h"
#include "mssm.h"
#include "mssm_probes.h"

namespace {

thread_local std::string g_last_error;
thread_local mssm_variant g_forced = MSSM_VARIANT_AUTO;
thread_local mssm_variant g_last_variant = MSSM_VARIANT_AUTO;

mssm_status fail(mssm_status s, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return s;
}

mssm_status hip_fail(hipError_t e, const char *what) {
    if (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation)
        return fail(MSSM_ERR_ALLOC, "%s: %s (%d)", what, hipGetErrorString(e), static_cast<int>(e));
    return fail(MSSM_ERR_HIP, "%s: %s (%d)", what, hipGetErrorString(e), static_cast<int>(e));
}

bool mul_ok(int64_t a, int64_t b, int64_t *out) {
    return !__builtin_mul_overflow(a, b, out);
}

// Byte range [p, p + n) of one operand, for the overlap check.
struct Range {
    const char *name;
    uintptr_t lo, hi;
};

Range range(const char *name, const void *p, int64_t bytes) {
    uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, p ? lo + static_cast<uintptr_t>(bytes) : lo};
}

bool overlaps(const Range &a, const Range &b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

// Fill n floats with zero.  A kernel rather than hipMemsetAsync so that the
// call stays safe to record into a HIP graph.
__global__ void zero_fill_kernel(float *p, int64_t n) {
    int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (; i < n; i += stride) p[i] = 0.0f;
}

hipError_t zero_fill(float *p, int64_t n, hipStream_t s) {
    if (n <= 0) return hipSuccess;
    int64_t blocks = (n + 255) / 256;
    if (blocks > 4096) blocks = 4096;
    hipLaunchKernelGGL(zero_fill_kernel, dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, s, p, n);
    return hipGetLastError();
}

// The same for a range of bytes that may start and end inside a word.
__global__ void zero_fill_bytes_kernel(unsigned char *p, int64_t n) {
    int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t head = min(n, static_cast<int64_t>((4 - (reinterpret_cast<uintptr_t>(p) & 3)) & 3));
    const int64_t words = (n - head) / 4, tail = head + 4 * words;
    uint32_t *w = reinterpret_cast<uint32_t *>(p + head);
    if (i < head) p[i] = 0;
    if (i < n - tail) p[tail + i] = 0;
    for (; i < words; i += stride) w[i] = 0;
}

hipError_t zero_fill_bytes(void *p, int64_t n, hipStream_t s) {
    if (n <= 0) return hipSuccess;
    int64_t blocks = (n / 4 + 255) / 256;
    if (blocks < 1) blocks = 1;
    if (blocks > 4096) blocks = 4096;
    hipLaunchKernelGGL(zero_fill_bytes_kernel, dim3(static_cast<uint32_t>(blocks)), dim3(256), 0, s,
                       static_cast<unsigned char *>(p), n);
    return hipGetLastError();
}

mssm_status check_dtypes(mssm_dtypes dt) {
    if (dt.io != MSSM_F32 && dt.io != MSSM_BF16)
        return fail(MSSM_ERR_INVALID_ARG, "unknown io dtype %d", dt.io);
    if (dt.param != MSSM_F32 && dt.param != MSSM_BF16)
        return fail(MSSM_ERR_INVALID_ARG, "unknown param dtype %d", dt.param);
    if (dt.param != MSSM_F32)
        return fail(MSSM_ERR_UNSUPPORTED, "param dtype must be MSSM_F32");
    return MSSM_OK;
}

// Shape-based choice.  Short sequences take the row-serial walk (its single
// lane per row has nothing to amortise).  Long sequences whose channels give
// the chunked kernel waves for under four fifths of the 1024 SIMDs of the
// chip are cut into segments and take the look-back kernel; everything else
// takes the chunked kernel, which walks each row in order.  The look-back
// kernel walks every segment twice (state only, then with output), about
// 1.47 times the chunked kernel's vector instructions, but keeps three
// workgroups on every compute unit: measured on the Mamba-130M layer (768
// waves, three quarters of the SIMDs), 237 us against 244 us for the
// chunked kernel, which at one wave per SIMD keeps its SIMDs about 58 %
// busy against the look-back's 66 %.  Nearer a full chip of waves the
// second walk no longer pays.
mssm_variant choose_scan_variant(const mssm::ScanArgs &a) {
    if (a.L < 128 || !mssm::scan_chunked_supported(a)) return MSSM_VARIANT_ROWSERIAL;
    if (a.L >= 2048 && 5 * mssm::scan_chunked_waves(a) < 4 * 1024 && mssm::scan_lookback_supported(a))
        return MSSM_VARIANT_LOOKBACK;
    return MSSM_VARIANT_CHUNKED;
}

// Outputs may not overlap inputs, nor each other; the one exception is an
// initial-state input passed as the final-state output itself (the same
// buffer, exactly), which continues a sequence in place.
mssm_status check_overlaps(const Range *ins, int nin, const Range *outs, int nout,
                           const void *h0, const void *h_last) {
    const bool in_place = h0 && h0 == h_last;
    for (int o = 0; o < nout; ++o)
        for (int i = 0; i < nin; ++i) {
            if (in_place && std::strcmp(ins[i].name, "h0") == 0 &&
                std::strcmp(outs[o].name, "h_last") == 0)
                continue;
            if (overlaps(outs[o], ins[i]))
                return fail(MSSM_ERR_INVALID_ARG, "output %s overlaps input %s", outs[o].name,
                            ins[i].name);
        }
    for (int o = 0; o < nout; ++o)
        for (int p = o + 1; p < nout; ++p)
            if (overlaps(outs[o], outs[p]))
                return fail(MSSM_ERR_INVALID_ARG, "%s overlaps %s", outs[o].name, outs[p].name);
    return MSSM_OK;
}

mssm_status scan_fwd(const void *u, const void *delta, const float *delta_bias, const float *A,
                     const void *B, const void *C, const float *D, const void *z, const float *h0,
                     void *y, float *h_last, mssm_scan_dims dims, mssm_dtypes dtypes,
                     void *stream, const float *conv_w = nullptr, const float *conv_b = nullptr,
                     bool no_alloc = false) {
    g_last_error.clear();
    if (mssm_status s = check_dtypes(dtypes)) return s;
    const int64_t batch = dims.batch, L = dims.seqlen, dim = dims.dim, N = dims.dstate;
    if (batch < 0 || L < 0 || dim < 0)
        return fail(MSSM_ERR_INVALID_ARG, "negative size (batch %lld, L %lld, dim %lld)",
                    (long long)batch, (long long)L, (long long)dim);
    if (N < 1) return fail(MSSM_ERR_INVALID_ARG, "dstate must be >= 1, got %lld", (long long)N);
    if (N > MSSM_MAX_DSTATE)
        return fail(MSSM_ERR_UNSUPPORTED, "dstate %lld exceeds MSSM_MAX_DSTATE (%d)",
                    (long long)N, MSSM_MAX_DSTATE);
    const int64_t esz = dtypes.io == MSSM_F32 ? 4 : 2;
    int64_t rows, act, act_bytes, bc, bc_bytes, dn, hl;
    if (!mul_ok(batch, dim, &rows) || !mul_ok(rows, L, &act) || !mul_ok(act, esz, &act_bytes) ||
        !mul_ok(batch, N, &bc) || !mul_ok(bc, L, &bc) || !mul_ok(bc, esz, &bc_bytes) ||
        !mul_ok(dim, N, &dn) || !mul_ok(rows, N, &hl) || !mul_ok(hl, 4, &hl))
        return fail(MSSM_ERR_INVALID_ARG, "sizes overflow int64");
    if (rows == 0) {
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (L == 0) {
        if (h_last && h0 != h_last) {
            if (h0) {
                if (overlaps(range("h_last", h_last, hl), range("h0", h0, hl)))
                    return fail(MSSM_ERR_INVALID_ARG, "output h_last overlaps input h0");
                hipError_t e = hipMemcpyAsync(h_last, h0, hl, hipMemcpyDeviceToDevice, st);
                if (e != hipSuccess) return hip_fail(e, "copy of h0 to h_last");
            } else {
                hipError_t e = zero_fill(h_last, rows * N, st);
                if (e != hipSuccess) return hip_fail(e, "zero-fill of h_last");
            }
        }
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    if (!u) return fail(MSSM_ERR_INVALID_ARG, "u is null");
    if (!delta) return fail(MSSM_ERR_INVALID_ARG, "delta is null");
    if (!A) return fail(MSSM_ERR_INVALID_ARG, "A is null");
    if (!B) return fail(MSSM_ERR_INVALID_ARG, "B is null");
    if (!C) return fail(MSSM_ERR_INVALID_ARG, "C is null");
    if (!y) return fail(MSSM_ERR_INVALID_ARG, "y is null");

    const Range ins[] = {
        range("u", u, act_bytes),          range("delta", delta, act_bytes),
        range("z", z, act_bytes),          range("B", B, bc_bytes),
        range("C", C, bc_bytes),           range("A", A, dn * 4),
        range("D", D, dim * 4),            range("delta_bias", delta_bias, dim * 4),
        range("h0", h0, hl),               range("conv_w", conv_w, dim * 4 * MSSM_CONV_WIDTH),
        range("conv_b", conv_b, dim * 4)};
    const Range outs[] = {range("y", y, act_bytes), range("h_last", h_last, hl)};
    if (mssm_status c = check_overlaps(ins, 11, outs, 2, h0, h_last)) return c;

    mssm::ScanArgs a{u, delta, delta_bias, A, B, C, D, z, h0, y, h_last, batch, L, dim, N,
                     dtypes.io == MSSM_F32 ? mssm::IO_F32 : mssm::IO_BF16, conv_w, conv_b};

    mssm_variant v = g_forced;
    if (v == MSSM_VARIANT_AUTO) v = choose_scan_variant(a);
    hipError_t e;
    switch (v) {
        case MSSM_VARIANT_ROWSERIAL:
            if (!mssm::scan_rowserial_supported(a))
                return fail(MSSM_ERR_UNSUPPORTED, "row-serial variant does not support this shape");
            e = mssm::launch_scan_rowserial(a, st);
            break;
        case MSSM_VARIANT_CHUNKED:
            if (!mssm::scan_chunked_supported(a))
                return fail(MSSM_ERR_UNSUPPORTED, "chunked variant does not support this shape");
            e = mssm::launch_scan_chunked(a, st);
            break;
        case MSSM_VARIANT_LOOKBACK:
            if (!mssm::scan_lookback_supported(a))
                return fail(MSSM_ERR_UNSUPPORTED, "look-back variant does not support this shape");
            if (no_alloc) {
                const size_t need = mssm::scan_lookback_scratch_bytes(a);
                if (need > mssm::kNoAllocScratchBytes)
                    return fail(MSSM_ERR_UNSUPPORTED,
                                "look-back scratch of %zu bytes exceeds the %zu bytes of the "
                                "no-alloc entry point", need, mssm::kNoAllocScratchBytes);
                e = mssm::launch_scan_lookback_noalloc(a, st);
            } else {
                e = mssm::launch_scan_lookback(a, st);
            }
            break;
        case MSSM_VARIANT_PAIRSCAN:
        case MSSM_VARIANT_PAIRSCAN2:
            if (!mssm::scan_pairscan_supported(a))
                return fail(MSSM_ERR_UNSUPPORTED, "pair-scan variant does not support this shape "
                            "(N <= 16, no convolution prologue)");
            e = mssm::launch_scan_pairscan(a, st, v == MSSM_VARIANT_PAIRSCAN2 ? 2 : 1);
            break;
        default:
            return fail(MSSM_ERR_UNSUPPORTED, "variant %d does not apply to the selective scan",
                        static_cast<int>(v));
    }
    if (e != hipSuccess) return hip_fail(e, "selective-scan launch");
    g_last_variant = v;
    return MSSM_OK;
}

mssm_status ssd_fwd(const void *x, const void *dt, const float *dt_bias, const float *A,
                    const void *B, const void *C, const float *D, const void *z, const float *h0,
                    void *y, float *h_last, mssm_ssd_dims dims, mssm_dtypes dtypes,
                    void *stream) {
    g_last_error.clear();
    if (mssm_status s = check_dtypes(dtypes)) return s;
    const int64_t batch = dims.batch, L = dims.seqlen, H = dims.nheads, P = dims.headdim,
                  N = dims.dstate, G = dims.ngroups, Q = dims.chunk;
    if (batch < 0 || L < 0 || H < 0)
        return fail(MSSM_ERR_INVALID_ARG, "negative size (batch %lld, L %lld, H %lld)",
                    (long long)batch, (long long)L, (long long)H);
    if (P < 1 || N < 1) return fail(MSSM_ERR_INVALID_ARG, "headdim and dstate must be >= 1");
    if (G < 1) return fail(MSSM_ERR_INVALID_ARG, "ngroups must be >= 1");
    if (H % G != 0)
        return fail(MSSM_ERR_INVALID_ARG, "nheads %lld is not a multiple of ngroups %lld",
                    (long long)H, (long long)G);
    if (Q < 0) return fail(MSSM_ERR_INVALID_ARG, "chunk must be >= 0");
    if (P > MSSM_SSD_MAX_HEADDIM || N > MSSM_SSD_MAX_DSTATE)
        return fail(MSSM_ERR_UNSUPPORTED, "headdim %lld / dstate %lld beyond limits (%d / %d)",
                    (long long)P, (long long)N, MSSM_SSD_MAX_HEADDIM, MSSM_SSD_MAX_DSTATE);
    const int64_t esz = dtypes.io == MSSM_F32 ? 4 : 2;
    int64_t bl, xs, x_bytes, dts, dt_bytes, bcs, bc_bytes, pairs, hl;
    if (!mul_ok(batch, L, &bl) || !mul_ok(bl, H, &dts) || !mul_ok(dts, P, &xs) ||
        !mul_ok(xs, esz, &x_bytes) || !mul_ok(dts, esz, &dt_bytes) ||
        !mul_ok(bl, G, &bcs) || !mul_ok(bcs, N, &bcs) || !mul_ok(bcs, esz, &bc_bytes) ||
        !mul_ok(batch, H, &pairs) || !mul_ok(pairs, P, &hl) || !mul_ok(hl, N, &hl) ||
        !mul_ok(hl, 4, &hl))
        return fail(MSSM_ERR_INVALID_ARG, "sizes overflow int64");
    if (pairs == 0) {
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (L == 0) {
        if (h_last && h0 != h_last) {
            if (h0) {
                if (overlaps(range("h_last", h_last, hl), range("h0", h0, hl)))
                    return fail(MSSM_ERR_INVALID_ARG, "output h_last overlaps input h0");
                hipError_t e = hipMemcpyAsync(h_last, h0, hl, hipMemcpyDeviceToDevice, st);
                if (e != hipSuccess) return hip_fail(e, "copy of h0 to h_last");
            } else {
                hipError_t e = zero_fill(h_last, hl / 4, st);
                if (e != hipSuccess) return hip_fail(e, "zero-fill of h_last");
            }
        }
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    if (!x) return fail(MSSM_ERR_INVALID_ARG, "x is null");
    if (!dt) return fail(MSSM_ERR_INVALID_ARG, "dt is null");
    if (!A) return fail(MSSM_ERR_INVALID_ARG, "A is null");
    if (!B) return fail(MSSM_ERR_INVALID_ARG, "B is null");
    if (!C) return fail(MSSM_ERR_INVALID_ARG, "C is null");
    if (!y) return fail(MSSM_ERR_INVALID_ARG, "y is null");
    const Range ins[] = {range("x", x, x_bytes),   range("dt", dt, dt_bytes),
                         range("B", B, bc_bytes),  range("C", C, bc_bytes),
                         range("A", A, H * 4),     range("D", D, H * 4),
                         range("dt_bias", dt_bias, H * 4), range("h0", h0, hl),
                         range("z", z, x_bytes)};
    const Range outs[] = {range("y", y, x_bytes), range("h_last", h_last, hl)};
    if (mssm_status c = check_overlaps(ins, 9, outs, 2, h0, h_last)) return c;

    mssm::SSDArgs a{x, dt, dt_bias, A, B, C, D, z, h0, y, h_last, batch, L, H, P, N, G,
                    Q == 0 ? 256 : Q, dtypes.io == MSSM_F32 ? mssm::IO_F32 : mssm::IO_BF16};
    // The matrix-core form needs bf16 operands and a few chunks to pay off;
    // everything else takes the recurrent form.
    mssm_variant v = g_forced;
    if (v == MSSM_VARIANT_AUTO)
        v = (mssm::ssd_chunked_supported(a) && a.L >= 2 * a.chunk) ? MSSM_VARIANT_SSD_CHUNKED
                                                                    : MSSM_VARIANT_SSD_RECURRENT;
    hipError_t e;
    switch (v) {
        case MSSM_VARIANT_SSD_RECURRENT:
            if (!mssm::ssd_recurrent_supported(a))
                return fail(MSSM_ERR_UNSUPPORTED, "recurrent SSD variant does not support this shape");
            e = mssm::launch_ssd_recurrent(a, st);
            break;
        case MSSM_VARIANT_SSD_CHUNKED:
            if (!mssm::ssd_chunked_supported(a))
                return fail(MSSM_ERR_UNSUPPORTED, "chunked SSD variant needs bf16 I/O, dstate <= 128 "
                            "and chunk 64, 128 or 256");
            e = mssm::launch_ssd_chunked(a, st);
            break;
        default:
            return fail(MSSM_ERR_UNSUPPORTED, "variant %d does not apply to the SSD scan",
                        static_cast<int>(v));
    }
    if (e != hipSuccess) return hip_fail(e, "SSD launch");
    g_last_variant = v;
    return MSSM_OK;
}

// A caller's workspace of `need` bytes (null: none given), as the range that
// the overlap check takes.
mssm_status check_workspace(const void *p, int64_t bytes, size_t need, Range *out) {
    *out = range("workspace", p, static_cast<int64_t>(need));
    if (!p) return MSSM_OK;
    if (bytes < 0 || static_cast<size_t>(bytes) < need)
        return fail(MSSM_ERR_INVALID_ARG, "workspace of %lld bytes is smaller than the %zu needed",
                    (long long)bytes, need);
    if (reinterpret_cast<uintptr_t>(p) % 256 != 0)
        return fail(MSSM_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    return MSSM_OK;
}

mssm::IoType io_type(mssm_dtypes dt) { return dt.io == MSSM_F32 ? mssm::IO_F32 : mssm::IO_BF16; }

// Sizes in bytes of a layer norm's operands, after the checks both passes share.
struct NormSizes {
    int64_t act_bytes, dim_bytes, row_bytes;
};

mssm_status check_norm(mssm_norm_dims d, mssm_dtypes dtypes, NormSizes *z) {
    if (mssm_status s = check_dtypes(dtypes)) return s;
    if (d.rows < 0 || d.dim < 0)
        return fail(MSSM_ERR_INVALID_ARG, "negative size (rows %lld, dim %lld)", (long long)d.rows,
                    (long long)d.dim);
    const int64_t lim = int64_t(1) << 31;
    if (d.rows >= lim || d.dim >= lim)
        return fail(MSSM_ERR_UNSUPPORTED, "rows %lld or dim %lld reaches 2^31", (long long)d.rows,
                    (long long)d.dim);
    if (!mul_ok(d.rows, d.dim, &z->act_bytes) ||
        !mul_ok(z->act_bytes, dtypes.io == MSSM_F32 ? 4 : 2, &z->act_bytes))
        return fail(MSSM_ERR_INVALID_ARG, "sizes overflow int64");
    z->dim_bytes = d.dim * 4;
    z->row_bytes = d.rows * 4;
    return MSSM_OK;
}

struct RecurrenceSizes {
    int64_t rows, act_bytes;   // rows = batch * dim
};

mssm_status check_recurrence(mssm_recurrence_dims d, float scale, mssm_dtypes dtypes,
                             RecurrenceSizes *z) {
    if (mssm_status s = check_dtypes(dtypes)) return s;
    if (d.batch < 0 || d.seqlen < 0 || d.dim < 0)
        return fail(MSSM_ERR_INVALID_ARG, "negative size (batch %lld, L %lld, dim %lld)",
                    (long long)d.batch, (long long)d.seqlen, (long long)d.dim);
    if (!(scale >= 0.0f) || !std::isfinite(scale))
        return fail(MSSM_ERR_INVALID_ARG, "scale must be finite and >= 0, got %g", (double)scale);
    const int64_t lim = int64_t(1) << 31;
    if (d.batch >= lim || d.seqlen >= lim || d.dim >= lim)
        return fail(MSSM_ERR_UNSUPPORTED, "a size reaches 2^31 (batch %lld, L %lld, dim %lld)",
                    (long long)d.batch, (long long)d.seqlen, (long long)d.dim);
    int64_t state_bytes;
    if (!mul_ok(d.batch, d.dim, &z->rows) || !mul_ok(z->rows, 4, &state_bytes) ||
        !mul_ok(z->rows, d.seqlen, &z->act_bytes) ||
        !mul_ok(z->act_bytes, dtypes.io == MSSM_F32 ? 4 : 2, &z->act_bytes))
        return fail(MSSM_ERR_INVALID_ARG, "sizes overflow int64");
    return MSSM_OK;
}

// An empty sequence: the state `out` (n floats, may be null) receives `in`,
// or zeros.
mssm_status copy_or_zero_state(const char *out_name, float *out, const char *in_name,
                               const float *in, int64_t n, hipStream_t st) {
    g_last_variant = MSSM_VARIANT_AUTO;
    if (!out || out == in || n == 0) return MSSM_OK;
    hipError_t e;
    if (in) {
        if (overlaps(range(out_name, out, n * 4), range(in_name, in, n * 4)))
            return fail(MSSM_ERR_INVALID_ARG, "output %s overlaps input %s", out_name, in_name);
        e = hipMemcpyAsync(out, in, n * 4, hipMemcpyDeviceToDevice, st);
    } else {
        e = zero_fill(out, n, st);
    }
    if (e != hipSuccess) return hip_fail(e, "copy of the state of an empty sequence");
    return MSSM_OK;
}

bool on_16(const void *p, const void *q) {
    return ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0;
}

struct LossSizes {
    int64_t hidden_bytes, weight_bytes;
};

mssm_status check_loss(mssm_loss_dims d, mssm_dtypes dtypes, LossSizes *z) {
    if (mssm_status s = check_dtypes(dtypes)) return s;
    if (d.tokens < 0)
        return fail(MSSM_ERR_INVALID_ARG, "negative size (tokens %lld)", (long long)d.tokens);
    if (d.dim < 1 || d.vocab < 1)
        return fail(MSSM_ERR_INVALID_ARG, "dim and vocab must be >= 1, got %lld and %lld",
                    (long long)d.dim, (long long)d.vocab);
    const int64_t lim = int64_t(1) << 20;
    if (d.tokens >= lim || d.vocab >= (int64_t(1) << 30) || d.dim >= lim)
        return fail(MSSM_ERR_UNSUPPORTED,
                    "tokens %lld or dim %lld reaches 2^20, or vocab %lld reaches 2^30",
                    (long long)d.tokens, (long long)d.dim, (long long)d.vocab);
    const int64_t esz = dtypes.io == MSSM_F32 ? 4 : 2;   // at most 2^52 bytes
    z->hidden_bytes = d.tokens * d.dim * esz;
    z->weight_bytes = d.vocab * d.dim * esz;
    return MSSM_OK;
}

// Sizes in bytes of a norm with rotation, after the checks both passes share.
struct HeadNormSizes {
    int64_t q_bytes, k_bytes;
};

mssm_status check_head_norm(mssm_head_norm_dims d, double base, float eps, mssm_dtypes dtypes, HeadNormSizes *z) {
    if (mssm_status s = check_dtypes(dtypes)) return s;
    if (d.tokens < 0 || d.q_heads < 0 || d.k_heads < 0)
        return fail(MSSM_ERR_INVALID_ARG, "negative size (tokens %lld, heads %lld and %lld)", (long long)d.tokens,
                    (long long)d.q_heads, (long long)d.k_heads);
    if (d.dim < 1) return fail(MSSM_ERR_INVALID_ARG, "dim must be >= 1, got %lld", (long long)d.dim);
    if (d.dim > MSSM_MAX_HEAD_DIM)
        return fail(MSSM_ERR_UNSUPPORTED, "dim %lld exceeds MSSM_MAX_HEAD_DIM (%d)", (long long)d.dim, MSSM_MAX_HEAD_DIM);
    if (d.rotary < 0 || d.rotary > d.dim || d.rotary % 2)
        return fail(MSSM_ERR_INVALID_ARG, "rotary must be even and in [0, dim], got %lld", (long long)d.rotary);
    if (!(base > 0.0) || !std::isfinite(base))
        return fail(MSSM_ERR_INVALID_ARG, "base must be finite and > 0, got %g", base);
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return fail(MSSM_ERR_INVALID_ARG, "eps must be finite and >= 0, got %g", (double)eps);
    int64_t q, k;
    const int64_t lim = int64_t(1) << 31;
    if (!mul_ok(d.tokens, d.q_heads, &q) || !mul_ok(d.tokens, d.k_heads, &k) || q >= lim || k >= lim || d.tokens >= lim ||
        d.q_heads >= (lim >> 8) || d.k_heads >= (lim >> 8))
        return fail(MSSM_ERR_UNSUPPORTED, "tokens %lld times heads %lld or %lld is 2^31 or more, or heads 2^23",
                    (long long)d.tokens, (long long)d.q_heads, (long long)d.k_heads);
    const int64_t esz = dtypes.io == MSSM_F32 ? 4 : 2;
    *z = HeadNormSizes{q * d.dim * esz, k * d.dim * esz};
    return MSSM_OK;
}

// Sizes of a linear attention: bytes but for `states`, the states' elements.
struct AttentionSizes {
    int64_t key_bytes, value_bytes, states, state_bytes;
};

mssm_status check_attention(mssm_attention_dims d, float scale, bool packed, mssm_dtypes dtypes, AttentionSizes *z) {
    if (mssm_status s = check_dtypes(dtypes)) return s;
    if (d.seqs < 0 || d.seqlen < 0 || d.total < 0 || d.heads < 0)
        return fail(MSSM_ERR_INVALID_ARG, "negative size (seqs %lld, seqlen %lld, total %lld, heads %lld)",
                    (long long)d.seqs, (long long)d.seqlen, (long long)d.total, (long long)d.heads);
    if (d.key < 1 || d.value < 1)
        return fail(MSSM_ERR_INVALID_ARG, "key and value must be >= 1, got %lld and %lld", (long long)d.key,
                    (long long)d.value);
    if (!std::isfinite(scale)) return fail(MSSM_ERR_INVALID_ARG, "scale must be finite, got %g", (double)scale);
    if (d.key > MSSM_MAX_HEAD_DIM || d.value > MSSM_MAX_HEAD_DIM)
        return fail(MSSM_ERR_UNSUPPORTED, "key %lld or value %lld exceeds MSSM_MAX_HEAD_DIM (%d)", (long long)d.key,
                    (long long)d.value, MSSM_MAX_HEAD_DIM);
    int64_t rows, bh, n;
    const int64_t lim = int64_t(1) << 31;
    if (!mul_ok(d.seqs, d.seqlen, &rows) || !mul_ok(d.seqs, d.heads, &bh) || !mul_ok(d.total, d.heads, &n) ||
        n >= (int64_t(1) << 48))
        return fail(MSSM_ERR_INVALID_ARG, "sizes overflow");
    if (!packed && rows != d.total)
        return fail(MSSM_ERR_INVALID_ARG, "total %lld is not seqs * seqlen (%lld)", (long long)d.total, (long long)rows);
    if (d.seqs >= (lim >> 11) || d.heads >= (lim >> 16) || bh >= (lim >> 11) || d.total >= lim || d.seqlen >= lim)
        return fail(MSSM_ERR_UNSUPPORTED, "heads %lld reach 2^15, seqs * heads %lld 2^20, or total %lld or seqlen %lld 2^31",
                    (long long)d.heads, (long long)bh, (long long)d.total, (long long)d.seqlen);
    const int64_t esz = dtypes.io == MSSM_F32 ? 4 : 2, states = bh * d.key * d.value;
    *z = AttentionSizes{n * d.key * esz, n * d.value * esz, states, states * 4};
    return MSSM_OK;
}

mssm::AttentionArgs attention_args(mssm_attention_dims d, mssm_dtypes dtypes) {
    mssm::AttentionArgs a{};
    a.seqs = d.seqs; a.seqlen = d.seqlen; a.total = d.total; a.heads = d.heads; a.key = d.key; a.value = d.value;
    a.io = io_type(dtypes);
    return a;
}

mssm_status check_beams(mssm_beam_dims d) {
    if (d.batch < 0) return fail(MSSM_ERR_INVALID_ARG, "negative size (batch %lld)", (long long)d.batch);
    if (d.beams < 1) return fail(MSSM_ERR_INVALID_ARG, "beams must be >= 1, got %lld", (long long)d.beams);
    if (d.beams > MSSM_MAX_BEAMS)
        return fail(MSSM_ERR_UNSUPPORTED, "beams %lld exceed MSSM_MAX_BEAMS (%d)", (long long)d.beams, MSSM_MAX_BEAMS);
    if (d.batch >= (int64_t(1) << 24))
        return fail(MSSM_ERR_UNSUPPORTED, "batch %lld reaches 2^24", (long long)d.batch);
    return MSSM_OK;
}

mssm_status check_selection(mssm_beam_dims d, mssm_dtypes dtypes) {
    if (mssm_status s = check_dtypes(dtypes)) return s;
    if (mssm_status s = check_beams(d)) return s;
    if (d.vocab < 1 || d.count < 1)
        return fail(MSSM_ERR_INVALID_ARG, "vocab and count must be >= 1, got %lld and %lld", (long long)d.vocab,
                    (long long)d.count);
    if (d.vocab >= (int64_t(1) << 30) || d.count > MSSM_MAX_BEAM_COUNT)
        return fail(MSSM_ERR_UNSUPPORTED, "vocab %lld reaches 2^30, or count %lld exceeds MSSM_MAX_BEAM_COUNT (%d)",
                    (long long)d.vocab, (long long)d.count, MSSM_MAX_BEAM_COUNT);
    if (d.count > d.beams * d.vocab)
        return fail(MSSM_ERR_INVALID_ARG, "count %lld exceeds beams * vocab", (long long)d.count);
    if (d.batch >= (int64_t(1) << 23))    // its second launch has 512 threads an entry, below 2^32 in all
        return fail(MSSM_ERR_UNSUPPORTED, "batch %lld reaches 2^23", (long long)d.batch);
    if (d.batch * d.beams * mssm::beam_select_pieces(d.vocab) >= (int64_t(1) << 24))
        return fail(MSSM_ERR_UNSUPPORTED, "batch %lld times beams %lld of %lld words is too large", (long long)d.batch,
                    (long long)d.beams, (long long)d.vocab);
    return MSSM_OK;
}

}  // namespace

namespace mssm {

namespace {
constexpr int kPoolDevices = 64;
std::mutex g_pool_mu;
hipMemPool_t g_pool[kPoolDevices] = {};
}  // namespace

// The current device's scratch pool, created on first use with an unlimited
// release threshold.
hipError_t scratch_alloc(void **ptr, size_t bytes, hipStream_t stream) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 0 || dev >= kPoolDevices) return hipErrorInvalidDevice;
    hipMemPool_t pool;
    {
        std::lock_guard<std::mutex> lk(g_pool_mu);
        if (!g_pool[dev]) {
            hipMemPoolProps props;
            std::memset(&props, 0, sizeof props);
            props.allocType = hipMemAllocationTypePinned;
            props.location.type = hipMemLocationTypeDevice;
            props.location.id = dev;
            hipMemPool_t p = nullptr;
            e = hipMemPoolCreate(&p, &props);
            if (e != hipSuccess) return e;
            uint64_t keep = UINT64_MAX;
            e = hipMemPoolSetAttribute(p, hipMemPoolAttrReleaseThreshold, &keep);
            if (e != hipSuccess) {
                (void)hipMemPoolDestroy(p);
                return e;
            }
            g_pool[dev] = p;
        }
        pool = g_pool[dev];
    }
    return hipMallocFromPoolAsync(ptr, bytes, pool, stream);
}

hipError_t scratch_free(void *ptr, hipStream_t stream) { return hipFreeAsync(ptr, stream); }

}  // namespace mssm

extern "C" {

mssm_status mssm_selective_scan_fwd(const void *u, const void *delta,
                                    const float *delta_bias, const float *A,
                                    const void *B, const void *C,
                                    const float *D, const void *z, void *y,
                                    float *h_last, mssm_scan_dims dims,
                                    mssm_dtypes dtypes, void *stream) {
    return scan_fwd(u, delta, delta_bias, A, B, C, D, z, nullptr, y, h_last, dims, dtypes,
                    stream);
}

mssm_status mssm_selective_scan_fwd_h0(const void *u, const void *delta,
                                       const float *delta_bias, const float *A,
                                       const void *B, const void *C, const float *D,
                                       const void *z, const float *h0, void *y,
                                       float *h_last, mssm_scan_dims dims,
                                       mssm_dtypes dtypes, void *stream) {
    return scan_fwd(u, delta, delta_bias, A, B, C, D, z, h0, y, h_last, dims, dtypes, stream);
}

mssm_status mssm_selective_scan_fwd_h0_noalloc(const void *u, const void *delta,
                                               const float *delta_bias, const float *A,
                                               const void *B, const void *C, const float *D,
                                               const void *z, const float *h0, void *y,
                                               float *h_last, mssm_scan_dims dims,
                                               mssm_dtypes dtypes, void *stream) {
    return scan_fwd(u, delta, delta_bias, A, B, C, D, z, h0, y, h_last, dims, dtypes, stream,
                    nullptr, nullptr, true);
}

mssm_status mssm_selective_scan_fwd_conv(const void *x, const float *conv_w,
                                         const float *conv_b, const void *delta,
                                         const float *delta_bias, const float *A, const void *B,
                                         const void *C, const float *D, const void *z,
                                         const float *h0, void *y, float *h_last,
                                         mssm_scan_dims dims, mssm_dtypes dtypes, void *stream) {
    if (!conv_w) {
        g_last_error.clear();
        return fail(MSSM_ERR_INVALID_ARG, "conv_w is null");
    }
    return scan_fwd(x, delta, delta_bias, A, B, C, D, z, h0, y, h_last, dims, dtypes, stream,
                    conv_w, conv_b);
}

mssm_status mssm_selective_scan_bwd(const void *u, const void *delta, const float *delta_bias,
                                    const float *A, const void *B, const void *C, const float *D,
                                    const void *z, const float *h0, const void *dy,
                                    const float *dh_last, float *du, float *ddelta,
                                    float *ddelta_bias, float *dA, float *dB, float *dC, float *dD,
                                    float *dz, float *dh0, mssm_scan_dims dims, mssm_dtypes dtypes,
                                    void *stream) {
    g_last_error.clear();
    if (mssm_status s = check_dtypes(dtypes)) return s;
    const int64_t batch = dims.batch, L = dims.seqlen, dim = dims.dim, N = dims.dstate;
    if (batch < 0 || L < 0 || dim < 0)
        return fail(MSSM_ERR_INVALID_ARG, "negative size (batch %lld, L %lld, dim %lld)",
                    (long long)batch, (long long)L, (long long)dim);
    if (N < 1) return fail(MSSM_ERR_INVALID_ARG, "dstate must be >= 1, got %lld", (long long)N);
    if (N > MSSM_MAX_DSTATE)
        return fail(MSSM_ERR_UNSUPPORTED, "dstate %lld exceeds MSSM_MAX_DSTATE (%d)",
                    (long long)N, MSSM_MAX_DSTATE);
    if (dz && !z) return fail(MSSM_ERR_INVALID_ARG, "dz given without z");
    const int64_t esz = dtypes.io == MSSM_F32 ? 4 : 2;
    int64_t rows, act, act_bytes, act4, bc, bc_bytes, bc4, dn, hl;
    if (!mul_ok(batch, dim, &rows) || !mul_ok(rows, L, &act) || !mul_ok(act, esz, &act_bytes) ||
        !mul_ok(act, 4, &act4) || !mul_ok(batch, N, &bc) || !mul_ok(bc, L, &bc) ||
        !mul_ok(bc, esz, &bc_bytes) || !mul_ok(bc, 4, &bc4) || !mul_ok(dim, N, &dn) ||
        !mul_ok(rows, N, &hl) || !mul_ok(hl, 4, &hl))
        return fail(MSSM_ERR_INVALID_ARG, "sizes overflow int64");
    hipStream_t st = static_cast<hipStream_t>(stream);
    // the accumulated gradients start from zero, whatever else happens
    auto zero_sums = [&]() -> hipError_t {
        hipError_t e = hipSuccess;
        if (e == hipSuccess && dB) e = zero_fill(dB, bc, st);
        if (e == hipSuccess && dC) e = zero_fill(dC, bc, st);
        if (e == hipSuccess && dA) e = zero_fill(dA, dn, st);
        if (e == hipSuccess && dD) e = zero_fill(dD, dim, st);
        if (e == hipSuccess && ddelta_bias) e = zero_fill(ddelta_bias, dim, st);
        return e;
    };
    if (rows == 0 || L == 0) {
        const Range outs0[] = {range("dB", dB, bc4), range("dC", dC, bc4), range("dA", dA, dn * 4),
                               range("dD", dD, dim * 4), range("ddelta_bias", ddelta_bias, dim * 4),
                               range("dh0", dh0, hl)};
        for (int i = 0; i < 6; ++i)
            for (int j = i + 1; j < 6; ++j)
                if (overlaps(outs0[i], outs0[j]))
                    return fail(MSSM_ERR_INVALID_ARG, "%s overlaps %s", outs0[i].name, outs0[j].name);
        hipError_t e = zero_sums();
        // with L == 0 the initial state is the final state: dh0 = dh_last
        if (e == hipSuccess && dh0 && rows > 0) {
            e = dh_last ? hipMemcpyAsync(dh0, dh_last, hl, hipMemcpyDeviceToDevice, st)
                        : zero_fill(dh0, rows * N, st);
        }
        if (e != hipSuccess) return hip_fail(e, "zero-fill of the gradients");
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    if (!u) return fail(MSSM_ERR_INVALID_ARG, "u is null");
    if (!delta) return fail(MSSM_ERR_INVALID_ARG, "delta is null");
    if (!A) return fail(MSSM_ERR_INVALID_ARG, "A is null");
    if (!B) return fail(MSSM_ERR_INVALID_ARG, "B is null");
    if (!C) return fail(MSSM_ERR_INVALID_ARG, "C is null");
    if (!dy) return fail(MSSM_ERR_INVALID_ARG, "dy is null");
    if (!du) return fail(MSSM_ERR_INVALID_ARG, "du is null");
    if (!ddelta) return fail(MSSM_ERR_INVALID_ARG, "ddelta is null");
    const Range ins[] = {
        range("u", u, act_bytes),          range("delta", delta, act_bytes),
        range("z", z, act_bytes),          range("B", B, bc_bytes),
        range("C", C, bc_bytes),           range("A", A, dn * 4),
        range("D", D, dim * 4),            range("delta_bias", delta_bias, dim * 4),
        range("h0", h0, hl),               range("dy", dy, act_bytes),
        range("dh_last", dh_last, hl)};
    const Range outs[] = {
        range("du", du, act4),             range("ddelta", ddelta, act4),
        range("dz", dz, act4),             range("dB", dB, bc4),
        range("dC", dC, bc4),              range("dA", dA, dn * 4),
        range("dD", dD, dim * 4),          range("ddelta_bias", ddelta_bias, dim * 4),
        range("dh0", dh0, hl)};
    if (mssm_status c = check_overlaps(ins, 11, outs, 9, nullptr, nullptr)) return c;

    mssm::BwdArgs a{u, delta, delta_bias, A, B, C, D, z, h0, dy, dh_last, du, ddelta, ddelta_bias,
                    dA, dB, dC, dD, dz, dh0, batch, L, dim, N,
                    dtypes.io == MSSM_F32 ? mssm::IO_F32 : mssm::IO_BF16};
    // AUTO: the chunked backward where it applies (N <= 16), else the
    // row-serial one; either can be forced
    mssm_variant v = g_forced;
    if (v == MSSM_VARIANT_AUTO)
        v = mssm::scan_bwd_chunked_supported(a) ? MSSM_VARIANT_CHUNKED : MSSM_VARIANT_ROWSERIAL;
    if (v == MSSM_VARIANT_CHUNKED) {
        if (!mssm::scan_bwd_chunked_supported(a))
            return fail(MSSM_ERR_UNSUPPORTED, "chunked backward needs N <= 16");
    } else if (v == MSSM_VARIANT_ROWSERIAL) {
        if (!mssm::scan_bwd_supported(a))
            return fail(MSSM_ERR_UNSUPPORTED, "backward does not support this shape");
    } else {
        return fail(MSSM_ERR_UNSUPPORTED, "variant %d does not apply to the backward",
                    static_cast<int>(v));
    }
    hipError_t e = zero_sums();
    if (e == hipSuccess)
        e = v == MSSM_VARIANT_CHUNKED ? mssm::launch_scan_bwd_chunked(a, st) : mssm::launch_scan_bwd(a, st);
    if (e != hipSuccess) return hip_fail(e, "selective-scan backward launch");
    g_last_variant = v;
    return MSSM_OK;
}

mssm_status mssm_ssd_scalar_fwd(const void *x, const void *dt, const float *dt_bias,
                                const float *A, const void *B, const void *C,
                                const float *D, void *y, float *h_last,
                                mssm_ssd_dims dims, mssm_dtypes dtypes, void *stream) {
    return ssd_fwd(x, dt, dt_bias, A, B, C, D, nullptr, nullptr, y, h_last, dims, dtypes, stream);
}

mssm_status mssm_ssd_scalar_fwd_h0(const void *x, const void *dt, const float *dt_bias,
                                   const float *A, const void *B, const void *C,
                                   const float *D, const float *h0, void *y, float *h_last,
                                   mssm_ssd_dims dims, mssm_dtypes dtypes, void *stream) {
    return ssd_fwd(x, dt, dt_bias, A, B, C, D, nullptr, h0, y, h_last, dims, dtypes, stream);
}

mssm_status mssm_ssd_scalar_fwd_gated(const void *x, const void *dt, const float *dt_bias,
                                      const float *A, const void *B, const void *C,
                                      const float *D, const void *z, const float *h0, void *y,
                                      float *h_last, mssm_ssd_dims dims, mssm_dtypes dtypes,
                                      void *stream) {
    return ssd_fwd(x, dt, dt_bias, A, B, C, D, z, h0, y, h_last, dims, dtypes, stream);
}

mssm_status mssm_selective_state_update(float *state, const void *x, const void *dt,
                                        const float *dt_bias, const float *A, const void *B,
                                        const void *C, const float *D, const void *z, void *y,
                                        mssm_step_dims dims, mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    if (mssm_status s = check_dtypes(dtypes)) return s;
    const int64_t batch = dims.batch, dim = dims.dim, N = dims.dstate;
    if (batch < 0 || dim < 0)
        return fail(MSSM_ERR_INVALID_ARG, "negative size (batch %lld, dim %lld)", (long long)batch,
                    (long long)dim);
    if (N < 1) return fail(MSSM_ERR_INVALID_ARG, "dstate must be >= 1, got %lld", (long long)N);
    if (N > MSSM_MAX_DSTATE)
        return fail(MSSM_ERR_UNSUPPORTED, "dstate %lld exceeds MSSM_MAX_DSTATE (%d)",
                    (long long)N, MSSM_MAX_DSTATE);
    const int64_t esz = dtypes.io == MSSM_F32 ? 4 : 2;
    int64_t rows, row_bytes, st_bytes, bc_bytes, dn;
    if (!mul_ok(batch, dim, &rows) || !mul_ok(rows, esz, &row_bytes) ||
        !mul_ok(rows, N, &st_bytes) || !mul_ok(st_bytes, 4, &st_bytes) ||
        !mul_ok(batch, N, &bc_bytes) || !mul_ok(bc_bytes, esz, &bc_bytes) ||
        !mul_ok(dim, N, &dn))
        return fail(MSSM_ERR_INVALID_ARG, "sizes overflow int64");
    if (rows == 0) {
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    if (!state) return fail(MSSM_ERR_INVALID_ARG, "state is null");
    if (!x) return fail(MSSM_ERR_INVALID_ARG, "x is null");
    if (!dt) return fail(MSSM_ERR_INVALID_ARG, "dt is null");
    if (!A) return fail(MSSM_ERR_INVALID_ARG, "A is null");
    if (!B) return fail(MSSM_ERR_INVALID_ARG, "B is null");
    if (!C) return fail(MSSM_ERR_INVALID_ARG, "C is null");
    if (!y) return fail(MSSM_ERR_INVALID_ARG, "y is null");
    const Range ins[] = {range("x", x, row_bytes),   range("dt", dt, row_bytes),
                         range("z", z, row_bytes),   range("B", B, bc_bytes),
                         range("C", C, bc_bytes),    range("A", A, dn * 4),
                         range("D", D, dim * 4),     range("dt_bias", dt_bias, dim * 4)};
    const Range outs[] = {range("y", y, row_bytes), range("state", state, st_bytes)};
    if (mssm_status c = check_overlaps(ins, 8, outs, 2, nullptr, nullptr)) return c;

    mssm::StepArgs a{state, x, dt, dt_bias, A, B, C, D, z, y, batch, dim, N,
                     dtypes.io == MSSM_F32 ? mssm::IO_F32 : mssm::IO_BF16};
    if (!mssm::state_update_supported(a))
        return fail(MSSM_ERR_UNSUPPORTED, "state update does not support this shape");
    const hipError_t e = mssm::launch_state_update(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "state-update launch");
    g_last_variant = MSSM_VARIANT_AUTO;
    return MSSM_OK;
}

mssm_status mssm_layer_norm_fwd(const void *x, const float *weight, const float *bias, float eps,
                                void *y, float *mean, float *rstd, mssm_norm_dims dims,
                                mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    NormSizes z;
    if (mssm_status s = check_norm(dims, dtypes, &z)) return s;
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return fail(MSSM_ERR_INVALID_ARG, "eps must be finite and >= 0, got %g", (double)eps);
    if (dims.rows == 0 || dims.dim == 0) {
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    if (!x) return fail(MSSM_ERR_INVALID_ARG, "x is null");
    if (!y) return fail(MSSM_ERR_INVALID_ARG, "y is null");
    const Range ins[] = {range("x", x, z.act_bytes), range("weight", weight, z.dim_bytes),
                         range("bias", bias, z.dim_bytes)};
    const Range outs[] = {range("y", y, z.act_bytes), range("mean", mean, z.row_bytes),
                          range("rstd", rstd, z.row_bytes)};
    if (mssm_status c = check_overlaps(ins, 3, outs, 3, nullptr, nullptr)) return c;
    mssm::NormArgs a{x, weight, bias, eps, y, mean, rstd, nullptr, nullptr, nullptr, nullptr,
                     dims.rows, dims.dim, io_type(dtypes)};
    const hipError_t e = mssm::launch_layer_norm_fwd(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "layer-norm launch");
    g_last_variant = MSSM_VARIANT_AUTO;
    return MSSM_OK;
}

mssm_status mssm_layer_norm_bwd(const void *dy, const void *x, const float *mean, const float *rstd,
                                const float *weight, void *dx, float *dweight, float *dbias,
                                void *workspace, int64_t workspace_bytes, mssm_norm_dims dims,
                                mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    NormSizes z;
    if (mssm_status s = check_norm(dims, dtypes, &z)) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    mssm::NormArgs a{x, weight, nullptr, 0.0f, nullptr, const_cast<float *>(mean),
                     const_cast<float *>(rstd), dy, dx, dweight, dbias, dims.rows, dims.dim, io_type(dtypes)};
    Range ws;
    if (mssm_status s = check_workspace(workspace, workspace_bytes, mssm::layer_norm_bwd_workspace(a), &ws)) return s;
    const Range outs[] = {range("dx", dx, z.act_bytes), range("dweight", dweight, z.dim_bytes),
                          range("dbias", dbias, z.dim_bytes), ws};
    if (dims.rows == 0 || dims.dim == 0) {
        if (overlaps(outs[1], outs[2])) return fail(MSSM_ERR_INVALID_ARG, "dweight overlaps dbias");
        hipError_t e = hipSuccess;
        if (dweight) e = zero_fill(dweight, dims.dim, st);
        if (e == hipSuccess && dbias) e = zero_fill(dbias, dims.dim, st);
        if (e != hipSuccess) return hip_fail(e, "zero-fill of the gradients");
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    if (!dy) return fail(MSSM_ERR_INVALID_ARG, "dy is null");
    if (!x) return fail(MSSM_ERR_INVALID_ARG, "x is null");
    if (!mean) return fail(MSSM_ERR_INVALID_ARG, "mean is null");
    if (!rstd) return fail(MSSM_ERR_INVALID_ARG, "rstd is null");
    if (!dx) return fail(MSSM_ERR_INVALID_ARG, "dx is null");
    const Range ins[] = {range("dy", dy, z.act_bytes), range("x", x, z.act_bytes),
                         range("mean", mean, z.row_bytes), range("rstd", rstd, z.row_bytes),
                         range("weight", weight, z.dim_bytes)};
    if (mssm_status c = check_overlaps(ins, 5, outs, 4, nullptr, nullptr)) return c;
    const hipError_t e = mssm::launch_layer_norm_bwd(a, workspace, st);
    if (e != hipSuccess) return hip_fail(e, "layer-norm backward launch");
    g_last_variant = MSSM_VARIANT_AUTO;
    return MSSM_OK;
}

mssm_status mssm_gated_recurrence_fwd(const void *x, const void *r, const void *i, const float *lam,
                                      float scale, const float *h0, void *y, float *h_last,
                                      void *workspace, int64_t workspace_bytes,
                                      mssm_recurrence_dims dims, mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    RecurrenceSizes z;
    if (mssm_status s = check_recurrence(dims, scale, dtypes, &z)) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (z.rows == 0) {
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    if (dims.seqlen == 0) return copy_or_zero_state("h_last", h_last, "h0", h0, z.rows, st);
    if (!x) return fail(MSSM_ERR_INVALID_ARG, "x is null");
    if (!r) return fail(MSSM_ERR_INVALID_ARG, "r is null");
    if (!i) return fail(MSSM_ERR_INVALID_ARG, "i is null");
    if (!lam) return fail(MSSM_ERR_INVALID_ARG, "lam is null");
    if (!y) return fail(MSSM_ERR_INVALID_ARG, "y is null");
    const Range ins[] = {range("x", x, z.act_bytes), range("r", r, z.act_bytes),
                         range("i", i, z.act_bytes), range("lam", lam, dims.dim * 4),
                         range("h0", h0, z.rows * 4)};
    mssm::RecurrenceArgs a{};
    a.x = x; a.r = r; a.i = i; a.lam = lam; a.scale = scale; a.h0 = h0; a.y = y; a.h_last = h_last;
    a.batch = dims.batch; a.L = dims.seqlen; a.dim = dims.dim;
    a.io = io_type(dtypes);
    if (!mssm::gated_recurrence_supported(a))
        return fail(MSSM_ERR_UNSUPPORTED, "gated recurrence does not support this shape");
    Range ws;
    if (mssm_status s = check_workspace(workspace, workspace_bytes, mssm::gated_recurrence_workspace(a, false), &ws))
        return s;
    const Range outs[] = {range("y", y, z.act_bytes), range("h_last", h_last, z.rows * 4), ws};
    if (mssm_status c = check_overlaps(ins, 5, outs, 3, h0, h_last)) return c;
    const hipError_t e = mssm::launch_gated_recurrence_fwd(a, workspace, st);
    if (e != hipSuccess) return hip_fail(e, "gated-recurrence launch");
    g_last_variant = MSSM_VARIANT_AUTO;
    return MSSM_OK;
}

mssm_status mssm_gated_recurrence_bwd(const void *x, const void *r, const void *i, const float *lam,
                                      float scale, const float *h0, const void *y, const void *dy,
                                      const float *dh_last, void *dx, void *dr, void *di,
                                      float *dlam, float *dh0, void *workspace,
                                      int64_t workspace_bytes, mssm_recurrence_dims dims,
                                      mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    RecurrenceSizes z;
    if (mssm_status s = check_recurrence(dims, scale, dtypes, &z)) return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    Range outs[] = {range("dx", dx, z.act_bytes), range("dr", dr, z.act_bytes),
                          range("di", di, z.act_bytes), range("dlam", dlam, dims.dim * 4),
                          range("dh0", dh0, z.rows * 4), Range{}};
    if (z.rows == 0 || dims.seqlen == 0) {
        if (overlaps(outs[3], outs[4])) return fail(MSSM_ERR_INVALID_ARG, "dlam overlaps dh0");
        if (overlaps(outs[3], range("dh_last", dh_last, z.rows * 4)))
            return fail(MSSM_ERR_INVALID_ARG, "output dlam overlaps input dh_last");
        if (dh0 && dh0 == dh_last) return fail(MSSM_ERR_INVALID_ARG, "output dh0 overlaps input dh_last");
        if (mssm_status s = copy_or_zero_state("dh0", dh0, "dh_last", dh_last, z.rows, st)) return s;
        if (dlam) {
            const hipError_t e = zero_fill(dlam, dims.dim, st);
            if (e != hipSuccess) return hip_fail(e, "zero-fill of dlam");
        }
        return MSSM_OK;
    }
    if (!x) return fail(MSSM_ERR_INVALID_ARG, "x is null");
    if (!r) return fail(MSSM_ERR_INVALID_ARG, "r is null");
    if (!i) return fail(MSSM_ERR_INVALID_ARG, "i is null");
    if (!lam) return fail(MSSM_ERR_INVALID_ARG, "lam is null");
    if (!y) return fail(MSSM_ERR_INVALID_ARG, "y is null");
    if (!dy) return fail(MSSM_ERR_INVALID_ARG, "dy is null");
    if (!dx) return fail(MSSM_ERR_INVALID_ARG, "dx is null");
    if (!dr) return fail(MSSM_ERR_INVALID_ARG, "dr is null");
    if (!di) return fail(MSSM_ERR_INVALID_ARG, "di is null");
    const Range ins[] = {range("x", x, z.act_bytes), range("r", r, z.act_bytes),
                         range("i", i, z.act_bytes), range("lam", lam, dims.dim * 4),
                         range("h0", h0, z.rows * 4), range("y", y, z.act_bytes),
                         range("dy", dy, z.act_bytes), range("dh_last", dh_last, z.rows * 4)};
    mssm::RecurrenceArgs a{};
    a.x = x; a.r = r; a.i = i; a.lam = lam; a.scale = scale; a.h0 = h0;
    a.y = const_cast<void *>(y); a.dy = dy; a.dh_last = dh_last;
    a.dx = dx; a.dr = dr; a.di = di; a.dlam = dlam; a.dh0 = dh0;
    a.batch = dims.batch; a.L = dims.seqlen; a.dim = dims.dim;
    a.io = io_type(dtypes);
    if (!mssm::gated_recurrence_supported(a))
        return fail(MSSM_ERR_UNSUPPORTED, "gated recurrence does not support this shape");
    if (mssm_status s = check_workspace(workspace, workspace_bytes, mssm::gated_recurrence_workspace(a, true), &outs[5]))
        return s;
    if (mssm_status c = check_overlaps(ins, 8, outs, 6, nullptr, nullptr)) return c;
    const hipError_t e = mssm::launch_gated_recurrence_bwd(a, workspace, st);
    if (e != hipSuccess) return hip_fail(e, "gated-recurrence backward launch");
    g_last_variant = MSSM_VARIANT_AUTO;
    return MSSM_OK;
}

mssm_status mssm_gated_recurrence_update(float *state, const void *x, const void *r, const void *i,
                                         const float *lam, float scale, void *y,
                                         mssm_recurrence_dims dims, mssm_dtypes dtypes, void *stream) {
    if (dims.batch > 0 && dims.dim > 0 && !state) {
        g_last_error.clear();
        return fail(MSSM_ERR_INVALID_ARG, "state is null");
    }
    dims.seqlen = 1;
    return mssm_gated_recurrence_fwd(x, r, i, lam, scale, state, y, state, nullptr, 0, dims, dtypes, stream);
}

mssm_status mssm_linear_cross_entropy_fwd(const void *hidden, const void *weight,
                                          const int64_t *targets, int64_t ignore_index, float *loss,
                                          float *lse, void *workspace, int64_t workspace_bytes,
                                          mssm_loss_dims dims, mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    LossSizes z;
    if (mssm_status s = check_loss(dims, dtypes, &z)) return s;
    if (dims.tokens == 0) {
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    if (!hidden) return fail(MSSM_ERR_INVALID_ARG, "hidden is null");
    if (!weight) return fail(MSSM_ERR_INVALID_ARG, "weight is null");
    if (!targets) return fail(MSSM_ERR_INVALID_ARG, "targets is null");
    if (!loss) return fail(MSSM_ERR_INVALID_ARG, "loss is null");
    const Range ins[] = {range("hidden", hidden, z.hidden_bytes), range("weight", weight, z.weight_bytes),
                         range("targets", targets, dims.tokens * 8)};
    mssm::LossArgs a{hidden, weight, targets, ignore_index, loss, lse, nullptr, nullptr, nullptr,
                     dims.tokens, dims.dim, dims.vocab, io_type(dtypes)};
    Range ws;
    if (mssm_status s = check_workspace(workspace, workspace_bytes,
                                        mssm::linear_cross_entropy_workspace(a, false, on_16(hidden, weight)), &ws))
        return s;
    const Range outs[] = {range("loss", loss, dims.tokens * 4), range("lse", lse, dims.tokens * 4), ws};
    if (mssm_status c = check_overlaps(ins, 3, outs, 3, nullptr, nullptr)) return c;
    const hipError_t e = mssm::launch_linear_cross_entropy_fwd(a, workspace, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "cross-entropy launch");
    g_last_variant = MSSM_VARIANT_AUTO;
    return MSSM_OK;
}

mssm_status mssm_linear_cross_entropy_bwd(const void *hidden, const void *weight,
                                          const int64_t *targets, int64_t ignore_index,
                                          const float *lse, const float *dloss, void *dhidden,
                                          void *dweight, void *workspace, int64_t workspace_bytes,
                                          mssm_loss_dims dims, mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    LossSizes z;
    if (mssm_status s = check_loss(dims, dtypes, &z)) return s;
    if (!dweight) return fail(MSSM_ERR_INVALID_ARG, "dweight is null");
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dims.tokens == 0) {
        // zero bits are zeros in either dtype; a bf16 buffer may start and
        // end inside a 4-byte word
        const hipError_t e = zero_fill_bytes(dweight, z.weight_bytes, st);
        if (e != hipSuccess) return hip_fail(e, "zero-fill of dweight");
        g_last_variant = MSSM_VARIANT_AUTO;
        return MSSM_OK;
    }
    if (!hidden) return fail(MSSM_ERR_INVALID_ARG, "hidden is null");
    if (!weight) return fail(MSSM_ERR_INVALID_ARG, "weight is null");
    if (!targets) return fail(MSSM_ERR_INVALID_ARG, "targets is null");
    if (!lse) return fail(MSSM_ERR_INVALID_ARG, "lse is null");
    if (!dloss) return fail(MSSM_ERR_INVALID_ARG, "dloss is null");
    if (!dhidden) return fail(MSSM_ERR_INVALID_ARG, "dhidden is null");
    const Range ins[] = {range("hidden", hidden, z.hidden_bytes), range("weight", weight, z.weight_bytes),
                         range("targets", targets, dims.tokens * 8), range("lse", lse, dims.tokens * 4),
                         range("dloss", dloss, dims.tokens * 4)};
    mssm::LossArgs a{hidden, weight, targets, ignore_index, nullptr, const_cast<float *>(lse), dloss,
                     dhidden, dweight, dims.tokens, dims.dim, dims.vocab, io_type(dtypes)};
    Range ws;
    if (mssm_status s = check_workspace(workspace, workspace_bytes,
                                        mssm::linear_cross_entropy_workspace(a, true, on_16(hidden, weight)), &ws))
        return s;
    const Range outs[] = {range("dhidden", dhidden, z.hidden_bytes),
                          range("dweight", dweight, z.weight_bytes), ws};
    if (mssm_status c = check_overlaps(ins, 5, outs, 3, nullptr, nullptr)) return c;
    const hipError_t e = mssm::launch_linear_cross_entropy_bwd(a, workspace, st);
    if (e != hipSuccess) return hip_fail(e, "cross-entropy backward launch");
    g_last_variant = MSSM_VARIANT_AUTO;
    return MSSM_OK;
}

int64_t mssm_layer_norm_bwd_workspace(mssm_norm_dims dims, mssm_dtypes dtypes) {
    g_last_error.clear();
    NormSizes z;
    if (check_norm(dims, dtypes, &z)) return -1;
    mssm::NormArgs a{};
    a.rows = dims.rows; a.dim = dims.dim; a.io = io_type(dtypes);
    return static_cast<int64_t>(mssm::layer_norm_bwd_workspace(a));
}

int64_t mssm_gated_recurrence_workspace(mssm_recurrence_dims dims, mssm_dtypes dtypes, int backward) {
    g_last_error.clear();
    RecurrenceSizes z;
    if (check_recurrence(dims, 0.0f, dtypes, &z)) return -1;
    if (z.rows == 0 || dims.seqlen == 0) return 0;
    mssm::RecurrenceArgs a{};
    a.batch = dims.batch; a.L = dims.seqlen; a.dim = dims.dim; a.io = io_type(dtypes);
    if (!mssm::gated_recurrence_supported(a)) {
        fail(MSSM_ERR_UNSUPPORTED, "gated recurrence does not support this shape");
        return -1;
    }
    return static_cast<int64_t>(mssm::gated_recurrence_workspace(a, backward != 0));
}

int64_t mssm_linear_cross_entropy_workspace(mssm_loss_dims dims, mssm_dtypes dtypes, int backward, int aligned) {
    g_last_error.clear();
    LossSizes z;
    if (check_loss(dims, dtypes, &z)) return -1;
    if (dims.tokens == 0) return 0;
    mssm::LossArgs a{};
    a.tokens = dims.tokens; a.dim = dims.dim; a.vocab = dims.vocab; a.io = io_type(dtypes);
    return static_cast<int64_t>(mssm::linear_cross_entropy_workspace(a, backward != 0, aligned != 0));
}

mssm_status mssm_qk_norm_rotary_fwd(const void *q, const void *k, const int64_t *positions,
                                    const float *q_weight, const float *k_weight, double base,
                                    float eps, void *q_out, void *k_out, mssm_head_norm_dims dims,
                                    mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    HeadNormSizes z;
    if (mssm_status s = check_head_norm(dims, base, eps, dtypes, &z)) return s;
    g_last_variant = MSSM_VARIANT_AUTO;
    if (z.q_bytes == 0 && z.k_bytes == 0) return MSSM_OK;
    if (z.q_bytes && !q) return fail(MSSM_ERR_INVALID_ARG, "q is null");
    if (z.k_bytes && !k) return fail(MSSM_ERR_INVALID_ARG, "k is null");
    if (dims.rotary && !positions) return fail(MSSM_ERR_INVALID_ARG, "positions is null");
    if (z.q_bytes && !q_out) return fail(MSSM_ERR_INVALID_ARG, "q_out is null");
    if (z.k_bytes && !k_out) return fail(MSSM_ERR_INVALID_ARG, "k_out is null");
    const Range ins[] = {range("q", q, z.q_bytes), range("k", k, z.k_bytes),
                         range("positions", positions, dims.tokens * 8),
                         range("q_weight", q_weight, dims.dim * 4), range("k_weight", k_weight, dims.dim * 4)};
    const Range outs[] = {range("q_out", q_out, z.q_bytes), range("k_out", k_out, z.k_bytes)};
    if (mssm_status c = check_overlaps(ins, 5, outs, 2, nullptr, nullptr)) return c;
    const mssm::HeadNormArgs a{q, k, positions, q_weight, k_weight, base, eps, q_out, k_out, nullptr, nullptr,
                               nullptr, nullptr, dims.tokens, dims.q_heads, dims.k_heads, dims.dim, dims.rotary,
                               io_type(dtypes)};
    const hipError_t e = mssm::launch_qk_norm_rotary_fwd(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "norm-and-rotation launch");
    return MSSM_OK;
}

mssm_status mssm_qk_norm_rotary_bwd(const void *dq_out, const void *dk_out, const void *q, const void *k,
                                    const int64_t *positions, const float *q_weight,
                                    const float *k_weight, double base, float eps, void *dq, void *dk,
                                    float *dq_weight, float *dk_weight, void *workspace,
                                    int64_t workspace_bytes, mssm_head_norm_dims dims,
                                    mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    HeadNormSizes z;
    if (mssm_status s = check_head_norm(dims, base, eps, dtypes, &z)) return s;
    g_last_variant = MSSM_VARIANT_AUTO;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const mssm::HeadNormArgs a{q, k, positions, q_weight, k_weight, base, eps, dq, dk, dq_out, dk_out,
                               dq_weight, dk_weight, dims.tokens, dims.q_heads, dims.k_heads, dims.dim, dims.rotary,
                               io_type(dtypes)};
    Range ws;
    if (mssm_status s = check_workspace(workspace, workspace_bytes, mssm::qk_norm_rotary_bwd_workspace(a), &ws)) return s;
    const Range outs[] = {range("dq", dq, z.q_bytes), range("dk", dk, z.k_bytes),
                          range("dq_weight", dq_weight, dims.dim * 4), range("dk_weight", dk_weight, dims.dim * 4), ws};
    if (z.q_bytes == 0 && z.k_bytes == 0) {
        if (overlaps(outs[2], outs[3])) return fail(MSSM_ERR_INVALID_ARG, "dq_weight overlaps dk_weight");
        hipError_t e = hipSuccess;
        if (dq_weight) e = zero_fill(dq_weight, dims.dim, st);
        if (e == hipSuccess && dk_weight) e = zero_fill(dk_weight, dims.dim, st);
        if (e != hipSuccess) return hip_fail(e, "zero-fill of the gradients");
        return MSSM_OK;
    }
    if (z.q_bytes && !dq_out) return fail(MSSM_ERR_INVALID_ARG, "dq_out is null");
    if (z.k_bytes && !dk_out) return fail(MSSM_ERR_INVALID_ARG, "dk_out is null");
    if (z.q_bytes && !q) return fail(MSSM_ERR_INVALID_ARG, "q is null");
    if (z.k_bytes && !k) return fail(MSSM_ERR_INVALID_ARG, "k is null");
    if (dims.rotary && !positions) return fail(MSSM_ERR_INVALID_ARG, "positions is null");
    if (z.q_bytes && !dq) return fail(MSSM_ERR_INVALID_ARG, "dq is null");
    if (z.k_bytes && !dk) return fail(MSSM_ERR_INVALID_ARG, "dk is null");
    const Range ins[] = {range("dq_out", dq_out, z.q_bytes), range("dk_out", dk_out, z.k_bytes),
                         range("q", q, z.q_bytes), range("k", k, z.k_bytes),
                         range("positions", positions, dims.tokens * 8),
                         range("q_weight", q_weight, dims.dim * 4), range("k_weight", k_weight, dims.dim * 4)};
    if (mssm_status c = check_overlaps(ins, 7, outs, 5, nullptr, nullptr)) return c;
    const hipError_t e = mssm::launch_qk_norm_rotary_bwd(a, workspace, st);
    if (e != hipSuccess) return hip_fail(e, "norm-and-rotation backward launch");
    return MSSM_OK;
}

int64_t mssm_qk_norm_rotary_bwd_workspace(mssm_head_norm_dims dims, mssm_dtypes dtypes) {
    g_last_error.clear();
    HeadNormSizes z;
    if (check_head_norm(dims, 1.0, 0.0f, dtypes, &z)) return -1;
    mssm::HeadNormArgs a{};
    a.tokens = dims.tokens; a.q_heads = dims.q_heads; a.k_heads = dims.k_heads;
    a.dim = dims.dim; a.rotary = dims.rotary; a.io = io_type(dtypes);
    return static_cast<int64_t>(mssm::qk_norm_rotary_bwd_workspace(a));
}

mssm_status mssm_linear_attention_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                                      float scale, const float *h0, const int64_t *cu_seqlens, void *o,
                                      float *h_last, void *workspace, int64_t workspace_bytes,
                                      mssm_attention_dims dims, mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    AttentionSizes z;
    if (mssm_status s = check_attention(dims, scale, cu_seqlens != nullptr, dtypes, &z)) return s;
    g_last_variant = MSSM_VARIANT_AUTO;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (z.states == 0) {
        // no sequence covers any row
        if (z.value_bytes && !o) return fail(MSSM_ERR_INVALID_ARG, "o is null");
        const hipError_t e = zero_fill_bytes(o, z.value_bytes, st);
        if (e != hipSuccess) return hip_fail(e, "zero-fill of o");
        return MSSM_OK;
    }
    if (dims.total == 0) {
        const Range ins[] = {range("log_decay", log_decay, dims.heads * 4), range("h0", h0, z.state_bytes),
                             range("cu_seqlens", cu_seqlens, (dims.seqs + 1) * 8)};
        const Range outs[] = {range("h_last", h_last, z.state_bytes)};
        if (mssm_status c = check_overlaps(ins, 3, outs, 1, h0, h_last)) return c;
        return copy_or_zero_state("h_last", h_last, "h0", h0, z.states, st);
    }
    if (!q) return fail(MSSM_ERR_INVALID_ARG, "q is null");
    if (!k) return fail(MSSM_ERR_INVALID_ARG, "k is null");
    if (!v) return fail(MSSM_ERR_INVALID_ARG, "v is null");
    if (!log_decay) return fail(MSSM_ERR_INVALID_ARG, "log_decay is null");
    if (!o) return fail(MSSM_ERR_INVALID_ARG, "o is null");
    mssm::AttentionArgs a = attention_args(dims, dtypes);
    a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.scale = scale; a.h0 = h0; a.cu_seqlens = cu_seqlens;
    a.o = o; a.h_last = h_last;
    Range ws;
    if (mssm_status s = check_workspace(workspace, workspace_bytes, mssm::linear_attention_workspace(a, false), &ws))
        return s;
    const Range ins[] = {range("q", q, z.key_bytes), range("k", k, z.key_bytes), range("v", v, z.value_bytes),
                         range("log_decay", log_decay, dims.heads * 4), range("h0", h0, z.state_bytes),
                         range("cu_seqlens", cu_seqlens, (dims.seqs + 1) * 8)};
    const Range outs[] = {range("o", o, z.value_bytes), range("h_last", h_last, z.state_bytes), ws};
    if (mssm_status c = check_overlaps(ins, 6, outs, 3, h0, h_last)) return c;
    const hipError_t e = mssm::launch_linear_attention_fwd(a, workspace, st);
    if (e != hipSuccess) return hip_fail(e, "linear-attention launch");
    return MSSM_OK;
}

mssm_status mssm_linear_attention_bwd(const void *q, const void *k, const void *v, const float *log_decay,
                                      float scale, const float *h0, const int64_t *cu_seqlens, const void *d_o,
                                      const float *dh_last, void *dq, void *dk, void *dv, float *dh0,
                                      void *workspace, int64_t workspace_bytes, mssm_attention_dims dims,
                                      mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    AttentionSizes z;
    if (mssm_status s = check_attention(dims, scale, cu_seqlens != nullptr, dtypes, &z)) return s;
    g_last_variant = MSSM_VARIANT_AUTO;
    hipStream_t st = static_cast<hipStream_t>(stream);
    Range outs[] = {range("dq", dq, z.key_bytes), range("dk", dk, z.key_bytes), range("dv", dv, z.value_bytes),
                    range("dh0", dh0, z.state_bytes), Range{}};
    if (z.states == 0) {
        if (z.key_bytes && !dq) return fail(MSSM_ERR_INVALID_ARG, "dq is null");
        if (z.key_bytes && !dk) return fail(MSSM_ERR_INVALID_ARG, "dk is null");
        if (z.value_bytes && !dv) return fail(MSSM_ERR_INVALID_ARG, "dv is null");
        if (mssm_status c = check_overlaps(nullptr, 0, outs, 3, nullptr, nullptr)) return c;
        hipError_t e = zero_fill_bytes(dq, z.key_bytes, st);
        if (e == hipSuccess) e = zero_fill_bytes(dk, z.key_bytes, st);
        if (e == hipSuccess) e = zero_fill_bytes(dv, z.value_bytes, st);
        if (e != hipSuccess) return hip_fail(e, "zero-fill of the gradients");
        return MSSM_OK;
    }
    if (dims.total == 0) {
        const Range ins[] = {range("log_decay", log_decay, dims.heads * 4), range("h0", h0, z.state_bytes),
                             range("cu_seqlens", cu_seqlens, (dims.seqs + 1) * 8), range("dh_last", dh_last, z.state_bytes)};
        if (mssm_status c = check_overlaps(ins, 4, &outs[3], 1, nullptr, nullptr)) return c;
        return copy_or_zero_state("dh0", dh0, "dh_last", dh_last, z.states, st);
    }
    if (!q) return fail(MSSM_ERR_INVALID_ARG, "q is null");
    if (!k) return fail(MSSM_ERR_INVALID_ARG, "k is null");
    if (!v) return fail(MSSM_ERR_INVALID_ARG, "v is null");
    if (!log_decay) return fail(MSSM_ERR_INVALID_ARG, "log_decay is null");
    if (!d_o) return fail(MSSM_ERR_INVALID_ARG, "d_o is null");
    if (!dq) return fail(MSSM_ERR_INVALID_ARG, "dq is null");
    if (!dk) return fail(MSSM_ERR_INVALID_ARG, "dk is null");
    if (!dv) return fail(MSSM_ERR_INVALID_ARG, "dv is null");
    mssm::AttentionArgs a = attention_args(dims, dtypes);
    a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.scale = scale; a.h0 = h0; a.cu_seqlens = cu_seqlens;
    a.dout = d_o; a.dh_last = dh_last; a.dq = dq; a.dk = dk; a.dv = dv; a.dh0 = dh0;
    if (mssm_status s = check_workspace(workspace, workspace_bytes, mssm::linear_attention_workspace(a, true), &outs[4]))
        return s;
    const Range ins[] = {range("q", q, z.key_bytes), range("k", k, z.key_bytes), range("v", v, z.value_bytes),
                         range("log_decay", log_decay, dims.heads * 4), range("h0", h0, z.state_bytes),
                         range("cu_seqlens", cu_seqlens, (dims.seqs + 1) * 8), range("d_o", d_o, z.value_bytes),
                         range("dh_last", dh_last, z.state_bytes)};
    if (mssm_status c = check_overlaps(ins, 8, outs, 5, nullptr, nullptr)) return c;
    const hipError_t e = mssm::launch_linear_attention_bwd(a, workspace, st);
    if (e != hipSuccess) return hip_fail(e, "linear-attention backward launch");
    return MSSM_OK;
}

mssm_status mssm_linear_attention_update(float *state, const void *q, const void *k, const void *v,
                                         const float *log_decay, float scale, void *o,
                                         mssm_attention_dims dims, mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    dims.seqlen = 1;
    dims.total = dims.seqs;
    AttentionSizes z;
    if (mssm_status s = check_attention(dims, scale, false, dtypes, &z)) return s;
    g_last_variant = MSSM_VARIANT_AUTO;
    if (z.states == 0) return MSSM_OK;
    if (!state) return fail(MSSM_ERR_INVALID_ARG, "state is null");
    if (!q) return fail(MSSM_ERR_INVALID_ARG, "q is null");
    if (!k) return fail(MSSM_ERR_INVALID_ARG, "k is null");
    if (!v) return fail(MSSM_ERR_INVALID_ARG, "v is null");
    if (!log_decay) return fail(MSSM_ERR_INVALID_ARG, "log_decay is null");
    if (!o) return fail(MSSM_ERR_INVALID_ARG, "o is null");
    mssm::AttentionArgs a = attention_args(dims, dtypes);
    a.q = q; a.k = k; a.v = v; a.log_decay = log_decay; a.scale = scale; a.o = o; a.h_last = state;
    const Range ins[] = {range("q", q, z.key_bytes), range("k", k, z.key_bytes), range("v", v, z.value_bytes),
                         range("log_decay", log_decay, dims.heads * 4)};
    const Range outs[] = {range("o", o, z.value_bytes), range("state", state, z.state_bytes)};
    if (mssm_status c = check_overlaps(ins, 4, outs, 2, nullptr, nullptr)) return c;
    const hipError_t e = mssm::launch_linear_attention_update(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "linear-attention step launch");
    return MSSM_OK;
}

int64_t mssm_linear_attention_workspace(mssm_attention_dims dims, mssm_dtypes dtypes, int backward) {
    g_last_error.clear();
    AttentionSizes z;
    if (check_attention(dims, 0.0f, true, dtypes, &z)) return -1;
    if (z.states == 0 || dims.total == 0) return 0;
    return static_cast<int64_t>(mssm::linear_attention_workspace(attention_args(dims, dtypes), backward != 0));
}

mssm_status mssm_beam_select(const void *logits, const float *scores, float *out_scores, int64_t *out_tokens,
                             int64_t *out_beams, void *workspace, int64_t workspace_bytes,
                             mssm_beam_dims dims, mssm_dtypes dtypes, void *stream) {
    g_last_error.clear();
    if (mssm_status s = check_selection(dims, dtypes)) return s;
    g_last_variant = MSSM_VARIANT_AUTO;
    if (dims.batch == 0) return MSSM_OK;
    if (!logits) return fail(MSSM_ERR_INVALID_ARG, "logits is null");
    if (!scores) return fail(MSSM_ERR_INVALID_ARG, "scores is null");
    if (!out_scores) return fail(MSSM_ERR_INVALID_ARG, "out_scores is null");
    if (!out_tokens) return fail(MSSM_ERR_INVALID_ARG, "out_tokens is null");
    if (!out_beams) return fail(MSSM_ERR_INVALID_ARG, "out_beams is null");
    const mssm::BeamArgs a{logits, scores, out_scores, out_tokens, out_beams, dims.batch, dims.beams, dims.vocab,
                           dims.count, io_type(dtypes)};
    Range ws;
    if (mssm_status s = check_workspace(workspace, workspace_bytes, mssm::beam_select_workspace(a), &ws)) return s;
    const int64_t rows = dims.batch * dims.beams, n = dims.batch * dims.count;
    const Range ins[] = {range("logits", logits, rows * dims.vocab * (dtypes.io == MSSM_F32 ? 4 : 2)),
                         range("scores", scores, rows * 4)};
    const Range outs[] = {range("out_scores", out_scores, n * 4), range("out_tokens", out_tokens, n * 8),
                          range("out_beams", out_beams, n * 8), ws};
    if (mssm_status c = check_overlaps(ins, 2, outs, 4, nullptr, nullptr)) return c;
    const hipError_t e = mssm::launch_beam_select(a, workspace, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "beam-selection launch");
    return MSSM_OK;
}

int64_t mssm_beam_select_workspace(mssm_beam_dims dims, mssm_dtypes dtypes) {
    g_last_error.clear();
    if (check_selection(dims, dtypes)) return -1;
    mssm::BeamArgs a{};
    a.batch = dims.batch; a.beams = dims.beams; a.vocab = dims.vocab; a.count = dims.count;
    return static_cast<int64_t>(mssm::beam_select_workspace(a));
}

mssm_status mssm_state_reorder(void *const *states, const int64_t *row_bytes, int64_t count, const int64_t *origins,
                               mssm_beam_dims dims, void *stream) {
    g_last_error.clear();
    if (mssm_status s = check_beams(dims)) return s;
    if (count < 0) return fail(MSSM_ERR_INVALID_ARG, "negative size (count %lld)", (long long)count);
    g_last_variant = MSSM_VARIANT_AUTO;
    if (dims.batch == 0 || count == 0) return MSSM_OK;
    if (!states) return fail(MSSM_ERR_INVALID_ARG, "states is null");
    if (!row_bytes) return fail(MSSM_ERR_INVALID_ARG, "row_bytes is null");
    if (!origins) return fail(MSSM_ERR_INVALID_ARG, "origins is null");
    const int64_t rows = dims.batch * dims.beams;
    const Range from = range("origins", origins, rows * 8);
    for (int64_t i = 0; i < count; ++i) {
        int64_t bytes;
        if (row_bytes[i] < 0) return fail(MSSM_ERR_INVALID_ARG, "negative size (row_bytes[%lld])", (long long)i);
        if (row_bytes[i] == 0) continue;
        if (!states[i]) return fail(MSSM_ERR_INVALID_ARG, "states[%lld] is null", (long long)i);
        if (!mul_ok(rows, row_bytes[i], &bytes)) return fail(MSSM_ERR_INVALID_ARG, "sizes overflow int64");
        if (row_bytes[i] >= (int64_t(1) << 40) ||
            mssm::state_reorder_blocks(states[i], row_bytes[i]) * dims.batch >= (int64_t(1) << 24))
            return fail(MSSM_ERR_UNSUPPORTED, "states[%lld]: %lld entries of %lld bytes a beam are too large", (long long)i,
                        (long long)dims.batch, (long long)row_bytes[i]);
        const Range mine = range("states", states[i], bytes);
        if (overlaps(mine, from)) return fail(MSSM_ERR_INVALID_ARG, "states[%lld] overlaps origins", (long long)i);
        for (int64_t j = 0; j < i; ++j)
            if (row_bytes[j] && overlaps(mine, range("states", states[j], rows * row_bytes[j])))
                return fail(MSSM_ERR_INVALID_ARG, "states[%lld] overlaps states[%lld]", (long long)i, (long long)j);
    }
    const hipError_t e = mssm::launch_state_reorder(states, row_bytes, count, origins, dims.batch, dims.beams,
                                                    static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "state-reorder launch");
    return MSSM_OK;
}

mssm_variant mssm_force_variant(mssm_variant v) {
    mssm_variant prev = g_forced;
    g_forced = v;
    return prev;
}

mssm_variant mssm_last_variant(void) { return g_last_variant; }

const char *mssm_status_string(mssm_status s) {
    switch (s) {
        case MSSM_OK: return "MSSM_OK";
        case MSSM_ERR_INVALID_ARG: return "MSSM_ERR_INVALID_ARG";
        case MSSM_ERR_UNSUPPORTED: return "MSSM_ERR_UNSUPPORTED";
        case MSSM_ERR_HIP: return "MSSM_ERR_HIP";
        case MSSM_ERR_ALLOC: return "MSSM_ERR_ALLOC";
    }
    return "MSSM_ERR_UNKNOWN";
}

const char *mssm_last_error(void) { return g_last_error.c_str(); }

int mssm_version(void) { return 100; }

mssm_status mssm_device_status(uint32_t *bits, int clear) {
    g_last_error.clear();
    if (!bits) return fail(MSSM_ERR_INVALID_ARG, "bits is null");
    uint32_t more = 0;
    hipError_t e = mssm::device_status(bits, clear != 0);
    if (e == hipSuccess) e = mssm::recurrence_status(&more, clear != 0);
    if (e != hipSuccess) return hip_fail(e, "device status read");
    *bits |= more;
    return MSSM_OK;
}

mssm_status mssm_probe_copy(const void *src, void *dst, int64_t bytes, void *stream) {
    g_last_error.clear();
    if (!src || !dst) return fail(MSSM_ERR_INVALID_ARG, "src and dst must not be null");
    if (bytes <= 0 || bytes % 16 != 0 || bytes >= (int64_t(1) << 43))
        return fail(MSSM_ERR_INVALID_ARG,
                    "bytes must be a positive multiple of 16 below 2^43, got %lld", (long long)bytes);
    if ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 15u)
        return fail(MSSM_ERR_INVALID_ARG, "src and dst must be 16-byte aligned");
    if (overlaps(range("src", src, bytes), range("dst", dst, bytes)))
        return fail(MSSM_ERR_INVALID_ARG, "src and dst overlap");
    const hipError_t e = mssm::launch_probe_copy(src, dst, bytes, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "copy probe launch");
    return MSSM_OK;
}

mssm_status mssm_probe_valu(int op, int32_t iters, float *out, void *stream) {
    g_last_error.clear();
    if (op < MSSM_PROBE_FMA || op > MSSM_PROBE_RCP)
        return fail(MSSM_ERR_INVALID_ARG, "unknown probe operation %d", op);
    if (iters < 1) return fail(MSSM_ERR_INVALID_ARG, "iters must be >= 1");
    if (!out) return fail(MSSM_ERR_INVALID_ARG, "out is null");
    const hipError_t e = mssm::launch_probe_valu(op, iters, out, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "ALU probe launch");
    return MSSM_OK;
}

#ifndef MSSM_SOURCE_HASH
#define MSSM_SOURCE_HASH "unknown"
#endif
const char *mssm_source_hash(void) { return MSSM_SOURCE_HASH; }

}  // extern "C"
