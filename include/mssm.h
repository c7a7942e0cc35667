/*
 * mssm.h -- C ABI of libmssm, the MI355X (gfx950) selective-scan forward.
 *
 * Sources (web pages on selective state-space models, cited by title and
 * section):
 *   [ybb]  "Mamba状态空间模型的硬件感知推理优化：从选择性扫描到并行前缀和"
 *          (ybb.press/llm/14642) -- section 1: recurrence h_t = A h_{t-1} +
 *          B x_t, output y_t = C h_t; section 3.1: one fused kernel computing
 *          the decay exp(A*softplus(dt)), the input term, the scan and
 *          y = C.h + D*x, returning the final state; section 4: the Mamba-2
 *          scalar per-step decay; section 5: chunked walk keeping the state
 *          on chip.
 *   [mhpq] essay at www.mhpq.cn/news/984979 -- section 2.2: zero-order-hold
 *          step A_d = exp(A dt) and the skip term D u; section 2.3: the pair
 *          operator (A1,B1) (+) (A2,B2) = (A2 A1, A2 B1 + B2) whose prefix is
 *          the scan; section 3.1: diagonal A, elementwise exponential.
 *   [csdn] "从硬件感知到算法革命：Mamba如何重塑序列建模的计算效率"
 *          (tencentcloud.csdn.net) -- section 2: Delta = softplus(.), B and C
 *          input-dependent; section 3: SSM output merged with a SiLU gate.
 *   [mlqm] essay at www.mlqm.cn/news/983902 -- section 5.4: token-by-token
 *          decoding keeps only the fixed-size evolving state between steps.
 * [ybb] section 2.1 also writes the recurrence as a product of augmented
 * matrices applied to [h_0; 1], and its section 5 walks the chunks from an
 * initial state h0; [mhpq] section 4.2 keeps the state in a preallocated
 * buffer updated in place.
 *
 * Conventions shared by every entry point:
 *   - Tensor arguments are DEVICE pointers owned by the caller, contiguous in
 *     the stated row-major layouts, 16-byte aligned for the fast path (any
 *     4-byte (f32) / 2-byte (bf16) aligned pointer is accepted).  They must
 *     stay valid until the work queued on `stream` has finished.  The library
 *     keeps no pointer after a call returns.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Calls are
 *     asynchronous: a return of MSSM_OK means the work was queued.  Faults
 *     inside a kernel surface at the caller's next synchronisation.
 *   - Outputs are overwritten, never accumulated into.  Outputs must not
 *     overlap any input (checked on the pointer ranges; MSSM_ERR_INVALID_ARG).
 *   - Validation happens before any HIP call.  On failure nothing is queued,
 *     the status is returned and mssm_last_error() (thread-local) describes
 *     it.  No call aborts, throws or prints.
 *   - Arithmetic is float32 with float32 state whatever the I/O dtype; bf16
 *     outputs are rounded to nearest even.
 *   - Scratch memory, where a kernel variant needs it, is allocated and freed
 *     stream-ordered on `stream` from a memory pool the library creates per
 *     device (hipMallocFromPoolAsync/hipFreeAsync).  The pool keeps freed
 *     memory for later calls (its release threshold is unlimited), so it
 *     holds up to the largest scratch in use at once until the process ends.
 */
#ifndef MSSM_H
#define MSSM_H

#include <stdint.h>

#if defined(MSSM_BUILDING_LIBRARY)
#define MSSM_API __attribute__((visibility("default")))
#else
#define MSSM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MSSM_OK = 0,
    MSSM_ERR_INVALID_ARG = 1,   /* null required pointer, bad dims, aliasing   */
    MSSM_ERR_UNSUPPORTED = 2,   /* valid but outside this build's limits       */
    MSSM_ERR_HIP = 3,           /* a HIP runtime call or launch failed          */
    MSSM_ERR_ALLOC = 4          /* scratch allocation failed                    */
} mssm_status;

typedef enum {
    MSSM_F32 = 0,
    MSSM_BF16 = 1
} mssm_dtype;

/* Kernel variant selection (for tests and tuning; AUTO picks by shape). */
typedef enum {
    MSSM_VARIANT_AUTO = 0,
    MSSM_VARIANT_ROWSERIAL = 1, /* one lane per (b,d) row, whole-L serial walk */
    MSSM_VARIANT_CHUNKED = 2,   /* lanes over (row, n), L walked in chunks     */
    MSSM_VARIANT_LOOKBACK = 3,  /* L split across workgroups, decoupled carry  */
    MSSM_VARIANT_SSD_RECURRENT = 4,
    MSSM_VARIANT_SSD_CHUNKED = 5,
    MSSM_VARIANT_PAIRSCAN = 6,  /* steps of a chunk split across lanes: pair
                                   scan across rows, N <= 16, no prologue   */
    MSSM_VARIANT_PAIRSCAN2 = 7  /* the same with two slices of waves per
                                   chunk, combined through LDS               */
} mssm_variant;

/* Sizes of a selective-scan problem. */
typedef struct {
    int64_t batch;   /* >= 0 */
    int64_t seqlen;  /* L >= 0 */
    int64_t dim;     /* channels D >= 0 */
    int64_t dstate;  /* state size N, 1 <= N <= MSSM_MAX_DSTATE */
} mssm_scan_dims;

/* Storage dtypes.  `io` covers the activations (u, delta, B, C, z, y; for
 * SSD x, dt, B, C, y).  `param` covers A, D, delta_bias / dt_bias and must
 * be MSSM_F32.  h_last is always float32. */
typedef struct {
    int32_t io;      /* mssm_dtype */
    int32_t param;   /* mssm_dtype, MSSM_F32 only */
} mssm_dtypes;

#define MSSM_MAX_DSTATE 64      /* selective scan: largest N this build runs */
#define MSSM_SSD_MAX_DSTATE 256 /* SSD: largest N */
#define MSSM_SSD_MAX_HEADDIM 256

/*
 * Selective-scan forward ([ybb] sections 1, 3.1; [mhpq] sections 2.2-2.3,
 * 3.1; [csdn] sections 2-3).  For every batch b and channel d, from h = 0:
 *
 *   dl        = softplus(delta[b,d,t] + delta_bias[d])
 *   h[n]      = exp(dl * A[d,n]) * h[n] + dl * B[b,n,t] * u[b,d,t]
 *   y[b,d,t]  = (sum_n C[b,n,t] * h[n] + D[d] * u[b,d,t]) * silu(z[b,d,t])
 *   h_last[b,d,n] = h[n] after t = L-1
 *
 * The recurrence is evaluated as a parallel scan over the pair operator
 * (a1,b1) (+) (a2,b2) = (a2 a1, a2 b1 + b2); the result equals the
 * sequential loop up to float32 rounding order.
 *
 * Arguments (device pointers unless stated):
 *   u, delta   (batch, dim, L), dtype `io`           required
 *   delta_bias (dim) float32                         nullable -> 0
 *   A          (dim, N) float32 (expected < 0)       required
 *   B, C       (batch, N, L), dtype `io`             required
 *   D          (dim) float32                         nullable -> no skip term
 *   z          (batch, dim, L), dtype `io`           nullable -> no gate
 *   y          (batch, dim, L), dtype `io`           required (output)
 *   h_last     (batch, dim, N) float32               nullable (output)
 * Errors: MSSM_ERR_INVALID_ARG for a null required pointer, a negative
 * size, N < 1, an unknown dtype, or an output overlapping an input;
 * MSSM_ERR_UNSUPPORTED for N > MSSM_MAX_DSTATE or param dtype != F32.
 * batch == 0 or dim == 0: nothing to do, MSSM_OK.  L == 0: h_last is
 * zero-filled, y is empty.
 */
MSSM_API mssm_status mssm_selective_scan_fwd(const void *u, const void *delta,
                                    const float *delta_bias, const float *A,
                                    const void *B, const void *C,
                                    const float *D, const void *z, void *y,
                                    float *h_last, mssm_scan_dims dims,
                                    mssm_dtypes dtypes, void *stream);

/*
 * The selective-scan forward fed by its convolution prologue ([csdn]
 * section 3: a local convolution and a SiLU precede the selective SSM in the
 * Mamba block, kernel size 4; [mlqm] section 3.3: d_conv = 4).  The scan
 * input is formed on chip from x and never stored:
 *
 *   u[b,d,t] = silu(conv_b[d] + sum_{k=0..3} conv_w[d,k] * x[b,d,t-3+k])
 *
 * with x = 0 before step 0 (a causal, zero-padded depthwise convolution);
 * then the selective scan of mssm_selective_scan_fwd_h0 on u, including
 * the skip term D[d] * u.
 *
 *   x       (batch, dim, L), dtype `io`        required (the prologue input)
 *   conv_w  (dim, MSSM_CONV_WIDTH) float32     required
 *   conv_b  (dim) float32                      nullable -> 0
 * Everything else (delta ... h_last, errors, variants) is as for
 * mssm_selective_scan_fwd_h0; h0 does not carry the convolution's window,
 * so a continued sequence restarts it from zero.
 */
#define MSSM_CONV_WIDTH 4
MSSM_API mssm_status mssm_selective_scan_fwd_conv(const void *x, const float *conv_w,
                                         const float *conv_b, const void *delta,
                                         const float *delta_bias, const float *A,
                                         const void *B, const void *C,
                                         const float *D, const void *z,
                                         const float *h0, void *y, float *h_last,
                                         mssm_scan_dims dims, mssm_dtypes dtypes,
                                         void *stream);

/*
 * Backward of the selective scan (the reverse-mode derivative of
 * mssm_selective_scan_fwd_h0; [mlqm] section 3.2: the block is trained,
 * forward and backward).  Given the forward's inputs and the gradients of a
 * loss with respect to y (dy) and h_last (dh_last), it writes the loss's
 * gradients with respect to every input.  The states are recomputed from
 * the inputs (stored every few steps in stream-ordered scratch), not read
 * from the forward.
 *
 * Inputs: u ... h0 as for mssm_selective_scan_fwd_h0;
 *   dy       (batch, dim, L), dtype `io`     required
 *   dh_last  (batch, dim, N) float32         nullable -> 0
 * Outputs, all float32 whatever the I/O dtype (like h_last):
 *   du, ddelta    (batch, dim, L) float32      required
 *   dz            (batch, dim, L) float32      nullable; needs z
 *   dB, dC        (batch, N, L) float32        nullable
 *   dA            (dim, N) float32             nullable
 *   dD, ddelta_bias (dim) float32              nullable (gradients at D
 *                                              = 0 / bias = 0 when those
 *                                              inputs are null)
 *   dh0           (batch, dim, N) float32      nullable
 * dB and dC sum over channels in a fixed order (deterministic); dA, dD and
 * ddelta_bias sum over batches with float32 atomic additions, so their last
 * bits depend on the order.  Scratch is allocated and freed stream-ordered:
 * the states every 16 steps (batch * dim * ceil(L / 16) * 64 bytes for
 * N <= 16) and, when dB or dC is requested,
 * per-wave partial sums of about batch * dim / 8 * L * 128 bytes for
 * 8 < N <= 16 (half that for N <= 8; 4.3 GB for L = 2^20 with 256
 * channels); an allocation failure returns MSSM_ERR_ALLOC.  Errors as for
 * the forward, plus MSSM_ERR_INVALID_ARG for dz without z or any output
 * overlapping an input or another output.
 */
MSSM_API mssm_status mssm_selective_scan_bwd(const void *u, const void *delta,
                                    const float *delta_bias, const float *A,
                                    const void *B, const void *C, const float *D,
                                    const void *z, const float *h0, const void *dy,
                                    const float *dh_last, float *du, float *ddelta,
                                    float *ddelta_bias, float *dA, float *dB,
                                    float *dC, float *dD, float *dz, float *dh0,
                                    mssm_scan_dims dims, mssm_dtypes dtypes,
                                    void *stream);

/* Sizes of a Mamba-2 scalar-decay (SSD) problem. */
typedef struct {
    int64_t batch;
    int64_t seqlen;   /* L */
    int64_t nheads;   /* H */
    int64_t headdim;  /* P, 1 <= P <= MSSM_SSD_MAX_HEADDIM */
    int64_t dstate;   /* N, 1 <= N <= MSSM_SSD_MAX_DSTATE */
    int64_t ngroups;  /* G >= 1, H % G == 0; head h reads group h / (H/G) */
    int64_t chunk;    /* chunk length of the matrix-core form; 0 -> 256 */
} mssm_ssd_dims;

/*
 * Mamba-2 scalar-decay forward ([ybb] section 4: one decay per step and head,
 * shared by all state elements; section 6.2: cumulative products taken in
 * log space).  For every batch b and head h (group g), from S = 0:
 *
 *   dl          = softplus(dt[b,t,h] + dt_bias[h])
 *   S[p][n]     = exp(dl * A[h]) * S[p][n] + dl * x[b,t,h,p] * B[b,t,g,n]
 *   y[b,t,h,p]  = sum_n C[b,t,g,n] * S[p][n] + D[h] * x[b,t,h,p]
 *   h_last[b,h,p,n] = S[p][n] after t = L-1
 *
 * Arguments (device pointers unless stated):
 *   x        (batch, L, H, P), dtype `io`     required
 *   dt       (batch, L, H),    dtype `io`     required
 *   dt_bias  (H) float32                      nullable -> 0
 *   A        (H) float32                      required
 *   B, C     (batch, L, G, N), dtype `io`     required
 *   D        (H) float32                      nullable -> no skip term
 *   y        (batch, L, H, P), dtype `io`     required (output)
 *   h_last   (batch, H, P, N) float32         nullable (output)
 * Errors as for mssm_selective_scan_fwd; also MSSM_ERR_INVALID_ARG when
 * H % G != 0 or chunk < 0, MSSM_ERR_UNSUPPORTED beyond the P/N limits.
 */
MSSM_API mssm_status mssm_ssd_scalar_fwd(const void *x, const void *dt,
                                const float *dt_bias, const float *A,
                                const void *B, const void *C, const float *D,
                                void *y, float *h_last, mssm_ssd_dims dims,
                                mssm_dtypes dtypes, void *stream);

/*
 * Both forwards from a given initial state ([ybb] sections 2.1 and 5): the
 * recurrence starts at h0 instead of 0, so a long sequence can be processed
 * in pieces, each call continuing from the h_last of the previous one.
 *
 *   h0  (batch, dim, N) float32 for the selective scan,
 *       (batch, H, P, N) float32 for SSD          nullable -> 0
 *
 * h0 may be the very buffer passed as h_last (same pointer): the state is
 * then advanced in place.  Any other overlap of h0 with an output is
 * MSSM_ERR_INVALID_ARG.  L == 0 copies h0 to h_last.  Everything else --
 * layouts, variants, errors -- is as for the entry points without h0, which
 * equal these with h0 = NULL.
 */
MSSM_API mssm_status mssm_selective_scan_fwd_h0(const void *u, const void *delta,
                                       const float *delta_bias, const float *A,
                                       const void *B, const void *C,
                                       const float *D, const void *z,
                                       const float *h0, void *y, float *h_last,
                                       mssm_scan_dims dims, mssm_dtypes dtypes,
                                       void *stream);
MSSM_API mssm_status mssm_ssd_scalar_fwd_h0(const void *x, const void *dt,
                                   const float *dt_bias, const float *A,
                                   const void *B, const void *C, const float *D,
                                   const float *h0, void *y, float *h_last,
                                   mssm_ssd_dims dims, mssm_dtypes dtypes,
                                   void *stream);

/*
 * mssm_selective_scan_fwd_h0 for callers that cannot allocate device memory:
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation.  It calls no hipMalloc, hipMallocAsync, hipFree or other
 * allocating routine.  The look-back variant's scratch (its published
 * carries, flags and work ticket) lives in a fixed device array of
 * MSSM_NOALLOC_SCRATCH_BYTES on each device the library runs on, held until
 * the process ends; the other variants need no scratch.  The flags and the
 * ticket are cleared by a kernel at the start of each call.
 *
 * Arguments, layouts, variants and results are those of
 * mssm_selective_scan_fwd_h0 (bitwise the same outputs).  The caller still
 * provides every input and output.
 * Limit: a problem whose look-back scratch exceeds the array returns
 * MSSM_ERR_UNSUPPORTED before anything is queued (the look-back variant
 * needs about 2 KB per (segment, 16-channel group) for N <= 16 and up to
 * 8 KB for larger N, with about 768 of them when AUTO chooses it: 1.5 MB for
 * a million-step sequence of 256 channels).
 * Every call on a device shares that device's array, so calls that overlap
 * on one device (on different streams or threads) race and must be
 * serialised by the caller.
 */
#define MSSM_NOALLOC_SCRATCH_BYTES (8u << 20)
MSSM_API mssm_status mssm_selective_scan_fwd_h0_noalloc(const void *u, const void *delta,
                                               const float *delta_bias, const float *A,
                                               const void *B, const void *C,
                                               const float *D, const void *z,
                                               const float *h0, void *y, float *h_last,
                                               mssm_scan_dims dims, mssm_dtypes dtypes,
                                               void *stream);

/*
 * The SSD forward with a SiLU gate on its output ([csdn] section 3: a SiLU
 * branch gates the SSM output; the same reading as the selective scan's z):
 *
 *   y[b,t,h,p] = (sum_n C[b,t,g,n] * S[p][n] + D[h] * x[b,t,h,p]) * silu(z[b,t,h,p])
 *
 *   z    (batch, L, H, P), dtype `io`, like x   nullable -> no gate
 *   h0   (batch, H, P, N) float32               nullable -> 0 (as in the
 *                                               _h0 entry point)
 * Everything else is as for mssm_ssd_scalar_fwd_h0, which equals this with
 * z = NULL.
 */
MSSM_API mssm_status mssm_ssd_scalar_fwd_gated(const void *x, const void *dt,
                                      const float *dt_bias, const float *A,
                                      const void *B, const void *C,
                                      const float *D, const void *z,
                                      const float *h0, void *y, float *h_last,
                                      mssm_ssd_dims dims, mssm_dtypes dtypes,
                                      void *stream);

/* Sizes of one decode step. */
typedef struct {
    int64_t batch;   /* >= 0 */
    int64_t dim;     /* channels D >= 0 */
    int64_t dstate;  /* state size N, 1 <= N <= MSSM_MAX_DSTATE */
} mssm_step_dims;

/*
 * One decode step of the selective scan ([mlqm] section 5.4: incremental
 * decoding carries only the fixed-size state; [mhpq] section 4.2: the state
 * cache is a preallocated buffer; the step itself is the recurrence of
 * mssm_selective_scan_fwd at a single time t):
 *
 *   dl              = softplus(dt[b,d] + dt_bias[d])
 *   state[b,d,n]    = exp(dl * A[d,n]) * state[b,d,n] + dl * B[b,n] * x[b,d]
 *   y[b,d]          = (sum_n C[b,n] * state[b,d,n] + D[d] * x[b,d]) * silu(z[b,d])
 *
 * It equals mssm_selective_scan_fwd_h0 with L = 1 and h0 = h_last = state.
 *
 * Arguments (device pointers unless stated):
 *   state    (batch, dim, N) float32       required, read and overwritten
 *   x, dt    (batch, dim), dtype `io`      required
 *   dt_bias  (dim) float32                 nullable -> 0
 *   A        (dim, N) float32              required
 *   B, C     (batch, N), dtype `io`        required
 *   D        (dim) float32                 nullable -> no skip term
 *   z        (batch, dim), dtype `io`      nullable -> no gate
 *   y        (batch, dim), dtype `io`      required (output)
 * Errors: as for mssm_selective_scan_fwd; state and y must not overlap any
 * input or each other.  batch == 0 or dim == 0: nothing to do, MSSM_OK.
 */
MSSM_API mssm_status mssm_selective_state_update(float *state, const void *x,
                                        const void *dt, const float *dt_bias,
                                        const float *A, const void *B,
                                        const void *C, const float *D,
                                        const void *z, void *y,
                                        mssm_step_dims dims, mssm_dtypes dtypes,
                                        void *stream);

/*
 * Workspaces.  The calls below that need scratch take it from the caller:
 * `workspace` is a device buffer of at least `workspace_bytes` bytes, as the
 * matching _workspace query says, 256-byte aligned, that overlaps no operand
 * and may be reused once the call's work on the stream has finished.  A call
 * then allocates nothing, so it may be captured into a HIP graph.  With
 * workspace NULL the call takes its scratch stream-ordered from the library's
 * pool.  Queries return the bytes (0: none needed), or -1 for sizes or dtypes
 * that the call would refuse (mssm_last_error() says why); they need no GPU.
 * A workspace that is too small or misaligned is MSSM_ERR_INVALID_ARG.
 */

/* Sizes of a layer norm: `rows` independent rows of `dim` values. */
typedef struct {
    int64_t rows;    /* >= 0 */
    int64_t dim;     /* >= 0 */
} mssm_norm_dims;

/*
 * Layer norm in front of a layer.  For every row:
 *
 *   mean     = sum_d x[d] / dim
 *   rstd     = 1 / sqrt(sum_d (x[d] - mean)^2 / dim + eps)
 *   y[d]     = (x[d] - mean) * rstd * weight[d] + bias[d]
 *
 * The variance is summed from the differences to the mean, in float32.
 *
 * Arguments (device pointers unless stated):
 *   x        (rows, dim), dtype `io`       required
 *   weight   (dim) float32                 nullable -> 1
 *   bias     (dim) float32                 nullable -> 0
 *   eps      (host) >= 0 and finite
 *   y        (rows, dim), dtype `io`       required (output)
 *   mean, rstd  (rows) float32             nullable (outputs, read by the
 *                                          backward)
 * Errors: MSSM_ERR_INVALID_ARG for a null required pointer, a negative size,
 * an unknown dtype, eps < 0 or not finite, or an output overlapping an input
 * or another output; MSSM_ERR_UNSUPPORTED for param dtype != F32 or
 * rows >= 2^31 or dim >= 2^31.  rows == 0 or dim == 0: nothing to do, MSSM_OK.
 */
MSSM_API mssm_status mssm_layer_norm_fwd(const void *x, const float *weight,
                                const float *bias, float eps, void *y,
                                float *mean, float *rstd, mssm_norm_dims dims,
                                mssm_dtypes dtypes, void *stream);

/*
 * Backward of the layer norm.  With xhat = (x - mean) * rstd and
 * e[d] = dy[d] * weight[d], per row:
 *
 *   dx[d]      = rstd * (e[d] - mean_d(e) - xhat[d] * mean_d(e * xhat))
 *   dweight[d] = sum_rows dy[d] * xhat[d],   dbias[d] = sum_rows dy[d]
 *
 *   dy, x       (rows, dim), dtype `io`    required
 *   mean, rstd  (rows) float32             required (of the forward)
 *   weight      (dim) float32              nullable -> 1
 *   dx          (rows, dim), dtype `io`    required (output)
 *   dweight, dbias  (dim) float32          nullable (outputs)
 * dweight and dbias are summed in an order that depends on the sizes alone
 * (repeatable bit for bit), through partial sums in the workspace.
 * rows == 0 zero-fills dweight and dbias.  Errors as for the forward.
 */
MSSM_API mssm_status mssm_layer_norm_bwd(const void *dy, const void *x,
                                const float *mean, const float *rstd,
                                const float *weight, void *dx, float *dweight,
                                float *dbias, void *workspace,
                                int64_t workspace_bytes, mssm_norm_dims dims,
                                mssm_dtypes dtypes, void *stream);
MSSM_API int64_t mssm_layer_norm_bwd_workspace(mssm_norm_dims dims, mssm_dtypes dtypes);

/* Sizes of a gated linear recurrence. */
typedef struct {
    int64_t batch;   /* >= 0 */
    int64_t seqlen;  /* L >= 0 (ignored by the single-step update) */
    int64_t dim;     /* channels >= 0 */
} mssm_recurrence_dims;

/*
 * Gated linear recurrence: one decay per step and channel, both gates formed
 * from inputs.  For every batch b and channel d, from h = h0:
 *
 *   log a_t   = -scale * softplus(lam[d]) * sigmoid(r[b,t,d])
 *   h         = a_t * h + sqrt(1 - a_t^2) * sigmoid(i[b,t,d]) * x[b,t,d]
 *   y[b,t,d]  = h;   h_last[b,d] = h after t = L-1
 *
 * 1 - a_t^2 is formed from a_t - 1 = expm1(log a_t), so that decays next to 1
 * lose nothing; fast decays keep their relative precision too.
 *
 * Arguments (device pointers unless stated):
 *   x, r, i  (batch, L, dim), dtype `io`   required (r, i before the sigmoid)
 *   lam      (dim) float32                 required
 *   scale    (host) >= 0 and finite
 *   h0       (batch, dim) float32          nullable -> 0; may be the very
 *                                          buffer passed as h_last
 *   y        (batch, L, dim), dtype `io`   required (output)
 *   h_last   (batch, dim) float32          nullable (output)
 * Long sequences are cut into segments whose carries pass between workgroups
 * in a fixed association (through the workspace): results are repeatable bit
 * for bit.
 * Errors as for mssm_selective_scan_fwd; also MSSM_ERR_INVALID_ARG for a scale
 * that is negative or not finite, MSSM_ERR_UNSUPPORTED for dim >= 2^21, for
 * another size or batch * dim >= 2^31, or where the sequences hold 2^30 or more
 * segments of 64 channels by 88 steps (66 for float32 or an odd dim).
 * batch == 0 or dim == 0: nothing to do, MSSM_OK.  L == 0: h_last receives h0
 * (or zeros), y is empty.
 */
MSSM_API mssm_status mssm_gated_recurrence_fwd(const void *x, const void *r,
                                const void *i, const float *lam, float scale,
                                const float *h0, void *y, float *h_last,
                                void *workspace, int64_t workspace_bytes,
                                mssm_recurrence_dims dims, mssm_dtypes dtypes,
                                void *stream);
/* For the forward (backward == 0) or the backward. */
MSSM_API int64_t mssm_gated_recurrence_workspace(mssm_recurrence_dims dims,
                                mssm_dtypes dtypes, int backward);

/*
 * Backward of the gated linear recurrence, given its inputs, its output y
 * (the states, in dtype `io`) and the gradients dy and dh_last.  With
 * m = sqrt(1 - a^2) and g_t = dy_t + a_{t+1} g_{t+1} (dh_last added at the
 * last step):
 *
 *   w    = g h_{t-1} a log(a) - g sigmoid(i) x a^2 (log(a) / m)
 *   dx   = g m sigmoid(i)          di = g m sigmoid(i) x (1 - sigmoid(i))
 *   dr   = w (1 - sigmoid(r))      dlam = sum w * sigmoid(lam) / softplus(lam)
 *   dh0  = a_0 g_0
 *
 * log(a) / m tends to 0 with log(a) and is taken as 0 where m is 0.
 *
 *   y, dy       (batch, L, dim), dtype `io`   required
 *   dh_last     (batch, dim) float32          nullable -> 0
 *   dx, dr, di  (batch, L, dim), dtype `io`   required (outputs)
 *   dlam        (dim) float32                 nullable (output)
 *   dh0         (batch, dim) float32          nullable (output)
 * dlam is summed in a fixed order (repeatable bit for bit), through partial
 * sums in the workspace.  L == 0: dlam is zero, dh0 = dh_last.  Errors as for
 * the forward; no output may overlap an input or another output.
 */
MSSM_API mssm_status mssm_gated_recurrence_bwd(const void *x, const void *r,
                                const void *i, const float *lam, float scale,
                                const float *h0, const void *y, const void *dy,
                                const float *dh_last, void *dx, void *dr,
                                void *di, float *dlam, float *dh0,
                                void *workspace, int64_t workspace_bytes,
                                mssm_recurrence_dims dims, mssm_dtypes dtypes,
                                void *stream);

/*
 * One decode step of the gated linear recurrence on a cached state, in
 * place: the forward at L = 1 with h0 = h_last = state.
 *
 *   state    (batch, dim) float32          required, read and overwritten
 *   x, r, i  (batch, dim), dtype `io`      required
 *   y        (batch, dim), dtype `io`      required (output)
 * Errors as for the forward; state and y must not overlap any input or each
 * other.
 */
MSSM_API mssm_status mssm_gated_recurrence_update(float *state, const void *x,
                                const void *r, const void *i, const float *lam,
                                float scale, void *y,
                                mssm_recurrence_dims dims, mssm_dtypes dtypes,
                                void *stream);

/* Sizes of a cross entropy over a vocabulary projection. */
typedef struct {
    int64_t tokens;  /* T >= 0 */
    int64_t dim;     /* width of the hidden states, >= 1 */
    int64_t vocab;   /* V >= 1 */
} mssm_loss_dims;

/*
 * Softmax cross entropy of a projection onto a vocabulary, the logits formed
 * in pieces on chip and never stored.  For every token t:
 *
 *   l[v]    = sum_d hidden[t,d] * weight[v,d]
 *   lse[t]  = log sum_v exp(l[v])
 *   loss[t] = lse[t] - l[targets[t]]      0 where targets[t] == ignore_index
 *
 * A target outside [0, vocab) that is not ignore_index reads nothing out of
 * range: its loss is NaN.  A logit of +infinity makes lse, and the loss of every
 * other word, infinite.
 *
 * Arguments (device pointers unless stated):
 *   hidden   (tokens, dim), dtype `io`     required
 *   weight   (vocab, dim), dtype `io`      required
 *   targets  (tokens) int64                required
 *   loss     (tokens) float32              required (output)
 *   lse      (tokens) float32              nullable (output, read by the
 *                                          backward)
 * Logits are float32 sums of exact products (bf16) or float32 products.
 * Errors: as for mssm_layer_norm_fwd; also MSSM_ERR_INVALID_ARG for dim < 1 or
 * vocab < 1, MSSM_ERR_UNSUPPORTED for tokens >= 2^20, vocab >= 2^30 or
 * dim >= 2^20.  tokens == 0: nothing to do, MSSM_OK.  The workspace holds the
 * pieces' maxima and sums and, where a row of dim values is not a multiple of
 * 16 bytes or an address is not 16-byte aligned, an aligned copy of hidden and
 * of a piece of weight.
 */
MSSM_API mssm_status mssm_linear_cross_entropy_fwd(const void *hidden,
                                const void *weight, const int64_t *targets,
                                int64_t ignore_index, float *loss, float *lse,
                                void *workspace, int64_t workspace_bytes,
                                mssm_loss_dims dims, mssm_dtypes dtypes,
                                void *stream);
/* For the forward (backward == 0) or the backward; `aligned`: nonzero when
 * hidden and weight start on 16-byte boundaries. */
MSSM_API int64_t mssm_linear_cross_entropy_workspace(mssm_loss_dims dims,
                                mssm_dtypes dtypes, int backward, int aligned);

/*
 * Backward of the projected cross entropy.  With
 * p[t,v] = (exp(l[t,v] - lse[t]) - [v == targets[t]]) * dloss[t]
 * (0 for ignored tokens, whatever their hidden state and dloss hold):
 *
 *   dhidden[t,:] = sum_v p[t,v] * weight[v,:]
 *   dweight[v,:] = sum_t p[t,v] * hidden[t,:]
 *
 *   lse      (tokens) float32              required (of the forward)
 *   dloss    (tokens) float32              required
 *   dhidden  (tokens, dim), dtype `io`     required (output)
 *   dweight  (vocab, dim), dtype `io`      required (output)
 * The logits are formed again, a piece of the vocabulary at a time; p is held
 * in dtype `io` for that piece only.  Sums are float32 in a fixed order
 * (repeatable bit for bit).  A target outside [0, vocab) that is not
 * ignore_index makes that token's dhidden and its terms of dweight NaN.
 * The workspace does not grow with the vocabulary past one piece of it.
 * tokens == 0 zero-fills dweight.  Errors as
 * for the forward.
 */
MSSM_API mssm_status mssm_linear_cross_entropy_bwd(const void *hidden,
                                const void *weight, const int64_t *targets,
                                int64_t ignore_index, const float *lse,
                                const float *dloss, void *dhidden,
                                void *dweight, void *workspace,
                                int64_t workspace_bytes, mssm_loss_dims dims,
                                mssm_dtypes dtypes, void *stream);

/* Largest head of the norm with rotation and of the linear attention, most
 * beams of an entry and most candidates of a selection. */
#define MSSM_MAX_HEAD_DIM 256
#define MSSM_MAX_BEAMS 32
#define MSSM_MAX_BEAM_COUNT 64

/* Sizes of a norm of queries and keys with their rotation. */
typedef struct {
    int64_t tokens;   /* >= 0 */
    int64_t q_heads;  /* >= 0 */
    int64_t k_heads;  /* >= 0 */
    int64_t dim;      /* of a head, 1 <= dim <= MSSM_MAX_HEAD_DIM */
    int64_t rotary;   /* values of a head that are rotated: even, 0 <= rotary <= dim */
} mssm_head_norm_dims;

/*
 * Norm of queries and keys for each head, with their rotation by position in
 * the same pass.  For every token and head x, with R = rotary:
 *
 *   n[d]       = x[d] * weight[d] / sqrt(sum_d x[d]^2 / dim + eps)
 *   a[j]       = positions[token] * base^(-2 j / R)            j < R/2
 *   y[j]       = n[j] cos a[j] - n[j + R/2] sin a[j]
 *   y[j + R/2] = n[j + R/2] cos a[j] + n[j] sin a[j];   y[d] = n[d] for d >= R
 *
 * Angles are formed in float64 and reduced to a fraction of a turn, so far
 * positions keep their digits.
 *
 * Arguments (device pointers unless stated):
 *   q          (tokens, q_heads, dim), dtype `io`   required
 *   k          (tokens, k_heads, dim), dtype `io`   required
 *   positions  (tokens) int64                       required (any value) if
 *                                                   rotary > 0
 *   q_weight, k_weight  (dim) float32               nullable -> 1
 *   base       (host) > 0 and finite
 *   eps        (host) >= 0 and finite
 *   q_out, k_out  like q and k                      required (outputs)
 * Operands with no elements may be null.
 * Errors: MSSM_ERR_INVALID_ARG for a null required pointer, a negative size,
 * dim < 1, a rotary that is odd or outside [0, dim], an unknown dtype, a bad
 * base or eps, or an output overlapping an input or another output;
 * MSSM_ERR_UNSUPPORTED for param dtype != F32, dim > MSSM_MAX_HEAD_DIM,
 * heads >= 2^23, tokens >= 2^31 or tokens * heads >= 2^31.  No elements: nothing to do, MSSM_OK.
 */
MSSM_API mssm_status mssm_qk_norm_rotary_fwd(const void *q, const void *k,
                                const int64_t *positions,
                                const float *q_weight, const float *k_weight,
                                double base, float eps, void *q_out,
                                void *k_out, mssm_head_norm_dims dims,
                                mssm_dtypes dtypes, void *stream);

/*
 * Backward of the norm with rotation, for the gradients dq_out and dk_out of
 * its outputs; the norms are formed again.  With dn the gradient turned back by
 * the token's angles, r = 1 / sqrt(mean(x^2) + eps) and e = dn * weight, per head:
 *
 *   dx[d]      = r * (e[d] - x[d] * r^2 * mean_d(e * x))
 *   dweight[d] = sum over tokens and heads of dn[d] * x[d] * r
 *
 *   dq_out, dk_out  like q and k                    required
 *   dq, dk          like q and k                    required (outputs)
 *   dq_weight, dk_weight  (dim) float32             nullable (outputs)
 * The weights' gradients are summed in an order that depends on the sizes
 * alone (repeatable bit for bit), through partial sums in the workspace; they
 * are zero without tokens.  Errors as for the forward.
 */
MSSM_API mssm_status mssm_qk_norm_rotary_bwd(const void *dq_out, const void *dk_out,
                                const void *q, const void *k,
                                const int64_t *positions,
                                const float *q_weight, const float *k_weight,
                                double base, float eps, void *dq, void *dk,
                                float *dq_weight, float *dk_weight,
                                void *workspace, int64_t workspace_bytes,
                                mssm_head_norm_dims dims, mssm_dtypes dtypes,
                                void *stream);
MSSM_API int64_t mssm_qk_norm_rotary_bwd_workspace(mssm_head_norm_dims dims,
                                mssm_dtypes dtypes);

/* Sizes of a linear attention. */
typedef struct {
    int64_t seqs;    /* sequences >= 0 */
    int64_t seqlen;  /* steps of each >= 0; with cu_seqlens the longest one's,
                        or an estimate: longer ones come out right, slower */
    int64_t total;   /* rows of q, k, v: seqs * seqlen, or of the packed tensors */
    int64_t heads;   /* >= 0 */
    int64_t key;     /* values of a query or key head, 1 <= key <= MSSM_MAX_HEAD_DIM */
    int64_t value;   /* values of a value head, 1 <= value <= MSSM_MAX_HEAD_DIM */
} mssm_attention_dims;

/*
 * Linear attention with a decay per head.  For every sequence and head, from
 * S = h0:
 *
 *   S   = exp(log_decay[h]) * S + k[t] v[t]^T          (key, value)
 *   o[t] = scale * S^T q[t];   h_last = S after the last step
 *
 * Arguments (device pointers unless stated):
 *   q, k       (total, heads, key), dtype `io`      required
 *   v          (total, heads, value), dtype `io`    required
 *   log_decay  (heads) float32                      required, expected <= 0
 *   scale      (host) finite
 *   h0         (seqs, heads, key, value) float32    nullable -> 0; may be the
 *                                                   very buffer passed as h_last
 *   cu_seqlens (seqs + 1) int64                     nullable: sequence b is rows
 *              cu_seqlens[b] .. cu_seqlens[b + 1] - 1; null: rows b * seqlen on.
 *              Offsets have to rise from 0 or more to at most total; others are
 *              held to that range, so that nothing outside is read or written.
 *   o          (total, heads, value), dtype `io`    required (output); rows in
 *              front of the first and behind the last sequence are set to 0
 *   h_last     (seqs, heads, key, value) float32    nullable (output)
 * A sequence of no steps has h_last = h0.  Sequences are walked in chunks whose
 * products run on the matrix cores: float32 sums of exact products of bfloat16
 * values; where `io` is bfloat16 what is not (the decayed products q.k of a chunk,
 * the state as it meets q, the decayed v) enters as the sum of two or three of them,
 * 2^-18 off or less, so that results are off by their own storage.  The state itself is
 * carried in float32.  Results are repeatable bit for bit.  A v that is infinite or NaN
 * makes its own column NaN from its step on in o, and not finite in the state; a q or k
 * that is not finite reaches what the formula says it does, as infinities or NaN.
 * Errors as for mssm_selective_scan_fwd; also MSSM_ERR_INVALID_ARG for a scale
 * that is not finite, key or value < 1, or total != seqs * seqlen without
 * cu_seqlens; MSSM_ERR_UNSUPPORTED for key or value > MSSM_MAX_HEAD_DIM,
 * heads >= 2^15, seqs or seqs * heads >= 2^20, total or seqlen >= 2^31.  seqs == 0 or
 * heads == 0: o is zeroed.
 */
MSSM_API mssm_status mssm_linear_attention_fwd(const void *q, const void *k,
                                const void *v, const float *log_decay,
                                float scale, const float *h0,
                                const int64_t *cu_seqlens, void *o,
                                float *h_last, void *workspace,
                                int64_t workspace_bytes,
                                mssm_attention_dims dims, mssm_dtypes dtypes,
                                void *stream);
/* For the forward (backward == 0) or the backward. */
MSSM_API int64_t mssm_linear_attention_workspace(mssm_attention_dims dims,
                                mssm_dtypes dtypes, int backward);

/*
 * Backward of the linear attention, for the gradients d_o of o and dh_last of
 * h_last.  With R_t = scale * q_t d_o_t^T + exp(log_decay) R_{t+1} (dh_last added
 * at the last step):
 *
 *   dq_t = scale * S_t d_o_t,   dk_t = R_t v_t,   dv_t = R_t^T k_t
 *   dh0  = exp(log_decay) R_0
 *
 * The states are formed again.  The decays are constants of the model and have
 * no gradient.
 *   d_o      (total, heads, value), dtype `io`      required
 *   dh_last  (seqs, heads, key, value) float32      nullable -> 0
 *   dq, dk   like q; dv like v                      required (outputs); rows of
 *            no sequence as for o
 *   dh0      (seqs, heads, key, value) float32      nullable (output)
 * Rounding as in the forward.  Errors as for the forward; no output may overlap
 * an input or another output.
 */
MSSM_API mssm_status mssm_linear_attention_bwd(const void *q, const void *k,
                                const void *v, const float *log_decay,
                                float scale, const float *h0,
                                const int64_t *cu_seqlens, const void *d_o,
                                const float *dh_last, void *dq, void *dk,
                                void *dv, float *dh0, void *workspace,
                                int64_t workspace_bytes,
                                mssm_attention_dims dims, mssm_dtypes dtypes,
                                void *stream);

/*
 * One decode step of the linear attention on a cached state, in place: the
 * forward at one step with h0 = h_last = state, in float32 throughout.
 *
 *   state    (seqs, heads, key, value) float32      required, read and overwritten
 *   q, k     (seqs, heads, key), v, o (seqs, heads, value), dtype `io`  required
 * `seqlen` and `total` are ignored.  Errors as for the forward; state and o must
 * not overlap any input or each other.
 */
MSSM_API mssm_status mssm_linear_attention_update(float *state, const void *q,
                                const void *k, const void *v,
                                const float *log_decay, float scale, void *o,
                                mssm_attention_dims dims, mssm_dtypes dtypes,
                                void *stream);

/* Sizes of a selection of beams. */
typedef struct {
    int64_t batch;   /* entries >= 0 */
    int64_t beams;   /* of an entry, 1 <= beams <= MSSM_MAX_BEAMS */
    int64_t vocab;   /* >= 1 */
    int64_t count;   /* candidates, 1 <= count <= min(MSSM_MAX_BEAM_COUNT, beams * vocab) */
} mssm_beam_dims;

/*
 * A beam search's selection over beams and vocabulary.  For every entry, the
 * `count` largest of
 *
 *   value[j, v] = scores[j] + logits[j, v] - log sum_v exp(logits[j, v])
 *
 * in order: words of one beam by their logits, exactly, words of different beams
 * by their values in float64, equal ones by the lowest j * vocab + v.  (With scores
 * so large that float64 adds nothing to them, that is the first beam's best words.)
 * A beam whose score or
 * log sum exp is not finite (a finished or empty beam, NaN or +infinity among
 * its logits, no finite logit) counts as -infinity for every word.
 *
 *   logits   (batch, beams, vocab), dtype `io`      required
 *   scores   (batch, beams) float32                 required
 *   out_scores  (batch, count) float32              required (output): the values
 *   out_tokens, out_beams  (batch, count) int64     required (outputs): v and j
 * The sum of the exponentials is float32.  Errors: as for mssm_layer_norm_fwd; also
 * MSSM_ERR_INVALID_ARG for beams, vocab or count < 1 or count > beams * vocab,
 * MSSM_ERR_UNSUPPORTED for beams > MSSM_MAX_BEAMS, count > MSSM_MAX_BEAM_COUNT,
 * vocab >= 2^30, batch >= 2^23 or 2^24 or more pieces of 4096 words in all beams'
 * vocabularies.  batch == 0: nothing to do, MSSM_OK.
 */
MSSM_API mssm_status mssm_beam_select(const void *logits, const float *scores,
                                float *out_scores, int64_t *out_tokens,
                                int64_t *out_beams, void *workspace,
                                int64_t workspace_bytes, mssm_beam_dims dims,
                                mssm_dtypes dtypes, void *stream);
MSSM_API int64_t mssm_beam_select_workspace(mssm_beam_dims dims, mssm_dtypes dtypes);

/*
 * Reorders the states of beams in place: for every state and entry b,
 *
 *   row (b, j) <- row (b, origins[b, j])       j < beams
 *
 * all rows at once, so beams may continue one another in any way.  Beams with
 * origins[b, j] == j are neither read nor written; an origin outside [0, beams)
 * leaves its beam as it is.
 *
 *   states     (host) array of `count` device pointers: (batch, beams, row_bytes[i])
 *              bytes each, of any alignment
 *   row_bytes  (host) array of `count` sizes >= 0
 *   origins    (batch, beams) int64, device                required
 * The host arrays may be reused when the call returns.  dims.vocab and
 * dims.count are ignored.  Errors: MSSM_ERR_INVALID_ARG for a null pointer, a
 * negative size or states that overlap each other or origins;
 * MSSM_ERR_UNSUPPORTED for beams > MSSM_MAX_BEAMS, batch >= 2^24 or a state whose entries have
 * 2^24 or more pieces of 256 times 16 bytes (4 or 1, where its address or row is
 * not a multiple of 16 or 4 bytes).  batch == 0 or count == 0: nothing to do.
 */
MSSM_API mssm_status mssm_state_reorder(void *const *states, const int64_t *row_bytes,
                                int64_t count, const int64_t *origins,
                                mssm_beam_dims dims, void *stream);

/* Force a kernel variant for subsequent calls made by THIS thread
 * (MSSM_VARIANT_AUTO restores the shape-based choice).  A variant that does
 * not apply to the entry point or shape makes that call return
 * MSSM_ERR_UNSUPPORTED.  Returns the previous setting. */
MSSM_API mssm_variant mssm_force_variant(mssm_variant v);

/* The variant the most recent successful call on this thread launched. */
MSSM_API mssm_variant mssm_last_variant(void);

/* Static description of a status code (never NULL). */
MSSM_API const char *mssm_status_string(mssm_status s);

/* Thread-local text of the last error on this thread ("" if none).  The
 * pointer stays valid until the next library call on the same thread. */
MSSM_API const char *mssm_last_error(void);

/* Library version as major*10000 + minor*100 + patch. */
MSSM_API int mssm_version(void);

/* Identity of the sources this binary was built from: 16 hex digits of a
 * SHA-256 over the kernel and host sources, this header and the compile
 * flags.  A binding compares it with the hash of the sources it ships with
 * and refuses a binary built from others.  Never NULL. */
MSSM_API const char *mssm_source_hash(void);

/* Status bits that kernels set on a device while they run. */
#define MSSM_DEVICE_LOOKBACK_TIMEOUT 0x1u /* a look-back wait gave up */
#define MSSM_DEVICE_RECURRENCE_TIMEOUT 0x2u /* the same in the gated recurrence */

/*
 * Device status of the CURRENT device.  Waits for all work queued on the
 * device (hipDeviceSynchronize), then writes into *bits the status bits set
 * by this library's kernels since they were last cleared, and clears them
 * when `clear` is nonzero.  The bits are the device's, shared by every
 * stream and thread.
 *
 * MSSM_DEVICE_LOOKBACK_TIMEOUT: a workgroup of the look-back variant
 * (MSSM_VARIANT_LOOKBACK) waited about a second per predecessor for a
 * predecessor's published carry and gave up.  Predecessors always publish
 * before they wait, so this marks a defect, not a slow device; that call's
 * outputs from the affected segment on (y and h_last) are NaN rather than
 * wrong numbers, and the call itself returned MSSM_OK when it was queued.
 * MSSM_DEVICE_RECURRENCE_TIMEOUT: the same for a segment of the gated linear
 * recurrence or its backward.
 *
 * Errors: MSSM_ERR_INVALID_ARG if bits is NULL; MSSM_ERR_HIP if the
 * synchronisation or a copy fails (including a fault of earlier work).
 */
MSSM_API mssm_status mssm_device_status(uint32_t *bits, int clear);

#ifdef __cplusplus
}
#endif

#endif /* MSSM_H */
