// internal.h -- interface between the C-ABI front end (mssm_api.cpp) and the
// kernel translation units.  Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mssm.h"

namespace mssm {

enum IoType : int { IO_F32 = 0, IO_BF16 = 1 };

// One selective-scan problem, already validated.  Layouts as in mssm.h:
// u, delta, z, y (batch, dim, L); B, C (batch, N, L); A (dim, N);
// delta_bias, D (dim); h0, h_last (batch, dim, N).  h0 may be the same
// buffer as h_last (each element is read before it is overwritten) but
// overlaps nothing else.
struct ScanArgs {
    const void *u;
    const void *delta;
    const float *delta_bias;  // may be null
    const float *A;
    const void *B;
    const void *C;
    const float *D;           // may be null
    const void *z;            // may be null
    const float *h0;          // may be null -> the state starts at 0
    void *y;
    float *h_last;            // may be null
    int64_t batch, L, dim, N;
    IoType io;
    // Convolution prologue: when conv_w is set, u holds the input x of a
    // causal width-4 depthwise convolution (conv_w (dim, 4), conv_b (dim)
    // may be null) and the scan runs on silu(conv(x)).
    const float *conv_w = nullptr;
    const float *conv_b = nullptr;
};

// Scratch memory of the variants that need it, stream-ordered on `stream`,
// from a memory pool the library keeps per device.  The pool keeps freed
// memory (release threshold: unlimited) instead of returning it at every
// synchronisation, so calls separated by synchronisations reuse it rather
// than map it again; it holds up to the largest scratch in use at once until
// the process ends.
hipError_t scratch_alloc(void **ptr, size_t bytes, hipStream_t stream);
hipError_t scratch_free(void *ptr, hipStream_t stream);

// One SSD problem, already validated.  Layouts as in mssm.h.
struct SSDArgs {
    const void *x;
    const void *dt;
    const float *dt_bias;     // may be null
    const float *A;
    const void *B;
    const void *C;
    const float *D;           // may be null
    const void *z;            // may be null -> no gate; (batch, L, H, P) like x
    const float *h0;          // may be null; may be the same buffer as h_last
    void *y;
    float *h_last;            // may be null
    int64_t batch, L, H, P, N, G, chunk;
    IoType io;
};

// One decode step of the selective scan, already validated: state
// (batch, dim, N) float32 updated in place; x, dt, z, y (batch, dim);
// B, C (batch, N); A (dim, N); dt_bias, D (dim).
struct StepArgs {
    float *state;
    const void *x;
    const void *dt;
    const float *dt_bias;     // may be null
    const float *A;
    const void *B;
    const void *C;
    const float *D;           // may be null
    const void *z;            // may be null
    void *y;
    int64_t batch, dim, N;
    IoType io;
};

// One selective-scan backward, already validated: the forward's inputs (as in
// ScanArgs), the output gradients dy (like u) and dh_last (batch, dim, N;
// may be null), and the gradient outputs, all float32: du, ddelta, dz
// (batch, dim, L), dB, dC (batch, N, L), dA (dim, N), dD and ddelta_bias
// (dim), dh0 (batch, dim, N).  dA, dB, dC, dD and ddelta_bias are
// accumulated into and must hold zeros on entry.  Optional outputs may be
// null.
struct BwdArgs {
    const void *u;
    const void *delta;
    const float *delta_bias;
    const float *A;
    const void *B;
    const void *C;
    const float *D;
    const void *z;
    const float *h0;
    const void *dy;
    const float *dh_last;
    float *du;
    float *ddelta;
    float *ddelta_bias;
    float *dA;
    float *dB;
    float *dC;
    float *dD;
    float *dz;
    float *dh0;
    int64_t batch, L, dim, N;
    IoType io;
};

// Each launcher queues its kernel(s) on `stream` and returns the launch
// status.  Shapes have been checked against the launcher's limits by the
// caller (see the *_supported helpers).
hipError_t launch_scan_rowserial(const ScanArgs &a, hipStream_t stream);
bool scan_rowserial_supported(const ScanArgs &a);

hipError_t launch_scan_chunked(const ScanArgs &a, hipStream_t stream);
bool scan_chunked_supported(const ScanArgs &a);
int64_t scan_chunked_waves(const ScanArgs &a);
// Rows start 16-byte aligned and L % 8 == 0: activations move as vectors.
// The chunk walk addresses 16 channel rows and the N rows of B / C with
// 32-bit byte offsets: max(16, N) * L elements must fit in 2^31 bytes.
bool scan_offsets_fit(const ScanArgs &a);
bool scan_rows_vectorizable(const ScanArgs &a);

// Steps of each chunk split across the lanes of the workgroup (a scan of
// (decay, state) pairs across rows and, with slices = 2, across waves).
hipError_t launch_scan_pairscan(const ScanArgs &a, hipStream_t stream, int slices);
bool scan_pairscan_supported(const ScanArgs &a);

// Chunk-parallel variant; allocates its look-back scratch stream-ordered.
hipError_t launch_scan_lookback(const ScanArgs &a, hipStream_t stream);
bool scan_lookback_supported(const ScanArgs &a);
// Bytes of look-back scratch a problem needs, and the variant that takes it
// from the device's fixed array of kNoAllocScratchBytes instead of
// allocating (the caller checks the size first).
constexpr size_t kNoAllocScratchBytes = MSSM_NOALLOC_SCRATCH_BYTES;
size_t scan_lookback_scratch_bytes(const ScanArgs &a);
hipError_t launch_scan_lookback_noalloc(const ScanArgs &a, hipStream_t stream);

// Status bits of the current device (mssm_device_status): waits for the
// device, reads them into *bits and clears them when asked.
hipError_t device_status(uint32_t *bits, bool clear);

// Backward: one lane per (batch, channel) row; stream-ordered scratch for the
// stored states.
hipError_t launch_scan_bwd(const BwdArgs &a, hipStream_t stream);
bool scan_bwd_supported(const BwdArgs &a);
// Backward with the chunked forward's decomposition (N <= 16): lanes over
// (channel, state element), states stored every 32 steps, per-workgroup
// partial sums of dB and dC; stream-ordered scratch.
hipError_t launch_scan_bwd_chunked(const BwdArgs &a, hipStream_t stream);
bool scan_bwd_chunked_supported(const BwdArgs &a);

// Measurement probes (include/mssm_probes.h); arguments already checked.
hipError_t launch_probe_copy(const void *src, void *dst, int64_t bytes, hipStream_t stream);
hipError_t launch_probe_valu(int op, int iters, float *out, hipStream_t stream);

hipError_t launch_state_update(const StepArgs &a, hipStream_t stream);
bool state_update_supported(const StepArgs &a);

// One layer norm, already validated: x, y, dy, dx (rows, dim); weight, bias,
// dweight, dbias (dim); mean, rstd (rows).  The forward leaves dy, dx and the
// weight gradients null.
struct NormArgs {
    const void *x;
    const float *weight;      // may be null -> 1
    const float *bias;        // may be null -> 0
    float eps;
    void *y;
    float *mean;              // forward: output, may be null
    float *rstd;
    const void *dy;
    void *dx;
    float *dweight;           // may be null
    float *dbias;             // may be null
    int64_t rows, dim;
    IoType io;
};
hipError_t launch_layer_norm_fwd(const NormArgs &a, hipStream_t stream);
// workspace: null to allocate from the pool; else at least the bytes said.
hipError_t launch_layer_norm_bwd(const NormArgs &a, void *workspace, hipStream_t stream);
size_t layer_norm_bwd_workspace(const NormArgs &a);

// One gated linear recurrence, already validated: activations (batch, L, dim),
// states (batch, dim), lam (dim).  h0 may be the same buffer as h_last.
struct RecurrenceArgs {
    const void *x;
    const void *r;
    const void *i;
    const float *lam;
    float scale;
    const float *h0;          // may be null -> 0
    void *y;                  // forward: output; backward: input
    float *h_last;            // may be null
    const void *dy;           // backward only, from here on
    const float *dh_last;     // may be null -> 0
    void *dx;
    void *dr;
    void *di;
    float *dlam;              // may be null
    float *dh0;               // may be null
    int64_t batch, L, dim;
    IoType io;
};
bool gated_recurrence_supported(const RecurrenceArgs &a);
size_t gated_recurrence_workspace(const RecurrenceArgs &a, bool bwd);
hipError_t launch_gated_recurrence_fwd(const RecurrenceArgs &a, void *workspace, hipStream_t stream);
hipError_t launch_gated_recurrence_bwd(const RecurrenceArgs &a, void *workspace, hipStream_t stream);
// Its kernels' status bits, as device_status.
hipError_t recurrence_status(uint32_t *bits, bool clear);

// One cross entropy over a vocabulary projection, already validated: hidden,
// dhidden (tokens, dim); weight, dweight (vocab, dim); the rest (tokens).
struct LossArgs {
    const void *hidden;
    const void *weight;
    const int64_t *targets;
    int64_t ignore_index;
    float *loss;              // forward
    float *lse;               // forward: output, may be null; backward: input
    const float *dloss;       // backward only, from here on
    void *dhidden;
    void *dweight;
    int64_t tokens, dim, vocab;
    IoType io;
};
// aligned: hidden and weight start on 16-byte boundaries.
size_t linear_cross_entropy_workspace(const LossArgs &a, bool bwd, bool aligned);
hipError_t launch_linear_cross_entropy_fwd(const LossArgs &a, void *workspace, hipStream_t stream);
hipError_t launch_linear_cross_entropy_bwd(const LossArgs &a, void *workspace, hipStream_t stream);

// One norm of queries and keys with their rotation, already validated: q, dq,
// q_in, dq_in (tokens, q_heads, dim), the same of k; positions (tokens);
// weights and their gradients (dim).
struct HeadNormArgs {
    const void *q;
    const void *k;
    const int64_t *positions;
    const float *q_weight;    // may be null -> 1
    const float *k_weight;    // may be null -> 1
    double base;
    float eps;
    void *q_out;              // forward: normed; backward: gradients of q, k
    void *k_out;
    const void *dq;           // backward only, from here on: of the outputs
    const void *dk;
    float *dq_weight;         // may be null
    float *dk_weight;         // may be null
    int64_t tokens, q_heads, k_heads, dim, rotary;
    IoType io;
};
hipError_t launch_qk_norm_rotary_fwd(const HeadNormArgs &a, hipStream_t stream);
hipError_t launch_qk_norm_rotary_bwd(const HeadNormArgs &a, void *workspace, hipStream_t stream);
size_t qk_norm_rotary_bwd_workspace(const HeadNormArgs &a);

// One linear attention, already validated: q, k, dq, dk (rows, heads, key), v, o
// and their gradients (rows, heads, value) with seqs * seqlen rows or, packed,
// `total`; states (seqs, heads, key, value).  The step has its state in h_last.
struct AttentionArgs {
    const void *q;
    const void *k;
    const void *v;
    const float *log_decay;
    float scale;
    const float *h0;              // may be null -> 0
    const int64_t *cu_seqlens;    // (seqs + 1) of packed sequences, else null
    void *o;
    float *h_last;                // may be null
    const void *dout;             // backward only, from here on
    const float *dh_last;         // may be null -> 0
    void *dq;
    void *dk;
    void *dv;
    float *dh0;                   // may be null
    int64_t seqs, seqlen, total, heads, key, value;
    IoType io;
};
size_t linear_attention_workspace(const AttentionArgs &a, bool bwd);
hipError_t launch_linear_attention_fwd(const AttentionArgs &a, void *workspace, hipStream_t stream);
hipError_t launch_linear_attention_bwd(const AttentionArgs &a, void *workspace, hipStream_t stream);
hipError_t launch_linear_attention_update(const AttentionArgs &a, hipStream_t stream);

// One selection of beams, already validated: logits (batch, beams, vocab),
// scores (batch, beams), the outputs (batch, count).
struct BeamArgs {
    const void *logits;
    const float *scores;
    float *out_scores;
    int64_t *out_tokens;
    int64_t *out_beams;
    int64_t batch, beams, vocab, count;
    IoType io;
};
int64_t beam_select_pieces(int64_t vocab);   // workgroups of a beam
size_t beam_select_workspace(const BeamArgs &a);
hipError_t launch_beam_select(const BeamArgs &a, void *workspace, hipStream_t stream);
// Workgroups of one entry of a state; the reordering in place of `count` states of
// (batch, beams, row_bytes[i]) bytes.
int64_t state_reorder_blocks(const void *state, int64_t row_bytes);
hipError_t launch_state_reorder(void *const *states, const int64_t *row_bytes, int64_t count, const int64_t *origins,
                                int64_t batch, int64_t beams, hipStream_t stream);

hipError_t launch_ssd_recurrent(const SSDArgs &a, hipStream_t stream);
bool ssd_recurrent_supported(const SSDArgs &a);

// Chunked matrix-core form (bf16 I/O, N <= 128, chunk 64 / 128 / 256).
hipError_t launch_ssd_chunked(const SSDArgs &a, hipStream_t stream);
bool ssd_chunked_supported(const SSDArgs &a);

}  // namespace mssm
