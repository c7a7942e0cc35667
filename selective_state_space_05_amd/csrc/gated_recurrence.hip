// gated_recurrence.hip -- the elementwise gated linear recurrence, forward and
// backward.
//
//   log a_t = -c softplus(lam) sigmoid(r_t)
//   h_t     = a_t h_{t-1} + m_t sigmoid(i_t) x_t,   m_t = sqrt(1 - a_t^2),   y_t = h_t
// and from the end, with the carry G,
//   g_t = dy_t + G,   G <- a_t g_t
//   w   = g h_{t-1} a log a - g sigmoid(i) x a^2 (log a / m)
//   dx = g m sigmoid(i),  di = dx x (1 - sigmoid(i)),  dr = w (1 - sigmoid(r)),
//   dlam = sum w sigmoid(lam) / softplus(lam)
//
// Both walks are one affine recurrence s <- a s + b (backward: time reversed,
// b = a dy), so a run of steps composes into one pair (A, H): s <- A s + H.
// The operator reads three tensors and writes one (backward: five and three),
// so it is bound by HBM if it reads them once; in bfloat16 the forward's
// vector work (about 50 instruction slots an element, a third of them the six
// transcendentals) takes nearly as long as its 8 bytes an element.  Hence one
// pass: a workgroup holds a segment of steps of a 128-byte run of channels in
// registers, as decays and input terms, while the state that enters the
// segment is found, and finishes it from there.
//
//   1. Each half-wave holds K consecutive steps ("slot"), each lane V
//      channels; a lane composes its steps, the slots' pairs meet in LDS.
//   2. The segment's pair is published; the entering state is the fold, in
//      order, of the pairs of the earlier segments of the same block of
//      kBlock segments onto the state at the block's start, which the last
//      segment of the block before published.  So a segment reads at most
//      kBlock pairs however long the sequence is, and only one hand-over per
//      kBlock segments lies on the serial path.
//   3. Every lane folds the slots before its own and walks its steps again
//      from registers.
// The association is fixed by the sizes alone, so results repeat bit for bit.
//
// Segments are handed out by a ticket in segment-major order.  A workgroup
// takes its tickets in increasing order and waits only for lower ones, so the
// lowest unfinished ticket is always being worked on and every wait ends.
// Published values cross the XCDs' L2 caches: all accesses to them are
// agent-scope atomics, a flag is stored after the values it announces have
// been acknowledged.
#include "device_math.h"
#include "internal.h"

namespace mssm {

// Status bits of this translation unit's kernels (mssm_device_status).
__device__ uint32_t g_recurrence_status_bits;

namespace {

constexpr int kRowThreads = 64;
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kSlots = 2 * kWaves;       // half-waves
constexpr int kBlock = 64;               // segments between published states
constexpr uint32_t kMaxSpins = 1u << 24;
constexpr float kSeriesLimit = 0.35f;

// Below this many steps one lane walks a row.
constexpr int64_t kRowSteps = 8;

// 1 / (1 + 2^(-x log2 e)).
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-x * kLog2e));
}

// e^x - 1 for x <= 0.  From -0.35 up the Taylor series (its remainder is below
// 2e-8 of the value), below that 2^y - 1, where the subtraction loses at most
// a factor 3.4.  a = 1 + expm1 is then rounded once, and 1 - a^2 =
// -expm1 (2 + expm1) loses nothing as a nears 1.
__device__ __forceinline__ float expm1_series(float x) {
    float p = 1.0f / 5040.0f;
    p = fmaf(p, x, 1.0f / 720.0f);
    p = fmaf(p, x, 1.0f / 120.0f);
    p = fmaf(p, x, 1.0f / 24.0f);
    p = fmaf(p, x, 1.0f / 6.0f);
    p = fmaf(p, x, 0.5f);
    return fmaf(p * x, x, x);
}
template <bool NEAR>
__device__ __forceinline__ float expm1_neg(float x) {
    const float p = expm1_series(x);
    if (NEAR) return p;
    return x >= -kSeriesLimit ? p : fast_exp2(x * kLog2e) - 1.0f;
}

// 1 - a^2 from a - 1.
__device__ __forceinline__ float one_minus_square(float p) { return -fmaf(p, p, p + p); }

// V consecutive elements at any element address.
template <typename T, int V> struct Pack;
template <> struct Pack<float, 1> {
    float v;
    __device__ __forceinline__ float get(int) const { return v; }
    __device__ __forceinline__ void set(const float *f) { v = f[0]; }
};
template <> struct Pack<uint16_t, 1> {
    uint16_t v;
    __device__ __forceinline__ float get(int) const { return bf16_to_f32(v); }
    __device__ __forceinline__ void set(const float *f) { v = f32_to_bf16(f[0]); }
};
template <> struct Pack<uint16_t, 2> {
    uint32_t v;
    __device__ __forceinline__ float get(int k) const { return __uint_as_float(k ? v & 0xffff0000u : v << 16); }
    __device__ __forceinline__ void set(const float *f) {
        typedef float f2 __attribute__((ext_vector_type(2)));
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        v = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){f[0], f[1]}, b2));
    }
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const unsigned char *base, uint32_t off) {
    Pack<T, V> p;
    __builtin_memcpy(&p, base + off, sizeof p);
    return p;
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(unsigned char *base, uint32_t off, const float *f) {
    Pack<T, V> p;
    p.set(f);
    __builtin_memcpy(base + off, &p, sizeof p);
}
// The same from a row's elements one by one, those past the `n` existing ones
// mirroring the last (loads) or left out (stores).
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_some(const unsigned char *row, int c0, int n) {
    float f[V];
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = Io<T>::load(reinterpret_cast<const T *>(row), min(c0 + v, n - 1));
    Pack<T, V> p;
    p.set(f);
    return p;
}
template <typename T, int V>
__device__ __forceinline__ void store_some(unsigned char *row, int c0, int n, const float *f) {
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (c0 + v < n) Io<T>::store(reinterpret_cast<T *>(row), c0 + v, f[v]);
}

// ---- a few steps: one lane walks a row -------------------------------------------

template <typename T>
__global__ __launch_bounds__(kRowThreads) void row_fwd_kernel(const T *__restrict__ x, const T *__restrict__ r,
                                                              const T *__restrict__ i,
                                                              const float *__restrict__ lam, float scale,
                                                              const float *h0, T *__restrict__ y, float *h_last,
                                                              int64_t rows, int L, int64_t dim) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
    if (row >= rows) return;
    const int64_t b = row / dim, d = row - b * dim;
    float h = h0 ? h0[row] : 0.0f;
    const float rate = -scale * softplus_libm(lam[d]);
    int64_t at = b * L * dim + d;
    for (int t = 0; t < L; ++t, at += dim) {
        const float p = expm1_neg<false>(rate * sigmoid(Io<T>::load(r, at)));
        const float m = __builtin_amdgcn_sqrtf(one_minus_square(p));
        h = fmaf(1.0f + p, h, m * sigmoid(Io<T>::load(i, at)) * Io<T>::load(x, at));
        Io<T>::store(y, at, h);
    }
    if (h_last) h_last[row] = h;
}

// ---- segments ----------------------------------------------------------------------

// What segments exchange: pairs (A, H) of NC channels per (segment, group),
// states of NC channels per (block, group), one flag for each, the ticket.
struct Exchange {
    uint64_t *pairs;
    float *states;
    uint32_t *flags, *state_flags, *ticket;
    int nseg, groups;
};

template <int NC>
struct Shared {
    float2 slot[kSlots][NC];             // pairs of the half-waves
    float2 fold[kThreads / NC][NC];      // folds of earlier segments' pairs
    float base[NC];                      // state at the block's start
    float red[kSlots][NC];
    int next;
    int bad[kWaves];
};

__device__ __forceinline__ uint32_t load_flag(const uint32_t *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Wait until this wave's stores are acknowledged: agent-scope loads see them.
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Waits for a flag; false if the wait gave up (a defect: values announced by
// lower tickets always arrive).
__device__ __forceinline__ bool wait_flag(const uint32_t *p) {
    uint32_t spins = 0;
    while (load_flag(p) == 0) {
        __builtin_amdgcn_s_sleep(1);
        if (++spins == kMaxSpins) return false;
    }
    return true;
}

// The state that enters this lane's slot, from the slots' pairs (A, H) and the
// segments before.  `init` is the caller's initial state of this group's
// channels (null: zero); `valid` channels of the group exist.  c0: the lane's
// first channel (lanes past the channels mirror the last ones, writing the
// same values to the same places).  end: the state after the whole segment, in the
// first NC threads.
template <int V, int NC>
__device__ __forceinline__ void enter(const float *A, const float *H, float *h, float *end, int seg, int group,
                                      const float *init, int valid, int tid, int c0, const Exchange &ex, Shared<NC> &sm) {
    constexpr int kFolds = kThreads / NC, kPer = kBlock / kFolds, kPerWave = kBlock / kWaves;
    static_assert(kPer % 4 == 0 && kBlock % kWaves == 0, "whole batches of pairs");
    const int lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int slot = tid / 32;
    const int q = seg % kBlock, block = seg / kBlock;
#pragma unroll
    for (int v = 0; v < V; ++v) sm.slot[slot][c0 + v] = make_float2(A[v], H[v]);
    // the initial state is read before this segment's pair is published: the
    // last segment, which may write the same buffer, waits for that pair
    if (block == 0 && tid < NC) sm.base[tid] = init ? init[min(tid, valid - 1)] : 0.0f;
    if (lane == 0) sm.bad[wave] = 0;
    __syncthreads();
    if (ex.nseg > 1) {
        if (tid < NC && seg < ex.nseg - 1) {
            float2 t = sm.slot[0][tid];
#pragma unroll
            for (int s = 1; s < kSlots; ++s) {
                const float2 n = sm.slot[s][tid];
                t = make_float2(n.x * t.x, fmaf(n.x, t.y, n.y));
            }
            const uint64_t bits = static_cast<uint64_t>(__float_as_uint(t.x)) |
                                  static_cast<uint64_t>(__float_as_uint(t.y)) << 32;
            __hip_atomic_store(ex.pairs + (static_cast<int64_t>(seg) * ex.groups + group) * NC + tid, bits,
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            stores_done();
            if (tid == 0)
                __hip_atomic_store(ex.flags + static_cast<int64_t>(seg) * ex.groups + group, 1u, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        }
        // each wave waits for the kPerWave pairs that its lanes fold
        const int seg0 = block * kBlock;
        if (wave * kPerWave < q) {
            const int j = wave * kPerWave + lane;
            bool ok = true;
            if (lane < kPerWave && j < q)
                ok = wait_flag(ex.flags + static_cast<int64_t>(seg0 + j) * ex.groups + group);
            if (!__all(ok) && lane == 0) sm.bad[wave] = 1;
        }
        const int ch = tid % NC, fold = tid / NC;
        float2 t = make_float2(1.0f, 0.0f);
#pragma unroll
        for (int k0 = 0; k0 < kPer; k0 += 4) {
            uint64_t bits[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = min(fold * kPer + k0 + k, q - 1);
                if (j >= 0)
                    bits[k] = __hip_atomic_load(
                        ex.pairs + (static_cast<int64_t>(seg0 + j) * ex.groups + group) * NC + ch, __ATOMIC_RELAXED,
                        __HIP_MEMORY_SCOPE_AGENT);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (fold * kPer + k0 + k < q) {
                    const float a = __uint_as_float(static_cast<uint32_t>(bits[k]));
                    t = make_float2(a * t.x, fmaf(a, t.y, __uint_as_float(static_cast<uint32_t>(bits[k] >> 32))));
                }
        }
        sm.fold[fold][ch] = t;
        if (block > 0 && tid < NC) {
            const int64_t at = static_cast<int64_t>(block - 1) * ex.groups + group;
            if (!__all(wait_flag(ex.state_flags + at)) && lane == 0) sm.bad[wave] = 1;
            sm.base[tid] = __uint_as_float(__hip_atomic_load(
                reinterpret_cast<const uint32_t *>(ex.states) + at * NC + tid, __ATOMIC_RELAXED,
                __HIP_MEMORY_SCOPE_AGENT));
        }
        __syncthreads();
    }
    int bad = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) bad |= sm.bad[w];
    if (bad && tid == 0)
        __hip_atomic_fetch_or(&g_recurrence_status_bits, MSSM_DEVICE_RECURRENCE_TIMEOUT, __ATOMIC_RELAXED,
                              __HIP_MEMORY_SCOPE_AGENT);
    const int folds = ex.nseg > 1 ? (q + kPer - 1) / kPer : 0;
    if (tid < NC) {
        float s = bad ? __builtin_nanf("") : sm.base[tid];
        for (int k = 0; k < folds; ++k) s = fmaf(sm.fold[k][tid].x, s, sm.fold[k][tid].y);
#pragma unroll
        for (int k = 0; k < kSlots; ++k) s = fmaf(sm.slot[k][tid].x, s, sm.slot[k][tid].y);
        *end = s;
        if (q == kBlock - 1 && seg < ex.nseg - 1) {
            const int64_t at = static_cast<int64_t>(block) * ex.groups + group;
            __hip_atomic_store(reinterpret_cast<uint32_t *>(ex.states) + at * NC + tid, __float_as_uint(s),
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            stores_done();
            if (tid == 0)
                __hip_atomic_store(ex.state_flags + at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = bad ? __builtin_nanf("") : sm.base[c0 + v];
    for (int k = 0; k < folds; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(sm.fold[k][c0 + v].x, h[v], sm.fold[k][c0 + v].y);
    for (int k = 0; k < slot; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = fmaf(sm.slot[k][c0 + v].x, h[v], sm.slot[k][c0 + v].y);
}

// Where a lane's part of a (segment, group) lies.  Row k of the lane is at
// byte off + k step (backward: off - k step) from the segment's base rows;
// `steps` of its K rows exist.  Its channels are c0 .. c0 + V - 1 of the
// group's `valid` ones.
struct Part {
    uint32_t off, step;
    int steps, c0, valid;
};

struct Walk {
    int64_t L;
    int dim, groups_per_batch, items;
};

// Decays and input terms of a lane's rows, and their composition (A, H).
// FULL: all K rows of every lane exist and the channels come in whole packs.
template <typename T, int V, int K, bool NEAR, bool FULL>
__device__ __forceinline__ void fwd_terms(const unsigned char *x, const unsigned char *r, const unsigned char *i,
                                          const Part &pt, const float *rate, float (*a)[V], float (*b)[V], float *A,
                                          float *H) {
    Pack<T, V> xr[K], rr[K], ir[K];
    if (FULL) {
        uint32_t o = pt.off + pt.c0 * sizeof(T);
#pragma unroll
        for (int k = 0; k < K; ++k, o += pt.step) {
            rr[k] = load_pack<T, V>(r, o);
            ir[k] = load_pack<T, V>(i, o);
            xr[k] = load_pack<T, V>(x, o);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.0f, H[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!FULL) {
            __builtin_amdgcn_sched_barrier(0);   // a row at a time: few registers
            const uint32_t o = pt.off + max(min(k, pt.steps - 1), 0) * pt.step;
            rr[k] = load_some<T, V>(r + o, pt.c0, pt.valid);
            ir[k] = load_some<T, V>(i + o, pt.c0, pt.valid);
            xr[k] = load_some<T, V>(x + o, pt.c0, pt.valid);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float p = expm1_neg<NEAR>(rate[v] * sigmoid(rr[k].get(v)));
            float in = __builtin_amdgcn_sqrtf(one_minus_square(p)) * sigmoid(ir[k].get(v)) * xr[k].get(v);
            if (!FULL && k >= pt.steps) p = 0.0f, in = 0.0f;
            a[k][v] = 1.0f + p;
            b[k][v] = in;
            A[v] *= a[k][v];
            H[v] = fmaf(a[k][v], H[v], in);
        }
    }
}

// The next (segment, group) of a workgroup: its block index, or tickets.
__device__ __forceinline__ int take_ticket(const Exchange &ex) {
    return static_cast<int>(__hip_atomic_fetch_add(ex.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads, 4) void segment_fwd_kernel(const T *__restrict__ x, const T *__restrict__ r,
                                                                  const T *__restrict__ i,
                                                                  const float *__restrict__ lam, float scale,
                                                                  const float *h0, T *__restrict__ y,
                                                                  float *h_last, Walk w, Exchange ex) {
    constexpr int NC = 32 * V, S = kSlots * K;
    __shared__ Shared<NC> sm;
    int item = blockIdx.x;
    if (ex.nseg > 1) {
        if (threadIdx.x == 0) sm.next = take_ticket(ex);
        __syncthreads();
        item = __builtin_amdgcn_readfirstlane(sm.next);
    }
    while (item < w.items) {
        // hidden from the optimiser, which would otherwise keep every address
        // that follows from the lane's place in registers across segments,
        // and spill
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int slot = tid / 32;
        int next = w.items;
        if (ex.nseg > 1 && tid == 0) next = take_ticket(ex);
        const int seg = item / ex.groups, group = item - seg * ex.groups;
        const int batch = group / w.groups_per_batch, ch0 = (group - batch * w.groups_per_batch) * NC;
        const int64_t t0 = static_cast<int64_t>(seg) * S, row = static_cast<int64_t>(batch) * w.dim + ch0;
        const int64_t at = (batch * w.L + t0) * w.dim + ch0;
        Part pt;
        pt.step = static_cast<uint32_t>(w.dim) * sizeof(T);
        pt.c0 = (tid % 32) * V;
        pt.valid = min(NC, w.dim - ch0);
        const int64_t left = w.L - t0 - slot * K;
        pt.steps = left < K ? static_cast<int>(max(left, static_cast<int64_t>(0))) : K;
        pt.off = (left > 0 ? slot * K : 0) * pt.step;   // a slot past the end reads the first row
        const bool full = t0 + S <= w.L && pt.valid % V == 0;
        if (full) pt.c0 = min(pt.c0, pt.valid - V);      // lanes past the channels mirror the last
        float rate[V];
        bool near = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            rate[v] = -scale * softplus_libm(lam[ch0 + min(pt.c0 + v, pt.valid - 1)]);
            near = near && rate[v] >= -kSeriesLimit;
        }
        const float *init = h0 ? h0 + row : nullptr;
        const unsigned char *xb = reinterpret_cast<const unsigned char *>(x + at),
                            *rb = reinterpret_cast<const unsigned char *>(r + at),
                            *ib = reinterpret_cast<const unsigned char *>(i + at);
        unsigned char *yb = reinterpret_cast<unsigned char *>(y + at);
        float a[K][V], b[K][V], A[V], H[V], h[V], end = 0.0f;
        if (full) {
            // log a is above the series' limit for every r where the rate is
            if (__all(near)) fwd_terms<T, V, K, true, true>(xb, rb, ib, pt, rate, a, b, A, H);
            else fwd_terms<T, V, K, false, true>(xb, rb, ib, pt, rate, a, b, A, H);
        } else {
            fwd_terms<T, V, K, false, false>(xb, rb, ib, pt, rate, a, b, A, H);
        }
        enter<V, NC>(A, H, h, &end, seg, group, init, pt.valid, tid, pt.c0, ex, sm);
        uint32_t o = pt.off;
#pragma unroll
        for (int k = 0; k < K; ++k, o += pt.step) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(a[k][v], h[v], b[k][v]);
            if (full) store_pack<T, V>(yb, o + pt.c0 * sizeof(T), h);
            else if (k < pt.steps) store_some<T, V>(yb + o, pt.c0, pt.valid, h);
        }
        if (h_last && seg == ex.nseg - 1 && tid < pt.valid) h_last[row + tid] = end;
        if (ex.nseg == 1) return;
        if (tid == 0) sm.next = next;
        __syncthreads();
        item = __builtin_amdgcn_readfirstlane(sm.next);
        __syncthreads();
    }
}

// One element of the backward.  G: the carry, advanced past this step.
struct Grad {
    float dx, dr, di, w;
};
__device__ __forceinline__ Grad grad_step(float la, float sr, float p, float x, float i, float dy, float before,
                                          float *G) {
    const float em = one_minus_square(p);
    const float rm = em > 0.0f ? __builtin_amdgcn_rsqf(em) : 0.0f;   // log a / m -> 0 with log a
    const float a = 1.0f + p, si = sigmoid(i), u = si * x;
    const float g = dy + *G, gm = g * (em * rm);
    *G = a * g;
    Grad o;
    o.w = *G * la * fmaf(-u * a, rm, before);
    o.dx = gm * si;
    o.di = gm * u * (1.0f - si);
    o.dr = o.w * (1.0f - sr);
    return o;
}

// What a lane holds of a row for the walk: the inputs as they are stored,
// sigmoid(r) and a - 1.  y: the state before the row, one row down in the
// output (the caller looks after the sequence's first step).
template <typename T, int V, int K>
struct Held {
    Pack<T, V> x[K], i[K], y[K], dy[K];
    float sr[K][V], p[K][V];
};

template <typename T, int V, int K, bool NEAR, bool FULL>
__device__ __forceinline__ void bwd_terms(const unsigned char *x, const unsigned char *r, const unsigned char *i,
                                          const unsigned char *y, const unsigned char *dy, const Part &pt,
                                          const float *rate, Held<T, V, K> &hd, float *A, float *H) {
    Pack<T, V> rr[K];
    if (FULL) {
        uint32_t o = pt.off + pt.c0 * sizeof(T);
#pragma unroll
        for (int k = 0; k < K; ++k, o -= pt.step) {
            rr[k] = load_pack<T, V>(r, o);
            hd.dy[k] = load_pack<T, V>(dy, o);
            hd.x[k] = load_pack<T, V>(x, o);
            hd.i[k] = load_pack<T, V>(i, o);
            hd.y[k] = load_pack<T, V>(y, o - pt.step);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.0f, H[v] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (!FULL) {
            __builtin_amdgcn_sched_barrier(0);   // a row at a time: few registers
            const uint32_t o = pt.off - max(min(k, pt.steps - 1), 0) * pt.step;
            rr[k] = load_some<T, V>(r + o, pt.c0, pt.valid);
            hd.dy[k] = load_some<T, V>(dy + o, pt.c0, pt.valid);
            hd.x[k] = load_some<T, V>(x + o, pt.c0, pt.valid);
            hd.i[k] = load_some<T, V>(i + o, pt.c0, pt.valid);
            hd.y[k] = load_some<T, V>(y + (o >= pt.step ? o - pt.step : o), pt.c0, pt.valid);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            hd.sr[k][v] = sigmoid(rr[k].get(v));
            hd.p[k][v] = expm1_neg<NEAR>(rate[v] * hd.sr[k][v]);
            const float a = 1.0f + hd.p[k][v];
            if (FULL || k < pt.steps) {
                A[v] *= a;
                H[v] = a * (hd.dy[k].get(v) + H[v]);
            }
        }
    }
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads, 4) void segment_bwd_kernel(
    const T *__restrict__ x, const T *__restrict__ r, const T *__restrict__ i, const float *__restrict__ lam,
    float scale, const float *__restrict__ h0, const T *__restrict__ y, const T *__restrict__ dy,
    const float *__restrict__ dh_last, T *__restrict__ dx, T *__restrict__ dr, T *__restrict__ di,
    float *__restrict__ part, float *__restrict__ dh0, Walk w, Exchange ex) {
    constexpr int NC = 32 * V, S = kSlots * K;
    __shared__ Shared<NC> sm;
    int item = blockIdx.x;
    if (ex.nseg > 1) {
        if (threadIdx.x == 0) sm.next = take_ticket(ex);
        __syncthreads();
        item = __builtin_amdgcn_readfirstlane(sm.next);
    }
    while (item < w.items) {
        // hidden from the optimiser, which would otherwise keep every address
        // that follows from the lane's place in registers across segments,
        // and spill
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int slot = tid / 32;
        int next = w.items;
        if (ex.nseg > 1 && tid == 0) next = take_ticket(ex);
        const int seg = item / ex.groups, group = item - seg * ex.groups;
        const int batch = group / w.groups_per_batch, ch0 = (group - batch * w.groups_per_batch) * NC;
        const int64_t row = static_cast<int64_t>(batch) * w.dim + ch0;
        // the segment's steps run from t_hi down; its base row is the one
        // before them, or the sequence's first
        const int64_t t_hi = w.L - 1 - static_cast<int64_t>(seg) * S;
        const bool whole = t_hi >= S;
        const int64_t t_base = whole ? t_hi - S : 0, at = (batch * w.L + t_base) * w.dim + ch0;
        Part pt;
        pt.step = static_cast<uint32_t>(w.dim) * sizeof(T);
        pt.c0 = (tid % 32) * V;
        pt.valid = min(NC, w.dim - ch0);
        const int64_t t_lane = t_hi - slot * K;          // of the lane's row 0
        pt.steps = t_lane + 1 < K ? static_cast<int>(max(t_lane + 1, static_cast<int64_t>(0))) : K;
        pt.off = static_cast<uint32_t>(max(t_lane - t_base, static_cast<int64_t>(0))) * pt.step;
        const int first = whole ? K : static_cast<int>(t_lane);
        const bool full = whole && pt.valid % V == 0;
        if (full) pt.c0 = min(pt.c0, pt.valid - V);      // lanes past the channels mirror the last
        float rate[V], start[V], sum[V];
        bool near = true;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = min(pt.c0 + v, pt.valid - 1);
            rate[v] = -scale * softplus_libm(lam[ch0 + c]);
            near = near && rate[v] >= -kSeriesLimit;
            start[v] = h0 ? h0[row + c] : 0.0f;
            sum[v] = 0.0f;
        }
        const float *init = dh_last ? dh_last + row : nullptr;
        const auto in = [&](const T *p) { return reinterpret_cast<const unsigned char *>(p + at); };
        const auto out = [&](T *p) { return reinterpret_cast<unsigned char *>(p + at); };
        Held<T, V, K> hd;
        float A[V], H[V], G[V], end = 0.0f;
        if (full) {
            if (__all(near)) bwd_terms<T, V, K, true, true>(in(x), in(r), in(i), in(y), in(dy), pt, rate, hd, A, H);
            else bwd_terms<T, V, K, false, true>(in(x), in(r), in(i), in(y), in(dy), pt, rate, hd, A, H);
        } else {
            bwd_terms<T, V, K, false, false>(in(x), in(r), in(i), in(y), in(dy), pt, rate, hd, A, H);
        }
        enter<V, NC>(A, H, G, &end, seg, group, init, pt.valid, tid, pt.c0, ex, sm);
        unsigned char *dxb = out(dx), *drb = out(dr), *dib = out(di);
        uint32_t o = pt.off;
#pragma unroll
        for (int k = 0; k < K; ++k, o -= pt.step) {
            if (!full && k >= pt.steps) break;
            float ox[V], og[V], oi[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float before = k == first ? start[v] : hd.y[k].get(v);
                const Grad gr = grad_step(rate[v] * hd.sr[k][v], hd.sr[k][v], hd.p[k][v], hd.x[k].get(v),
                                          hd.i[k].get(v), hd.dy[k].get(v), before, &G[v]);
                ox[v] = gr.dx;
                og[v] = gr.dr;
                oi[v] = gr.di;
                sum[v] += gr.w;
            }
            if (full) {
                store_pack<T, V>(dxb, o + pt.c0 * sizeof(T), ox);
                store_pack<T, V>(drb, o + pt.c0 * sizeof(T), og);
                store_pack<T, V>(dib, o + pt.c0 * sizeof(T), oi);
            } else {
                store_some<T, V>(dxb + o, pt.c0, pt.valid, ox);
                store_some<T, V>(drb + o, pt.c0, pt.valid, og);
                store_some<T, V>(dib + o, pt.c0, pt.valid, oi);
            }
        }
        if (dh0 && seg == ex.nseg - 1 && tid < pt.valid) dh0[row + tid] = end;
        if (part) {
#pragma unroll
            for (int v = 0; v < V; ++v) sm.red[slot][pt.c0 + v] = sum[v];
            __syncthreads();
            if (tid < pt.valid) {
                float s = 0.0f;
#pragma unroll
                for (int k = 0; k < kSlots; ++k) s += sm.red[k][tid];
                part[static_cast<int64_t>(seg) * (ex.groups / w.groups_per_batch) * w.dim + row + tid] = s;
            }
        }
        if (ex.nseg == 1) return;
        if (tid == 0) sm.next = next;
        __syncthreads();
        item = __builtin_amdgcn_readfirstlane(sm.next);
        __syncthreads();
    }
}

// dlam = sum of the parts, times sigmoid(lam) / softplus(lam) (which tends to
// 1 as lam falls).  32 channels and 16 slices of the parts a workgroup.
constexpr int kSlices = 16;
__global__ __launch_bounds__(32 * kSlices) void dlam_kernel(const float *__restrict__ part,
                                                            const float *__restrict__ lam,
                                                            float *__restrict__ dlam, int64_t parts, int64_t dim) {
    __shared__ float sh[kSlices][32];
    const int c = threadIdx.x % 32, slice = threadIdx.x / 32;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + c;
    float s = 0.0f;
    if (d < dim)
        for (int64_t k = slice; k < parts; k += kSlices) s += part[k * dim + d];
    sh[slice][c] = s;
    __syncthreads();
    if (slice == 0 && d < dim) {
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < kSlices; ++k) s += sh[k][c];
        const float sp = softplus_libm(lam[d]), sg = 1.0f / (1.0f + expf(-lam[d]));
        dlam[d] = s * (sp > 0.0f ? sg / sp : 1.0f);
    }
}

__global__ void clear_kernel(uint32_t *p, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) p[i] = 0u;
}

// Steps a lane holds.  More steps a lane make fewer segments and fewer pairs
// to exchange; short sequences take fewer, so that more lanes share them.
int steps_per_lane(const RecurrenceArgs &a, bool bwd) {
    if (bwd) return a.L <= 2 * kSlots ? 2 : 8;
    return a.L <= 2 * kSlots ? 2 : 16;
}

struct Plan {
    int64_t groups_per_batch, groups, nseg, parts;
    int nc, k;
    size_t at_pairs, at_states, at_part, at_flags, bytes;
    int64_t flags;                       // 32-bit words to clear
};

Plan make_plan(const RecurrenceArgs &a, bool bwd) {
    Plan p{};
    p.nc = a.io == IO_F32 ? 32 : 64;
    p.k = steps_per_lane(a, bwd);
    p.groups_per_batch = (a.dim + p.nc - 1) / p.nc;
    p.groups = a.batch * p.groups_per_batch;
    p.nseg = (a.L + kSlots * p.k - 1) / (kSlots * p.k);
    size_t size = 0;
    const auto add = [&](int64_t bytes) {
        const size_t at = size;
        size += (static_cast<size_t>(bytes) + 255) / 256 * 256;
        return at;
    };
    if (!bwd && a.L <= kRowSteps) return p;
    if (p.nseg > 1) {
        const int64_t items = p.nseg * p.groups, blocks = (p.nseg + kBlock - 1) / kBlock * p.groups;
        p.at_pairs = add(items * p.nc * 8);
        p.at_states = add(blocks * p.nc * 4);
        p.flags = items + blocks + 1;
        p.at_flags = add(p.flags * 4);
    }
    if (bwd) {
        p.parts = p.nseg * a.batch;
        p.at_part = add(p.parts * a.dim * 4);
    }
    p.bytes = size;
    return p;
}

hipError_t make_exchange(const Plan &p, unsigned char *base, Exchange *ex, hipStream_t stream) {
    *ex = Exchange{};
    ex->nseg = static_cast<int>(p.nseg);
    ex->groups = static_cast<int>(p.groups);
    if (p.nseg == 1) return hipSuccess;
    ex->pairs = reinterpret_cast<uint64_t *>(base + p.at_pairs);
    ex->states = reinterpret_cast<float *>(base + p.at_states);
    ex->flags = reinterpret_cast<uint32_t *>(base + p.at_flags);
    ex->state_flags = ex->flags + p.nseg * p.groups;
    ex->ticket = ex->flags + p.flags - 1;
    hipLaunchKernelGGL(clear_kernel, dim3(static_cast<uint32_t>((p.flags + 255) / 256)), dim3(256), 0, stream,
                       ex->flags, p.flags);
    return hipGetLastError();
}

// Workgroups of 512 lanes that stay resident: two a compute unit.
uint32_t segment_grid(const Plan &p) {
    const int64_t items = p.nseg * p.groups;
    return static_cast<uint32_t>(p.nseg == 1 || items < 512 ? items : 512);
}

template <typename T, int V, int K>
hipError_t fwd_segments(const RecurrenceArgs &a, const Plan &p, unsigned char *base, hipStream_t stream) {
    Exchange ex;
    hipError_t e = make_exchange(p, base, &ex, stream);
    if (e != hipSuccess) return e;
    const Walk w{a.L, static_cast<int>(a.dim), static_cast<int>(p.groups_per_batch),
                 static_cast<int>(p.nseg * p.groups)};
    hipLaunchKernelGGL((segment_fwd_kernel<T, V, K>), dim3(segment_grid(p)), dim3(kThreads), 0, stream,
                       static_cast<const T *>(a.x), static_cast<const T *>(a.r), static_cast<const T *>(a.i), a.lam,
                       a.scale, a.h0, static_cast<T *>(a.y), a.h_last, w, ex);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t fwd(const RecurrenceArgs &a, void *workspace, hipStream_t stream) {
    if (a.L <= kRowSteps) {
        const int64_t rows = a.batch * a.dim;
        hipLaunchKernelGGL(row_fwd_kernel<T>, dim3(static_cast<uint32_t>((rows + kRowThreads - 1) / kRowThreads)),
                           dim3(kRowThreads), 0, stream, static_cast<const T *>(a.x), static_cast<const T *>(a.r),
                           static_cast<const T *>(a.i), a.lam, a.scale, a.h0, static_cast<T *>(a.y), a.h_last, rows,
                           static_cast<int>(a.L), a.dim);
        return hipGetLastError();
    }
    const Plan p = make_plan(a, false);
    void *mem = workspace;
    hipError_t e = hipSuccess;
    if (!mem && p.bytes) e = scratch_alloc(&mem, p.bytes, stream);
    if (e != hipSuccess) return e;
    unsigned char *base = static_cast<unsigned char *>(mem);
    e = p.k == 2 ? fwd_segments<T, V, 2>(a, p, base, stream) : fwd_segments<T, V, 16>(a, p, base, stream);
    if (mem && !workspace) {
        const hipError_t f = scratch_free(mem, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

template <typename T, int V, int K>
hipError_t bwd_segments(const RecurrenceArgs &a, const Plan &p, unsigned char *base, hipStream_t stream) {
    Exchange ex;
    hipError_t e = make_exchange(p, base, &ex, stream);
    if (e != hipSuccess) return e;
    const Walk w{a.L, static_cast<int>(a.dim), static_cast<int>(p.groups_per_batch),
                 static_cast<int>(p.nseg * p.groups)};
    float *part = a.dlam ? reinterpret_cast<float *>(base + p.at_part) : nullptr;
    hipLaunchKernelGGL((segment_bwd_kernel<T, V, K>), dim3(segment_grid(p)), dim3(kThreads), 0, stream,
                       static_cast<const T *>(a.x), static_cast<const T *>(a.r), static_cast<const T *>(a.i), a.lam,
                       a.scale, a.h0, static_cast<const T *>(a.y), static_cast<const T *>(a.dy), a.dh_last,
                       static_cast<T *>(a.dx), static_cast<T *>(a.dr), static_cast<T *>(a.di), part, a.dh0, w, ex);
    e = hipGetLastError();
    if (e == hipSuccess && part) {
        hipLaunchKernelGGL(dlam_kernel, dim3(static_cast<uint32_t>((a.dim + 31) / 32)), dim3(32 * kSlices), 0,
                           stream, part, a.lam, a.dlam, p.parts, a.dim);
        e = hipGetLastError();
    }
    return e;
}

template <typename T, int V>
hipError_t bwd(const RecurrenceArgs &a, void *workspace, hipStream_t stream) {
    const Plan p = make_plan(a, true);
    void *mem = workspace;
    hipError_t e = hipSuccess;
    if (!mem && p.bytes) e = scratch_alloc(&mem, p.bytes, stream);
    if (e != hipSuccess) return e;
    unsigned char *base = static_cast<unsigned char *>(mem);
    e = p.k == 2 ? bwd_segments<T, V, 2>(a, p, base, stream) : bwd_segments<T, V, 8>(a, p, base, stream);
    if (mem && !workspace) {
        const hipError_t f = scratch_free(mem, stream);
        if (e == hipSuccess) e = f;
    }
    return e;
}

}  // namespace

size_t gated_recurrence_workspace(const RecurrenceArgs &a, bool bwd) { return make_plan(a, bwd).bytes; }

bool gated_recurrence_supported(const RecurrenceArgs &a) {
    // byte offsets inside a segment (at most 257 rows) fit 32 bits; one lane a
    // row, 64 a workgroup; items and flags fit 31 bits
    if (a.dim >= (int64_t(1) << 21) || a.batch * a.dim >= (int64_t(1) << 31)) return false;
    const int64_t nc = a.io == IO_F32 ? 32 : 64;
    return (a.L + 127) / 128 < (int64_t(1) << 30) / (a.batch * ((a.dim + nc - 1) / nc));
}

hipError_t launch_gated_recurrence_fwd(const RecurrenceArgs &a, void *workspace, hipStream_t stream) {
    return a.io == IO_F32 ? fwd<float, 1>(a, workspace, stream) : fwd<uint16_t, 2>(a, workspace, stream);
}

hipError_t launch_gated_recurrence_bwd(const RecurrenceArgs &a, void *workspace, hipStream_t stream) {
    return a.io == IO_F32 ? bwd<float, 1>(a, workspace, stream) : bwd<uint16_t, 2>(a, workspace, stream);
}

hipError_t recurrence_status(uint32_t *bits, bool clear) {
    void *p = nullptr;
    hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(g_recurrence_status_bits));
    if (e == hipSuccess) e = hipDeviceSynchronize();
    if (e == hipSuccess) e = hipMemcpy(bits, p, sizeof(uint32_t), hipMemcpyDeviceToHost);
    if (e == hipSuccess && clear) {
        const uint32_t zero = 0;
        e = hipMemcpy(p, &zero, sizeof(uint32_t), hipMemcpyHostToDevice);
    }
    return e;
}

}  // namespace mssm
